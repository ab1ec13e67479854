"""A server's steps through plan_step, norm_rope_store and paged_decode_shared_attn together, beside
the block manager, prefill and plain decode, against plain attention in 64 bits over each sequence's
own tokens.  (Bounds as in test_gpu_norm_rope and test_gpu_decode_shared.)"""
import numpy as np
import pytest
import torch

from oracle import steps
from test_gpu_decode_shared import HALF_STEP
from test_gpu_norm_rope import f64, frequencies

pytestmark = pytest.mark.gpu

HQ, HKV, D, BS = 8, 2, 64, 64
SCALE = D**-0.5
FREQ = frequencies(D)


class Model:
    """Projections of random activations, norm weights, and every sequence's keys and values so far as the cache is to hold them."""

    def __init__(self, lib, blocks, seed=0):
        self.lib = lib
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *s: torch.randn(*s, generator=self.gen, device="cuda")
        self.qw, self.kw = (torch.exp(0.2 * normal(D)).to(torch.bfloat16) for _ in range(2))
        self.turns = lib.rope_turns(FREQ)
        self.kc = torch.full((blocks, BS, HKV, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.vc = self.kc.clone()
        self.keys, self.values = {}, {}

    def projections(self, rows):
        x = torch.randn(rows, HQ + 2 * HKV, D, generator=self.gen, device="cuda").to(torch.bfloat16)
        return x

    @staticmethod
    def parts(x):
        return x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:]

    def rotated(self, x, weight, positions):
        want = steps.norm_rope(f64(x), positions, FREQ, f64(weight))
        return torch.from_numpy(want)

    def store(self, seq, x, positions):
        """What the rows of x [n, ...] at these positions are to add to the sequence, in 64 bits of the bf16 that the call is to store."""
        _, k, v = self.parts(x)
        k = self.rotated(k, self.kw, positions)
        self.keys.setdefault(seq, []).append(k)
        self.values.setdefault(seq, []).append(v.double().cpu())

    def attention(self, seq, q, n=None):
        """softmax(q K^T) V over the sequence's first n tokens; K as computed, so to its rounding to bf16."""
        k, v = (torch.cat(x[seq])[:n] for x in (self.keys, self.values))
        k = k.to(torch.bfloat16).double()
        z = torch.einsum("jgd,pjd->jgp", q.double().cpu().view(HKV, -1, D), k) * SCALE
        w = torch.softmax(z, -1)
        return torch.einsum("jgp,pjd->jgd", w, v).view(HQ, D), w, v

    def check(self, seq, got, q, n=None):
        want, w, v = self.attention(seq, q, n)
        # A key's bf16 may round the other way where its value is near the middle of a step: then it is off by a
        # whole step, 2 * HALF_STEP of itself, and its logit by |scale| |q| |k| times that.
        k = torch.cat(self.keys[seq])
        e = 2 * HALF_STEP * SCALE * q.double().cpu().norm(dim=-1).max() * k.norm(dim=-1).max()
        bound = HALF_STEP * want.abs() + (2 * e + 2.0**-12) * v.abs().max()
        err = (got.double().cpu() - want).abs()
        assert bool((err <= bound).all()), (seq, float((err / bound).nan_to_num(1e30).max()))


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def test_a_server_with_the_block_manager(lib):
    """Prompts that begin alike: admitted by the host's manager, their new tokens stored and attended, then decode steps in groups."""
    m = Model(lib, 80)
    bm = lib.BlockManager(80, BS)
    rng = np.random.default_rng(3)
    system, other = rng.integers(0, 1000, 3 * BS + 10).tolist(), rng.integers(0, 1000, 2 * BS).tolist()
    prompts = {10: system + [1, 2, 3], 11: system + list(range(90)), 12: other + [5], 13: system + [7], 14: rng.integers(0, 1000, 30).tolist(), 15: other + [6] * 70}
    # token by token the same activations: prefixes that are the same have the same rows
    rows = {}

    def row(seq, pos, tokens):
        key = tuple(tokens[: pos + 1])
        if key not in rows:
            rows[key] = m.projections(1)
        return rows[key]

    for seq, tokens in prompts.items():
        cached = bm.allocate(seq, tokens)
        x = torch.cat([row(seq, p, tokens) for p in range(len(tokens))])
        m.store(seq, x, np.arange(len(tokens)))
        new = x[cached:]
        q, k, v = m.parts(new)
        n, slots = len(tokens) - cached, bm.slots(seq, cached, len(tokens) - cached)
        q_out = torch.empty(n, HQ, D, dtype=torch.bfloat16, device="cuda")
        lib.norm_rope_store(q_out, q, k, v, i32(np.arange(cached, len(tokens))), m.turns, m.kc, m.vc, i32(slots), q_weight=m.qw, k_weight=m.kw)
        out = torch.empty_like(q_out)
        lib.paged_prefill_attn(out, q_out, m.kc, m.vc, i32([bm.block_table(seq, 8)]), i32([0, n]), i32([0, len(tokens)]), n, SCALE)
        torch.cuda.synchronize()
        for i in (0, n // 2, n - 1):
            m.check(seq, out[i], q_out[i], cached + i + 1)
    assert bm.allocate(99, prompts[10]) > 0 and (bm.free(99) or True)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids = list(prompts)
    for step in range(5):
        for seq in ids:
            bm.append(seq, 2000 + step)
        order, starts, shared = bm.prefix_groups(ids)
        batch = [ids[i] for i in order]
        assert sorted(zip(np.diff(starts).tolist(), shared.tolist())) == [(1, 0), (2, 2), (3, 3)]
        lens = [bm.num_tokens(s) for s in batch]
        x = m.projections(len(batch))
        q, k, v = m.parts(x)
        for i, seq in enumerate(batch):
            m.store(seq, x[i:i + 1], [lens[i] - 1])
        q_out = torch.empty(len(batch), HQ, D, dtype=torch.bfloat16, device="cuda")
        slots = [int(bm.slots(s, n - 1, 1)[0]) for s, n in zip(batch, lens)]
        lib.norm_rope_store(q_out, q, k, v, i32(lens) - 1, m.turns, m.kc, m.vc, i32(slots), q_weight=m.qw, k_weight=m.kw, dev_status=status)
        out = torch.empty_like(q_out)
        ws = lib.decode_shared_workspace(len(batch), len(shared), HQ, HKV, D)
        lib.paged_decode_shared_attn(out, q_out, m.kc, m.vc, i32([bm.block_table(s, 8) for s in batch]), i32(lens), i32(starts), i32(shared), SCALE, ws,
                                     dev_status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        for i, seq in enumerate(batch):
            m.check(seq, out[i], q_out[i])


@pytest.mark.parametrize("sharing", ["as it pays", "always"])
def test_a_captured_step(lib, sharing):
    """One graph of plan, rotation with its store, and attention, replayed step after step: sequences grow out of their blocks,
    pause, end and begin anew behind a prefix that the block manager holds."""
    lib.test_shared_fault(10**9, -1, int(sharing == "always"))
    try:
        _captured_step(lib)
    finally:
        lib.test_shared_fault(10**9, -1, 0)


def _captured_step(lib):
    S, wide, blocks, prefix = 5, 8, 60, 2  # (the last two rows of the batch share nothing)
    m = Model(lib, blocks, seed=1)
    bm = lib.BlockManager(20, BS)  # the pool's first 20 blocks: prefixes
    bm.allocate(0, list(range(prefix * BS)))
    x = m.projections(prefix * BS)
    q, k, v = m.parts(x)
    head = bm.block_table(0, prefix)
    lib.norm_rope_store(torch.empty(prefix * BS, HQ, D, dtype=torch.bfloat16, device="cuda"), q, k, v, i32(np.arange(prefix * BS)), m.turns, m.kc, m.vc,
                        i32(bm.slots(0, 0, prefix * BS)), q_weight=m.qw, k_weight=m.kw)
    shares = [True, True, True, False, False]
    begin = [prefix * BS if s else 0 for s in shares]

    def restart(s):
        m.keys.pop(s, None), m.values.pop(s, None)
        if shares[s]:
            m.store(s, x, np.arange(prefix * BS))

    tables = np.full((S, wide), -1, np.int32)
    tables[:3, :prefix] = head
    t = dict(new_lens=i32([1] * S), context_lens=i32(begin), block_tables=i32(tables), free_blocks=i32(np.arange(20, blocks)), num_free=i32([blocks - 20]))
    rows = S + 2  # padded
    out_of = dict(slot_mapping=i32([0] * rows), positions=i32([0] * rows), cu_seqlens_q=i32([0] * (S + 1)), cu_seqlens_k=i32([0] * (S + 1)))
    borrowed = i32([prefix if s else 0 for s in shares])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    px = torch.zeros(rows, HQ + 2 * HKV, D, dtype=torch.bfloat16, device="cuda")
    q_out = torch.empty(rows, HQ, D, dtype=torch.bfloat16, device="cuda")
    q_seq = torch.zeros(S, HQ, D, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q_seq)
    row_of = torch.zeros(S, dtype=torch.long, device="cuda")
    ws = lib.decode_shared_workspace(S, 3, HQ, HKV, D)

    def step():
        lib.plan_step(t["new_lens"], t["context_lens"], t["block_tables"], t["free_blocks"], t["num_free"], t["context_lens"], t["num_free"],
                      out_of["slot_mapping"], out_of["positions"], out_of["cu_seqlens_q"], out_of["cu_seqlens_k"], blocks, BS, borrowed_blocks=borrowed,
                      dev_status=status)
        q, k, v = m.parts(px)
        lib.norm_rope_store(q_out, q, k, v, out_of["positions"], m.turns, m.kc, m.vc, out_of["slot_mapping"], q_weight=m.qw, k_weight=m.kw, dev_status=status)
        torch.clamp(out_of["cu_seqlens_q"][:-1].long(), max=rows - 1, out=row_of)
        torch.index_select(q_out, 0, row_of, out=q_seq)
        lib.paged_decode_shared_attn(out, q_seq, m.kc, m.vc, t["block_tables"], t["context_lens"], groups, shared, SCALE, ws, dev_status=status)

    groups, shared = i32([0, 3, 4, 5]), i32([prefix, 0, 0])
    kept = {k: v.clone() for k, v in t.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        for k, v in kept.items():
            t[k].copy_(v)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    status.zero_()
    lens = list(begin)
    for s in range(S):
        restart(s)
    rng = np.random.default_rng(8)
    for it in range(150):
        new = [int(n) for n in rng.choice([1, 1, 1, 1, 0], S)]
        ended = None
        if it % 40 == 39:  # one ends; in the next step it begins anew
            ended = it // 40 % S
            new[ended] = -1
        t["new_lens"].copy_(i32(new))
        y = m.projections(rows)
        px.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        at = 0
        for s in range(S):
            if new[s] == 1:
                m.store(s, y[at:at + 1], [lens[s]])
                lens[s] += 1
                at += 1
            elif new[s] == -1:
                lens[s] = 0
        assert t["context_lens"].tolist() == lens
        if all(lens):
            assert int(status.item()) == 0
        status.zero_()
        if it % 7 == 0 or it > 140 or ended is not None:
            for s in range(S):
                if lens[s] > 0 and new[s] == 1:
                    m.check(s, out[s], q_seq[s])
        if ended is not None:
            lens[ended] = begin[ended]
            t["context_lens"].copy_(i32(lens))  # (its prefix is in its row still)
            restart(ended)
    assert t["num_free"].item() == blocks - 20 - sum(-(-n // BS) - (prefix if s else 0) for n, s in zip(lens, shares))
