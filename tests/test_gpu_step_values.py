"""A server's steps through plan_step, norm_rope_store and paged_decode_shared_attn, value by value:
the stored keys against the float64 oracle within norm_rope_store's bound, then attention against
plain attention in 64 bits over the very keys and values that were stored, within the bound of
paged_decode_shared_attn.  Each check also has to refuse outputs that are wrong in the ways such a
step can go wrong, so that its bounds are known to be narrow enough."""
import numpy as np
import pytest
import torch

from gpu_util import assert_close
from test_gpu_decode_shared import Shared
from test_gpu_norm_rope import Rows, f64, frequencies

pytestmark = pytest.mark.gpu

HQ, HKV, D, BS = 8, 2, 64, 64
SCALE = D**-0.5


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


class Server:
    """Caches (NaN where no token is), norm weights, and each sequence's stored keys and values, bit for bit."""

    def __init__(self, lib, blocks, seed=0):
        self.lib = lib
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *s: torch.randn(*s, generator=self.gen, device="cuda")
        self.qw, self.kw = (torch.exp(0.2 * normal(D)).to(torch.bfloat16) for _ in range(2))
        self.freq = frequencies(D)
        self.turns = lib.rope_turns(self.freq)
        self.kc = torch.full((blocks, BS, HKV, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.vc = self.kc.clone()
        self.held = {}

    def projections(self, rows):
        return torch.randn(rows, HQ + 2 * HKV, D, generator=self.gen, device="cuda").to(torch.bfloat16)

    @staticmethod
    def parts(x):
        return x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:]

    def store(self, x, positions, slots, q_out=None, **more):
        q, k, v = self.parts(x)
        q_out = torch.empty(len(x), HQ, D, dtype=torch.bfloat16, device="cuda") if q_out is None else q_out
        self.lib.norm_rope_store(q_out, q, k, v, positions, self.turns, self.kc, self.vc, slots, q_weight=self.qw, k_weight=self.kw, **more)
        return q_out

    def tokens(self, row, first, last):
        """K and V of the tokens [first, last) by a row of the block tables."""
        p = torch.arange(first, last, device="cuda")
        slots = torch.as_tensor(np.asarray(row), device="cuda").long()[p // BS] * BS + p % BS
        return self.kc.flatten(0, 1)[slots], self.vc.flatten(0, 1)[slots]

    def stored(self, seq, row, x, positions, q_out):
        """The rows x of a sequence are where its table says, within the bound, and what it held is as it was."""
        at = Rows.__new__(Rows)
        at.positions, at.inv_freq = torch.as_tensor(np.asarray(positions)), self.freq
        q, k, v = self.parts(x)
        first = int(positions[0])
        ck, cv = self.tokens(row, first, first + len(x))
        for got, src, weight in ((q_out, q, self.qw), (ck, k, self.kw)):
            want, bound = at.want(src, f64(weight))
            assert bool((np.abs(f64(got) - want) <= bound).all()), seq
            assert not bool((np.abs(f64(got) - np.roll(want, 1, axis=0 if len(x) > 1 else -1)) <= bound).all())
        assert torch.equal(cv.view(torch.int16), v.view(torch.int16)), seq
        if first > 0:
            hk, hv = self.tokens(row, 0, first)
            assert torch.equal(hk, self.held[seq][0]) and torch.equal(hv, self.held[seq][1]), seq
            ck, cv = torch.cat([hk, ck]), torch.cat([hv, cv])
        self.held[seq] = ck, cv

    def attention(self, seq, q, n, begin=0):
        """Plain attention in 64 bits over the sequence's tokens [begin, n), and the bound of paged_decode_shared_attn."""
        s = Shared.__new__(Shared)
        k, v = (x[begin:n] for x in self.held[seq])
        s.Hq, s.Hkv, s.D, s.block, s.scale = HQ, HKV, D, n - begin, SCALE
        s.kc, s.vc, s.q, s.ctx, s.tables = k[None], v[None], q[None], [n - begin], np.zeros((1, 1), np.int64)
        return s.want(0)

    def attended(self, seq, out, q, prefix=0):
        n = len(self.held[seq][0])
        want, bound = self.attention(seq, q, n)
        inside = lambda x: bool(((x.double() - want).abs() <= bound).all())
        assert inside(out), (seq, n)
        # the bounds tell these from what is right
        assert not inside(torch.zeros_like(out))
        assert not inside(torch.roll(out, 1, 0))  # (another head's)
        if n > 1:
            assert not inside(self.attention(seq, q, n - 1)[0]), "without the newest token"
        if 0 < prefix < n:
            assert not inside(self.attention(seq, q, n, prefix)[0]), "without the prefix"
            assert not inside(self.attention(seq, q, prefix)[0]), "without the tail"


def test_a_server_with_the_block_manager(lib):
    """Prompts that begin alike, admitted by the host's manager, then decode steps in groups."""
    m = Server(lib, 80)
    bm = lib.BlockManager(80, BS)
    rng = np.random.default_rng(3)
    system, other = rng.integers(0, 1000, 3 * BS + 10).tolist(), rng.integers(0, 1000, 2 * BS).tolist()
    prompts = {10: system + [1, 2, 3], 11: system + list(range(90)), 12: other + [5], 13: system + [7], 14: rng.integers(0, 1000, 30).tolist(), 15: other + [6] * 70}
    prefix = {10: 3 * BS, 11: 3 * BS, 12: 2 * BS, 13: 3 * BS, 15: 2 * BS}
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for seq, tokens in prompts.items():
        cached = bm.allocate(seq, tokens)
        n = len(tokens) - cached
        row, x, positions = bm.block_table(seq, 8), m.projections(n), np.arange(cached, len(tokens))
        if cached:  # what it found there: the tokens of an earlier sequence
            m.held[seq] = m.tokens(row, 0, cached)
        q_out = m.store(x, i32(positions), i32(bm.slots(seq, cached, n)), dev_status=status)
        out = torch.empty_like(q_out)
        lib.paged_prefill_attn(out, q_out, m.kc, m.vc, i32([row]), i32([0, n]), i32([0, len(tokens)]), n, SCALE, dev_status=status)
        torch.cuda.synchronize()
        m.stored(seq, row, x, positions, q_out)
        for i in (0, n // 2, n - 1):
            assert_close(out[i].double().cpu().numpy(), m.attention(seq, q_out[i], cached + i + 1)[0].cpu().numpy())
    ids = list(prompts)
    for step in range(70):  # (over a border of the blocks)
        for seq in ids:
            bm.append(seq, 2000 + step)
        order, starts, shared = bm.prefix_groups(ids)
        assert sorted(zip(np.diff(starts).tolist(), shared.tolist())) == [(1, 0), (2, 2), (3, 3)]
        batch = [ids[i] for i in order]
        lens = [bm.num_tokens(s) for s in batch]
        rows = [bm.block_table(s, 8) for s in batch]
        x = m.projections(len(batch))
        q_out = m.store(x, i32(lens) - 1, i32([int(bm.slots(s, n - 1, 1)[0]) for s, n in zip(batch, lens)]), dev_status=status)
        out = torch.empty_like(q_out)
        ws = lib.decode_shared_workspace(len(batch), len(shared), HQ, HKV, D)
        lib.test_shared_fault(10**9, -1, step % 2)
        try:
            lib.paged_decode_shared_attn(out, q_out, m.kc, m.vc, i32(rows), i32(lens), i32(starts), i32(shared), SCALE, ws, dev_status=status)
            torch.cuda.synchronize()
        finally:
            lib.test_shared_fault(10**9, -1, 0)
        assert int(status.item()) == 0
        for i, seq in enumerate(batch):
            m.stored(seq, rows[i], x[i:i + 1], [lens[i] - 1], q_out[i:i + 1])
            m.attended(seq, out[i], q_out[i], prefix.get(seq, 0))


@pytest.mark.parametrize("groups,steps", [([3, 1, 1], 150), ([40, 1, 130, 100, 1, 1, 50], 70)])
@pytest.mark.parametrize("sharing", ["as it pays", "always"])
def test_a_captured_step(lib, sharing, groups, steps):
    """One graph of plan, rotation with its store, and attention, replayed step after step: sequences grow out of their blocks,
    pause, end and begin anew behind their group's prefix (groups of one have none)."""
    lib.test_shared_fault(10**9, -1, int(sharing == "always"))
    try:
        captured_step(lib, groups, steps)
    finally:
        lib.test_shared_fault(10**9, -1, 0)


def captured_step(lib, members, steps):
    S, wide, prefix = sum(members), 8, 2
    fixed = prefix * len(members)  # blocks of the prefixes
    blocks = fixed + 4 * S
    m = Server(lib, blocks, seed=S)
    group = np.repeat(np.arange(len(members)), members)
    shares = [members[g] > 1 for g in group]
    begin = [prefix * BS if x else 0 for x in shares]
    tables = np.full((S, wide), -1, np.int32)
    n = prefix * BS
    heads = {}
    for g, size in enumerate(members):
        if size > 1:
            row = np.arange(g * prefix, (g + 1) * prefix)
            tables[group == g, :prefix] = row
            x = m.projections(n)
            q_out = m.store(x, i32(np.arange(n)), i32(np.repeat(row, BS) * BS + np.arange(n) % BS))
            m.stored(("prefix", g), row, x, np.arange(n), q_out)
            heads[g] = m.held[("prefix", g)]
    t = dict(new_lens=i32([1] * S), context_lens=i32(begin), block_tables=i32(tables), free_blocks=i32(np.arange(fixed, blocks)), num_free=i32([blocks - fixed]))
    rows = S + 2  # padded
    slots, positions, cu_q, cu_k = i32([0] * rows), i32([0] * rows), i32([0] * (S + 1)), i32([0] * (S + 1))
    borrowed = i32([prefix if x else 0 for x in shares])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    px = torch.zeros(rows, HQ + 2 * HKV, D, dtype=torch.bfloat16, device="cuda")
    q_out = torch.empty(rows, HQ, D, dtype=torch.bfloat16, device="cuda")
    q_seq = torch.zeros(S, HQ, D, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q_seq)
    row_of = torch.zeros(S, dtype=torch.long, device="cuda")
    starts, shared = i32(np.concatenate([[0], np.cumsum(members)])), i32([prefix if x > 1 else 0 for x in members])
    ws = lib.decode_shared_workspace(S, len(members), HQ, HKV, D)

    def step():
        lib.plan_step(t["new_lens"], t["context_lens"], t["block_tables"], t["free_blocks"], t["num_free"], t["context_lens"], t["num_free"], slots,
                      positions, cu_q, cu_k, blocks, BS, borrowed_blocks=borrowed, dev_status=status)
        m.store(px, positions, slots, q_out=q_out, dev_status=status)
        torch.clamp(cu_q[:-1].long(), max=rows - 1, out=row_of)
        torch.index_select(q_out, 0, row_of, out=q_seq)
        lib.paged_decode_shared_attn(out, q_seq, m.kc, m.vc, t["block_tables"], t["context_lens"], starts, shared, SCALE, ws, dev_status=status)

    kept = {k: v.clone() for k, v in t.items()}
    caches = m.kc.clone(), m.vc.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        for k, v in kept.items():
            t[k].copy_(v)
        m.kc.copy_(caches[0]), m.vc.copy_(caches[1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    status.zero_()
    lens = list(begin)

    def restart(s):
        m.held.pop(s, None)
        if shares[s]:
            m.held[s] = heads[group[s]]

    for s in range(S):
        restart(s)
    rng = np.random.default_rng(S)
    for it in range(steps):
        new = [int(x) for x in rng.choice([1, 1, 1, 1, 0], S)]
        ended = None
        if it % 30 == 29:  # one ends; in the next step it begins anew
            ended = it // 30 * 7 % S
            new[ended] = -1
        t["new_lens"].copy_(i32(new))
        y = m.projections(rows)
        px.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        table = t["block_tables"].cpu().numpy()
        look = set(range(S)) if S < 10 else {int(s) for s in rng.choice(S, 6)} | {0, S - 1}
        at = 0
        for s in range(S):
            if new[s] == 1:
                if s in look:
                    m.stored(s, table[s], y[at:at + 1], [lens[s]], q_out[at:at + 1])
                else:
                    k, v = m.tokens(table[s], lens[s], lens[s] + 1)
                    m.held[s] = tuple(torch.cat([a, b]) for a, b in zip(m.held[s], (k, v))) if lens[s] else (k, v)
                lens[s] += 1
                at += 1
            elif new[s] == -1:
                lens[s] = 0
        assert t["context_lens"].tolist() == lens
        if all(lens):
            assert int(status.item()) == 0
        status.zero_()
        if it % 5 == 0 or it > steps - 6 or ended is not None:
            for s in look:
                if lens[s] > 0 and new[s] == 1:
                    m.attended(s, out[s], q_seq[s], begin[s])
        if ended is not None:
            lens[ended] = begin[ended]
            t["context_lens"].copy_(i32(lens))  # (its prefix is in its row still)
            restart(ended)
    assert t["num_free"].item() == blocks - fixed - sum(-(-n // BS) - (prefix if x else 0) for n, x in zip(lens, shares))
