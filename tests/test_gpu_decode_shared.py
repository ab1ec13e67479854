"""paged_decode_shared_attn on the GPU against plain attention in 64 bits, sequence by sequence.

Tolerances, derived: a logit is scale times a sum of D products that are exact in fp32, summed
in fp32 in some order, each of the D additions off by at most 2^-23 (the tensor cores may
truncate) of the sum of magnitudes A <= |q| |k|, so the logit by e = |scale| A D 2^-23; the
product with log2(e) and its subtraction from the maximum by 2^-22 of |z| <= |scale| A, which e
covers from D = 8 on.  A weight exp(z - log sum) is then off by 2 e of itself, and by 2^-17 for
its two bf16 terms, a few 2^-22 for exponentials and the sums' positive terms: r = 2 e + 2^-16.
The output sum_p w_p v_p with both its weights and their sum off by r is off by 2 r max|v|, plus
the products' own accumulation, at most 2^-23 per key of max|v| w_p: n terms, and the joining of
parts, 2^-16 of max|v| for up to 128 keys in one accumulator's run between additions of parts of
equal size; that is bounded by K 2^-23 max|v|, K the keys of the context, as every one of the K
additions is off by 2^-23 of a partial sum of at most max|v| at most.  One rounding to bf16 ends
it, off by at most eps / 2 = 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import bits

pytestmark = pytest.mark.gpu

HALF_STEP = torch.finfo(torch.bfloat16).eps / 2


@pytest.fixture(autouse=True)
def share(request, lib):
    """Prefixes are shared however short (most of these are far too short to pay), but in tests of the choice."""
    always = not request.node.get_closest_marker("by_choice")
    lib.test_shared_fault(10**9, -1, int(always))
    yield
    lib.test_shared_fault(10**9, -1, 0)


class Shared:
    """groups: (shared blocks, [tokens behind them, one number per sequence]); a tail of None: an empty context."""

    def __init__(self, groups, Hq, Hkv, D, block=64, seed=0, k_size=1.0, scale=None, spare=2, poison=True, wide=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.Hq, self.Hkv, self.D, self.block = Hq, Hkv, D, block
        self.scale = D**-0.5 if scale is None else scale
        ctx, starts, shared = [], [0], []
        for blocks, tails in groups:
            ctx += [0 if t is None else blocks * block + t for t in tails]
            starts.append(len(ctx))
            shared.append(blocks)
        need = [-(-L // block) for L in ctx]
        own = [max(0, n - shared[gi]) for gi, (_, tails) in enumerate(groups) for n in [need[starts[gi] + i] for i in range(len(tails))]]
        NB = sum(shared) + sum(own) + spare
        pages = torch.randperm(NB, generator=g, device="cuda").cpu().numpy().astype(np.int32)
        tables = np.full((len(ctx), max(need + [1]) + wide), -1, np.int32)
        at = 0
        for gi, blocks in enumerate(shared):
            for s in range(starts[gi], starts[gi + 1]):
                if ctx[s] > 0:
                    tables[s, :blocks] = pages[at:at + blocks]
            at += blocks
            for s in range(starts[gi], starts[gi + 1]):
                k = own[s]
                tables[s, blocks:blocks + k] = pages[at:at + k]
                at += k
        self.ctx, self.starts, self.shared, self.tables = ctx, starts, shared, tables
        normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")
        self.kc = (k_size * normal(NB, block, Hkv, D)).to(torch.bfloat16)
        self.vc = normal(NB, block, Hkv, D).to(torch.bfloat16)
        self.q = normal(len(ctx), Hq, D).to(torch.bfloat16)
        if poison:  # slots that hold no token of the batch may hold anything
            held = torch.zeros(NB, block, dtype=torch.bool, device="cuda")
            for s, L in enumerate(ctx):
                for b in range(need[s]):
                    held[int(tables[s, b]), :min(block, L - b * block)] = True
            self.kc[~held] = float("nan")
            self.vc[~held] = float("nan")
        self.out = torch.full((len(ctx), Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def args(self, pkv, **more):
        i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")
        a = dict(out=self.out, q=self.q, k_cache=self.kc, v_cache=self.vc, block_tables=i32(self.tables), context_lens=i32(self.ctx),
                 group_starts=i32(self.starts), shared_blocks=i32(self.shared), scale=self.scale, dev_status=self.status)
        a.update(more)
        if "workspace" not in a:
            a["workspace"] = pkv.decode_shared_workspace(len(self.ctx), a["shared_blocks"].numel(), self.Hq, self.Hkv, self.D)
            a["workspace"].fill_(255)  # (needs no initialisation: as NaN)
        return a

    def want(self, s):
        """out of sequence s in 64 bits, and the bound on what it may be off."""
        L = min(self.ctx[s], self.tables.shape[1] * self.block)
        blocks = torch.as_tensor(self.tables[s, :-(-L // self.block)].astype(np.int64), device="cuda")
        k = self.kc[blocks].reshape(-1, self.Hkv, self.D)[:L].double()
        v = self.vc[blocks].reshape(-1, self.Hkv, self.D)[:L].double()
        q = self.q[s].double().view(self.Hkv, -1, self.D)
        z = torch.einsum("jgd,pjd->jgp", q, k) * self.scale
        w = torch.exp(z - z.amax(-1, keepdim=True))
        w = w / w.sum(-1, keepdim=True)
        out = torch.einsum("jgp,pjd->jgd", w, v)
        A = q.norm(dim=-1).amax() * k.norm(dim=-1).amax()
        r = 2 * abs(self.scale) * A * self.D * 2.0**-23 + 2.0**-16
        vmax = v.abs().amax()
        bound = HALF_STEP * out.abs() + (2 * r + L * 2.0**-23) * vmax
        return out.view(self.Hq, self.D), bound.view(self.Hq, self.D)

    def compare(self, only=None):
        for s, L in enumerate(self.ctx):
            if only is not None and s not in only:
                continue
            if L <= 0:
                assert (self.out[s] == 7.0).all(), s
                continue
            want, bound = self.want(s)
            err = (self.out[s].double() - want).abs()
            assert bool((err <= bound).all()), (s, L, float((err / bound).nan_to_num(1e30).max()), self.out[s].isnan().any())

    def check(self, pkv, status=0, **more):
        pkv.paged_decode_shared_attn(**self.args(pkv, **more))
        torch.cuda.synchronize()
        assert int(self.status.item()) == status
        self.compare()
        return self


@pytest.mark.parametrize("block", [64, 256])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (4, 2), (4, 1), (16, 2)])
def test_two_sequences(lib, Hq, Hkv, D, block):
    Shared([(1, [1, 70])], Hq, Hkv, D, block).check(lib)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("members", [3, 17, 33, 130])
def test_rows_of_a_group(lib, members, G, D):
    """Up to more rows than a unit has (256): parts of a row tile, two of them, several units."""
    tails = [(37 * i) % 150 for i in range(members)]
    Shared([(5, tails)], 2 * G, 2, D, seed=members).check(lib)


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("Hq,Hkv,D,block", [(16, 8, 128, 256), (8, 1, 64, 128), (12, 3, 128, 64), (5, 5, 64, 512)])
def test_random_groups(lib, seed, Hq, Hkv, D, block):
    rng = np.random.default_rng(seed)
    groups = []
    for _ in range(rng.integers(1, 9)):
        blocks = int(rng.choice([0, 0, 1, 2, 5, 9]))
        tails = [int(t) for t in rng.integers(0, 3 * block, rng.integers(1, 12))]
        groups.append((blocks, [t if blocks or t else 1 for t in tails]))
    Shared(groups, Hq, Hkv, D, block, seed=seed).check(lib)


def test_no_tail_at_all(lib):
    """Every context ends where the shared blocks do."""
    Shared([(3, [0, 0, 0]), (1, [0, 0])], 8, 2, 128).check(lib)


def test_nothing_shared(lib):
    Shared([(0, [1]), (0, [300]), (0, [64]), (2, [5]), (0, [9, 65])], 4, 2, 64).check(lib)


def test_one_sequence(lib):
    Shared([(4, [100])], 4, 2, 128).check(lib)
    Shared([(0, [1])], 8, 1, 64).check(lib)


def test_a_long_prefix(lib):
    Shared([(300, [5, 0, 77])], 2, 1, 128, 64).check(lib)
    Shared([(40, [5, 1000, 77, 1])], 16, 2, 64, 512).check(lib)


def test_many_small_groups(lib):
    """More units than CTAs: runs that go through several of them, groups with and without a prefix."""
    groups = [((i * 7) % 4, [(i * 13 + j * 29) % 90 + 1 for j in range(1 + i % 5)]) for i in range(150)]
    Shared(groups, 6, 3, 64, 64).check(lib)


def test_the_most_sequences(lib):
    groups = [(1, [i % 7, 1]) for i in range(4096)]
    Shared(groups, 1, 1, 64, 64, poison=False).check(lib)


def test_one_group_of_the_most_sequences(lib):
    s = Shared([(2, [i % 5 for i in range(8192)])], 2, 1, 64, 64, poison=False)
    lib.paged_decode_shared_attn(**s.args(lib))
    torch.cuda.synchronize()
    assert int(s.status.item()) == 0
    s.compare(only=set(range(0, 8192, 61)) | {8191})


@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-30, 2.0])
def test_scales(lib, scale):
    Shared([(4, [10, 0, 130]), (0, [33])], 8, 2, 128, scale=scale, k_size=0.5).check(lib)


def test_peaked_logits(lib):
    """Logits up to a few hundred: maxima that grow along the prefix, so that sums and outputs are rescaled."""
    s = Shared([(8, [10, 0, 130]), (3, [33, 2])], 8, 2, 128, k_size=6.0)
    first = torch.as_tensor(s.tables[0, :8].astype(np.int64), device="cuda")
    grow = torch.linspace(0.05, 1.0, 8, device="cuda").view(8, 1, 1, 1)
    s.kc[first] = (s.kc[first].float() * grow).to(torch.bfloat16)
    s.check(lib)


@pytest.mark.parametrize("D", [64, 128])
def test_weights_keep_more_bits_than_one_bf16(lib, D):
    """Values that nearly cancel under nearly equal weights: what one rounding of a weight to bf16 would leave is seen."""
    s = Shared([(4, [0, 3, 64])], 8, 2, D, k_size=0.01)
    s.vc *= 0.001
    sign = torch.where(torch.arange(s.block, device="cuda") % 2 == 0, 1000.0, -1000.0).view(1, -1, 1, 1)
    s.vc += sign.to(torch.bfloat16)
    s.check(lib)


def test_minus_infinity_among_the_keys(lib):
    """Logits of -inf (a key of infinities against a query of one sign) weigh nothing; a whole first step of them either."""
    s = Shared([(3, [20, 5]), (0, [70])], 2, 1, 64, 64)
    s.q.abs_()
    first = int(s.tables[0, 0])
    s.kc[first, :, :, :] = float("-inf")
    last = int(s.tables[2, 0])
    s.kc[last, 3] = float("-inf")
    lib.paged_decode_shared_attn(**s.args(lib))
    torch.cuda.synchronize()
    finite = s.kc.clone()
    for i, L in enumerate(s.ctx):
        blocks = torch.as_tensor(s.tables[i, :-(-L // 64)].astype(np.int64), device="cuda")
        k = finite[blocks].reshape(-1, 64)[:L].double()
        v = s.vc[blocks].reshape(-1, 64)[:L].double()
        z = (s.q[i].double() @ torch.where(torch.isinf(k), 0.0, k).T) * s.scale
        z[:, torch.isinf(k).any(1)] = float("-inf")
        want = torch.softmax(z, -1) @ v
        # (the bound of the finite keys: |q| |k| <= 64 * 12 for these draws, D = 64)
        assert ((s.out[i].double() - want).abs() <= HALF_STEP * want.abs() + 2 * (2 * 0.125 * 768 * 64 * 2.0**-23 + 2.0**-15) * v.abs().max()).all()


def test_empty_contexts_take_no_part(lib):
    """Rows that pad a batch: the first of a group, the last, all but one, a whole group."""
    s = Shared([(2, [None, 5, 70]), (3, [4, None, 9, None]), (2, [None, 7]), (1, [None, None]), (0, [None, 3])], 4, 2, 64)
    s.check(lib, status=lib.DEV_BAD_CONTEXT)


def test_a_group_shares_what_its_shortest_context_fills(lib):
    s = Shared([(5, [3, 100, 0, 64])], 8, 2, 128, poison=False)
    s.ctx[2] = 2 * 64 + 17
    s.check(lib)
    s.ctx[2] = 40  # not even one block
    s.check(lib)


def test_contexts_longer_than_their_table_are_clamped(lib):
    s = Shared([(2, [64, 64, 10])], 4, 2, 64, 64)
    s.ctx[1] = 10**6
    s.check(lib, status=lib.DEV_BAD_CONTEXT)


@pytest.mark.parametrize("shared", [[-1, 2], [3, 1000]])
def test_bad_numbers_of_shared_blocks(lib, shared):
    s = Shared([(3, [4, 70]), (2, [5, 9, 30])], 4, 2, 64, poison=False)
    s.shared = shared
    if shared[1] > 2:  # taken as what the table holds, then as what the shortest context fills: 2 blocks
        s.ctx = [L if i < 2 else 2 * 64 + (L % 64) for i, L in enumerate(s.ctx)]
    s.check(lib, status=lib.DEV_BAD_CONTEXT)


@pytest.mark.parametrize("starts", [[1, 2, 5], [0, 2, 4], [0, 6, 5], [0, -3, 5], [5, 2, 0]])
def test_bad_groups_are_attended_one_by_one(lib, starts):
    s = Shared([(3, [4, 70]), (2, [5, 9, 30])], 4, 2, 64)
    s.starts = starts
    s.check(lib, status=lib.DEV_BAD_SEQLEN)


def test_block_ids_out_of_range_are_flagged(lib):
    s = Shared([(2, [4, 70]), (2, [5, 9]), (0, [30])], 4, 2, 64, poison=False)
    s.tables[0, 1] = s.kc.shape[0]      # of the shared blocks of the first group
    s.tables[3, 2] = -1                 # of one sequence's own
    lib.paged_decode_shared_attn(**s.args(lib))
    torch.cuda.synchronize()
    assert int(s.status.item()) == lib.DEV_BAD_BLOCK
    s.compare(only={2, 4})


def test_the_same_call_gives_the_same_bits(lib):
    s = Shared([(9, [(53 * i) % 400 for i in range(40)]), (0, [777])], 16, 4, 128, 128)
    a = s.args(lib)
    lib.paged_decode_shared_attn(**a)
    torch.cuda.synchronize()
    first = bits(s.out)
    for _ in range(3):
        s.out.fill_(1.0)
        lib.paged_decode_shared_attn(**a)
        torch.cuda.synchronize()
        assert (bits(s.out) == first).all()


def test_against_decode_of_every_sequence(lib):
    """The same batch through paged_decode_attn: two roundings to bf16 apart at most, but for what the bound above allows."""
    s = Shared([(6, [(31 * i) % 300 + 1 for i in range(25)])], 8, 4, 128, 128, poison=False)
    a = s.args(lib)
    lib.paged_decode_shared_attn(**a)
    S, mtb = len(s.ctx), sum(-(-L // 128) for L in s.ctx)
    out = torch.empty_like(s.out)
    lib.paged_decode_attn(out, s.q, s.kc, s.vc, a["block_tables"], a["context_lens"], s.scale, lib.decode_workspace(S, 8, 4, 128, mtb), mtb)
    torch.cuda.synchronize()
    s.compare()
    for i in range(S):
        _, bound = s.want(i)
        assert ((s.out[i].double() - out[i].double()).abs() <= 2 * bound).all()


def test_against_the_oracle(lib):
    s = Shared([(2, [5, 0, 70]), (0, [130])], 4, 2, 64, poison=False).check(lib)
    want = oracle.paged_decode_attn(bits(s.q), bits(s.kc), bits(s.vc), s.tables, np.asarray(s.ctx, np.int32), s.scale)
    for i in range(len(s.ctx)):
        ours, _ = s.want(i)
        np.testing.assert_allclose(ours.cpu().numpy(), want[i], rtol=1e-12, atol=1e-12)


def test_on_streams_and_from_a_graph(lib):
    s = Shared([(6, [(31 * i) % 200 for i in range(20)]), (2, [5, 9])], 8, 2, 128)
    a = s.args(lib)
    lib.paged_decode_shared_attn(**a)
    torch.cuda.synchronize()
    want = bits(s.out)
    # two calls at a time, each with its own workspace and output
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(s.out) for _ in streams]
    spaces = [torch.empty_like(a["workspace"]) for _ in streams]
    for _ in range(5):
        for st, out, ws in zip(streams, outs, spaces):
            lib.paged_decode_shared_attn(**{**a, "out": out, "workspace": ws, "stream": st})
    torch.cuda.synchronize()
    for out in outs:
        assert (bits(out) == want).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.paged_decode_shared_attn(**a)
        lib.paged_decode_shared_attn(**{**a, "out": outs[0]})  # (one after the other: they may share the workspace)
    # replayed on other queries and shorter contexts
    s.q.copy_(torch.randn_like(s.q, dtype=torch.float32).to(torch.bfloat16))
    s.ctx = [L - 1 if L % 64 > 1 else L for L in s.ctx]
    a["context_lens"].copy_(torch.tensor(s.ctx, dtype=torch.int32))
    outs[0].zero_()
    graph.replay()
    torch.cuda.synchronize()
    s.compare()
    assert torch.equal(outs[0], s.out)


def test_behind_other_calls_of_the_library(lib):
    """Between decode, prefill and key-weight calls on one stream, none waited for on the host."""
    s = Shared([(4, [(31 * i) % 200 + 1 for i in range(12)])], 8, 2, 128, poison=False)
    a = s.args(lib)
    S, mtb = len(s.ctx), sum(-(-L // 64) for L in s.ctx)
    ws = lib.decode_workspace(S, 8, 2, 128, mtb)
    wws = lib.decode_weights_workspace(S, 8, 2, 128, 64, mtb)
    kw = torch.zeros(s.kc.shape[0], 2, 64, device="cuda")
    cu_q = torch.arange(S + 1, dtype=torch.int32, device="cuda")
    cu_k = torch.tensor([0, *np.cumsum(s.ctx)], dtype=torch.int32, device="cuda")
    outs = [torch.empty_like(s.out) for _ in range(6)]
    shared = []
    for i in range(3):
        lib.paged_prefill_attn(outs[0], s.q, s.kc, s.vc, a["block_tables"], cu_q, cu_k, 1, s.scale)
        lib.paged_decode_shared_attn(**a)
        lib.paged_prefill_attn(outs[1], s.q, s.kc, s.vc, a["block_tables"], cu_q, cu_k, 1, s.scale)
        lib.paged_decode_attn(outs[2], s.q, s.kc, s.vc, a["block_tables"], a["context_lens"], s.scale, ws, mtb)
        shared.append(torch.empty_like(s.out))
        lib.paged_decode_shared_attn(**{**a, "out": shared[-1]})
        lib.paged_decode_weights_attn(outs[3], kw, s.q, s.kc, s.vc, a["block_tables"], a["context_lens"], s.scale, wws, mtb)
    torch.cuda.synchronize()
    s.compare()
    for out in shared:
        assert torch.equal(out, s.out)
    for out in outs[:4]:
        for i in range(S):
            _, bound = s.want(i)
            # (those round their weights to bf16 once: 2^-8 of max|v| more)
            assert ((out[i].double() - s.out[i].double()).abs() <= 2 * bound + 2.0**-7 * s.vc.abs().max().double()).all()


def test_blocks_past_32_bits(lib):
    """A cache of more than 2^32 values: shared and own blocks at its end."""
    block, Hkv, D = 512, 8, 128
    NB = (1 << 32) // (block * Hkv * D) + 8
    s = Shared([(2, [40, 513, 0])], 16, Hkv, D, block, poison=False)
    kc = torch.zeros(NB, block, Hkv, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    n = s.kc.shape[0]
    kc[NB - n:], vc[NB - n:] = s.kc, s.vc
    s.kc, s.vc = kc, vc
    s.tables = np.where(s.tables >= 0, s.tables + NB - n, s.tables)
    s.check(lib)


def test_refusals_of_the_binding(lib):
    s = Shared([(1, [3, 4])], 4, 2, 64)
    a = s.args(lib)
    bad = [dict(out=s.out[:1]), dict(q=s.q.float()), dict(context_lens=a["context_lens"][:1]), dict(group_starts=a["group_starts"][:1]),
           dict(shared_blocks=a["shared_blocks"].long()), dict(v_cache=s.vc[:1]), dict(block_tables=a["block_tables"].t()),
           dict(workspace=a["workspace"].cpu()), dict(dev_status=torch.zeros(1, device="cuda"))]
    for more in bad:
        with pytest.raises((ValueError, TypeError)):
            lib.paged_decode_shared_attn(**{**a, **more})
    with pytest.raises(lib.PkvError, match="WORKSPACE"):
        lib.paged_decode_shared_attn(**{**a, "workspace": a["workspace"][:-256]})
    with pytest.raises(lib.PkvError, match="INVALID_ARG"):
        lib.paged_decode_shared_attn(**{**a, "scale": float("nan")})


@pytest.mark.by_choice
@pytest.mark.parametrize("groups", [[(1, [1, 70])], [(8, [5, 0, 200]), (0, [700])], [(150, [(37 * i) % 300 for i in range(40)])],
                                    [(30, [3, 9]), (60, list(range(60))), (0, [900, 5])]])
@pytest.mark.parametrize("G,D", [(2, 128), (8, 64)])
def test_shared_or_not_as_it_pays(lib, groups, G, D):
    """From batches too short for it to ones that are not."""
    Shared(groups, 4 * G, 4, D, 64).check(lib)


# Batches whose tables have little room are read whole, with no plan of the groups: with room
# for up to 1024 tokens (512 at eight heads to a kv head) in a single launch.  wide: columns of
# the tables that nobody uses.
SHORT_OR_SMALL = pytest.mark.parametrize("wide", [0, 20])


@pytest.mark.by_choice
@SHORT_OR_SMALL
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (4, 2), (4, 1), (16, 2)])
def test_a_small_batch(lib, Hq, Hkv, D, wide):
    Shared([(1, [0, 1, 63]), (2, [5, 70]), (0, [1, 15, 16, 17, 33])], Hq, Hkv, D, wide=wide).check(lib)


@pytest.mark.by_choice
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,tokens", [(1, 1024), (4, 1023), (4, 1025), (8, 512), (8, 513), (2, 961), (8, 449)])
def test_about_as_long_as_a_short_context_can_be(lib, G, tokens, D):
    """Every warp has tiles, and from one to all but one of them less than the others."""
    Shared([(3, [tokens - 192, 100, 0]), (0, [tokens, 7])], 2 * G, 2, D).check(lib)


@pytest.mark.by_choice
@pytest.mark.parametrize("n", [304, 305])
def test_about_as_many_sequences_as_a_short_batch_can_have(lib, n):
    Shared([(1, [(7 * i) % 150 for i in range(n)])], 2, 1, 64, 64).check(lib)


@pytest.mark.by_choice
def test_a_short_batch_on_streams_and_from_a_graph(lib):
    s = Shared([(2, [30, 5, 64]), (0, [200])], 8, 2, 128)
    a = s.args(lib)
    lib.paged_decode_shared_attn(**a)
    torch.cuda.synchronize()
    want = bits(s.out)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(s.out) for _ in streams]
    spaces = [torch.empty_like(a["workspace"]) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, out, ws in zip(streams, outs, spaces):
            lib.paged_decode_shared_attn(**{**a, "out": out, "workspace": ws, "stream": st})
    torch.cuda.synchronize()
    for out in outs:
        assert (bits(out) == want).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.paged_decode_shared_attn(**a)
    s.q.copy_(torch.randn_like(s.q, dtype=torch.float32).to(torch.bfloat16))
    s.ctx = [L - 1 for L in s.ctx]
    a["context_lens"].copy_(torch.tensor(s.ctx, dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    s.compare()


@pytest.mark.by_choice
def test_the_most_sequences_of_a_small_batch(lib):
    """384 of them, and one more, which is planned."""
    for n in (384, 385):
        Shared([(1, [i % 60 for i in range(n)])], 2, 1, 64, 64).check(lib)


@pytest.mark.by_choice
@SHORT_OR_SMALL
def test_a_small_batch_with_empty_contexts(lib, wide):
    Shared([(2, [None, 5, 64]), (0, [None, 64, None])], 4, 2, 64, wide=wide).check(lib, status=lib.DEV_BAD_CONTEXT)
    Shared([(0, [None, None])], 4, 2, 64, wide=wide).check(lib, status=lib.DEV_BAD_CONTEXT)


@pytest.mark.by_choice
@pytest.mark.parametrize("blocks", [2, 20])
def test_a_small_batch_with_clamped_contexts(lib, blocks):
    s = Shared([(blocks, [64, 64, 10])], 4, 2, 64, 64)
    s.ctx[1] = 10**6
    s.check(lib, status=lib.DEV_BAD_CONTEXT)


@pytest.mark.by_choice
@pytest.mark.parametrize("starts,shared", [([1, 2, 5], [3, 2]), ([0, 2, 4], [3, 2]), ([0, 6, 5], [3, 2]), ([0, -3, 5], [3, 2]), ([0, 2, 5], [-1, 2]),
                                           ([0, 2, 5], [3, 1000])])
@SHORT_OR_SMALL
def test_a_small_batch_with_bad_groups(lib, starts, shared, wide):
    s = Shared([(3, [4, 70]), (2, [5, 9, 30])], 4, 2, 64, wide=wide)
    flag = lib.DEV_BAD_SEQLEN if starts != s.starts else lib.DEV_BAD_CONTEXT
    s.starts, s.shared = starts, shared
    s.check(lib, status=flag)


@pytest.mark.by_choice
@SHORT_OR_SMALL
def test_a_small_batch_with_block_ids_out_of_range(lib, wide):
    s = Shared([(2, [4, 70]), (2, [5, 9]), (0, [30])], 4, 2, 64, poison=False, wide=wide)
    s.tables[0, 1] = s.kc.shape[0]
    s.tables[3, 2] = -1
    lib.paged_decode_shared_attn(**s.args(lib))
    torch.cuda.synchronize()
    assert int(s.status.item()) == lib.DEV_BAD_BLOCK
    s.compare(only={1, 2, 4})


@pytest.mark.by_choice
@SHORT_OR_SMALL
def test_small_and_large_batches_in_turn(lib, wide):
    """On one stream and workspace, none waited for on the host; then from a graph."""
    few = Shared([(1, [5, 9]), (0, [100, 3])], 8, 2, 128, wide=wide)
    many = Shared([(200, [(31 * i) % 200 for i in range(2)]), (0, [700, 1])], 8, 2, 128)
    a, b = few.args(lib), many.args(lib)
    assert a["workspace"].numel() == b["workspace"].numel()
    b["workspace"] = a["workspace"]
    for _ in range(4):
        lib.paged_decode_shared_attn(**a)
        lib.paged_decode_shared_attn(**b)
    torch.cuda.synchronize()
    few.compare(), many.compare()
    want = few.out.clone(), many.out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):
            lib.paged_decode_shared_attn(**b)
            lib.paged_decode_shared_attn(**a)
    few.out.zero_(), many.out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(few.out, want[0]) and torch.equal(many.out, want[1])


@pytest.mark.parametrize("loading", [0, 1, 20])
@pytest.mark.parametrize("D", [64, 128])
def test_a_wait_that_runs_out_then_the_next_call(lib, loading, D):
    """CTAs that load nothing: all else in them waits for tiles that never come, gives up and says so."""
    s = Shared([(60, [(37 * i) % 100 for i in range(30)]), (20, [5, 9])], 8, 4, D)
    a = s.args(lib)
    lib.test_shared_fault(2_000_000, loading, 1)
    lib.paged_decode_shared_attn(**a)
    torch.cuda.synchronize()
    lib.test_shared_fault(10**9, -1, 1)
    assert int(s.status.item()) == lib.DEV_TIMEOUT
    s.status.zero_()
    s.out.fill_(7.0)
    lib.paged_decode_shared_attn(**a)
    torch.cuda.synchronize()
    assert int(s.status.item()) == 0
    s.compare()
