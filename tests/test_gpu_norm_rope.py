"""norm_rope_store on the GPU against the float64 oracle.

Tolerances, derived: all arithmetic is fp32 and one rounding to bf16 ends it, off by at
most 2^-9 (half a step, eps / 2) of the value.  Before it, of a value y = x w / rms: the
sum of squares is of positive terms, each addition and product off by 2^-24 of the sum,
D of them, so the root by D 2^-25; rsqrtf by 2 ulps (2^-22), the mean's product, eps's
addition and the two products 2^-24 each: under (D / 2 + 8) 2^-24 <= 72 * 2^-24 < 2^-17 of
|y|.  The angle comes with 32 bits of a turn (2^-33 of a turn, 2^-30 radians), goes to fp32
(2^-25 of half a turn at most: 2^-23 radians) and sincospi gives 2 ulps: under 2^-21 of
the pair's length; the products and sum of the rotation add 3 * 2^-24.  So a value is off
by at most  2^-9 |y'| + 2^-16 * amplitude * length of the pair  (2^-17 + 2^-21 + 2^-22 <
2^-16; for values that do not turn the length is |y|).  eps / 2 of bf16 is 2^-8: torch's
eps is the step above one, 2^-7, so half a step relative to a value just above a power
of two is 2^-8, which is what is taken.
"""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from oracle import steps

pytestmark = pytest.mark.gpu

HALF_STEP = torch.finfo(torch.bfloat16).eps / 2


def frequencies(R, base=10000.0):
    return base ** (-np.arange(0, R, 2, dtype=np.float64) / max(R, 1))


def f64(t):
    return t.detach().double().cpu().numpy()


class Rows:
    def __init__(self, T, Hq, Hkv, D, R=None, packed=True, far=5000, block=64, seed=0, skip=0.2):
        g = torch.Generator().manual_seed(seed)
        R = D if R is None else R
        size = torch.exp(0.8 * torch.randn(Hq + 2 * Hkv, D, generator=g))
        x = (torch.randn(T, Hq + 2 * Hkv, D, generator=g) * size).to(torch.bfloat16).cuda()
        self.all = x
        self.q, self.k, self.v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        if not packed:
            self.q, self.k, self.v = self.q.contiguous(), self.k.contiguous(), self.v.contiguous()
        self.positions = torch.randint(0, far, (T,), generator=g, dtype=torch.int32).cuda()
        self.inv_freq = frequencies(R)
        self.qw = torch.exp(0.3 * torch.randn(D, generator=g)).to(torch.bfloat16).cuda()
        self.kw = torch.exp(0.3 * torch.randn(D, generator=g)).to(torch.bfloat16).cuda()
        NB = -(-T // block) + 2
        slots = torch.randperm(NB * block, generator=g)[:T].to(torch.int32)
        slots[torch.rand(T, generator=g) < skip] = -1
        self.slots = slots.cuda()
        self.kc = torch.randn(NB, block, Hkv, D, generator=g).to(torch.bfloat16).cuda()
        self.vc = torch.randn(NB, block, Hkv, D, generator=g).to(torch.bfloat16).cuda()
        self.q_out = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
        self.k_out = torch.full((T, Hkv, D), 7.0, dtype=torch.bfloat16, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(self, pkv, norm=True, store=True, k_out=False, **more):
        args = dict(q_out=self.q_out, q=self.q, k=self.k, v=self.v if store else None, positions=self.positions,
                    turns=pkv.rope_turns(self.inv_freq), dev_status=self.status)
        if store:
            args.update(k_cache=self.kc, v_cache=self.vc, slot_mapping=self.slots)
        if k_out or not store:
            args.update(k_out=self.k_out)
        if norm:
            args.update(q_weight=self.qw, k_weight=self.kw)
        args.update(more)
        pkv.norm_rope_store(**args)
        torch.cuda.synchronize()

    def want(self, x, weight, **more):
        """The oracle's values and the bound on what they may be off."""
        amplitude = abs(more.get("amplitude", 1.0))
        y = steps.norm_rope(f64(x), self.positions.cpu().numpy(), self.inv_freq, weight, **more)
        plain = steps.norm_rope(f64(x), self.positions.cpu().numpy(), [], weight, eps=more.get("eps", 1e-6))
        length = np.abs(plain)
        half = len(self.inv_freq)
        R = 2 * half
        a, b = (np.arange(0, R, 2), np.arange(1, R, 2)) if more.get("interleaved") else (np.arange(half), np.arange(half, R))
        pair = amplitude * np.hypot(plain[..., a], plain[..., b])
        length[..., a] = pair
        length[..., b] = pair
        return y, HALF_STEP * np.abs(y) + 2.0**-16 * length + 2.0**-133  # (a subnormal bf16's half step)

    def check(self, pkv, norm=True, store=True, k_out=False, interleaved=False, amplitude=1.0, eps=1e-6):
        more = dict(interleaved=interleaved, amplitude=amplitude, eps=eps)
        # (before the call: what it may overwrite)
        q, bound_q = self.want(self.q, f64(self.qw) if norm else None, **more)
        k, bound_k = self.want(self.k, f64(self.kw) if norm else None, **more)
        kc, vc, v = self.kc.clone(), self.vc.clone(), self.v.clone()
        self.call(pkv, norm=norm, store=store, k_out=k_out, **more)

        def near(got, want, bound, what):
            bad = ~(np.abs(f64(got) - want) <= bound)
            assert not bad.any(), (what, np.argwhere(bad)[:5], f64(got)[bad][:5], want[bad][:5])

        near(self.q_out, q, bound_q, "q_out")
        if k_out or not store:
            near(self.k_out, k, bound_k, "k_out")
        if store:
            kept = (self.slots >= 0).nonzero()[:, 0]
            flat = self.slots[kept].long()
            near(self.kc.flatten(0, 1)[flat], k[kept.cpu().numpy()], bound_k[kept.cpu().numpy()], "k_cache")
            assert torch.equal(self.vc.flatten(0, 1)[flat].view(torch.int16), v[kept].contiguous().view(torch.int16))
            rest = torch.ones(self.kc.shape[0] * self.kc.shape[1], dtype=torch.bool, device="cuda")
            rest[flat] = False
            assert torch.equal(self.kc.flatten(0, 1)[rest], kc.flatten(0, 1)[rest])
            assert torch.equal(self.vc.flatten(0, 1)[rest], vc.flatten(0, 1)[rest])
        assert int(self.status.item()) == 0


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("T,Hq,Hkv,D,R", [(1, 1, 1, 64, 64), (2, 4, 2, 64, 64), (3, 3, 1, 128, 128), (5, 16, 8, 128, 64), (17, 5, 5, 64, 16),
                                          (9, 8, 1, 128, 48), (4, 7, 3, 128, 96), (33, 4, 4, 64, 48), (6, 64, 8, 128, 112), (3, 2, 2, 128, 0)])
def test_shapes(lib, T, Hq, Hkv, D, R, norm, interleaved):
    Rows(T, Hq, Hkv, D, R, packed=T % 2 == 0).check(lib, norm=norm, interleaved=interleaved)


@pytest.mark.parametrize("T", [3 * 152, 3 * 152 + 1, 8 * 152 + 13])
@pytest.mark.parametrize("D", [64, 128])
def test_many_rows(lib, D, T):
    """The most tokens of one per CTA, and more."""
    Rows(T, 2, 1, D, 32).check(lib, norm=True)


@pytest.mark.parametrize("store,k_out", [(True, True), (False, True)])
@pytest.mark.parametrize("packed", [True, False])
def test_rotated_keys_as_a_tensor(lib, store, k_out, packed):
    Rows(19, 6, 3, 128, 64, packed=packed).check(lib, store=store, k_out=k_out)


@pytest.mark.parametrize("far", [1 << 20, (1 << 31) - 1])
def test_far_positions(lib, far):
    r = Rows(40, 2, 2, 64, 64, far=far)
    # the farthest there are, and backwards
    r.positions[0], r.positions[1], r.positions[2], r.positions[3] = 2**31 - 1, -2**31, -1, 0
    # (frequencies with few bits: the oracle's own product position * inv_freq is then exact in 64 bits,
    # and what is left is its cosine's argument of 2^31 radians, 2^-22 of a radian at most)
    r.inv_freq = np.array([float(np.float32(f)) for f in r.inv_freq])
    r.check(lib)


def test_amplitude_and_eps(lib):
    Rows(21, 4, 2, 128, 64).check(lib, amplitude=1.3466, eps=1e-3)
    Rows(21, 4, 2, 128, 64).check(lib, amplitude=-0.5, norm=False, interleaved=True)


def test_rows_of_zeros_and_tiny_and_huge_values(lib):
    r = Rows(6, 4, 2, 64, 64, packed=False)
    r.q[0] = 0
    r.k[1] = 0
    r.q[2] *= 1e-15   # squares far below eps
    r.k[3] *= 1e15    # squares up to 1e31
    r.check(lib)
    r.check(lib, eps=0.1)


def test_values_that_do_not_turn_keep_their_bits(lib):
    r = Rows(7, 3, 2, 128, 32, packed=False)
    bits = torch.randint(-2**15, 2**15, r.q.shape, dtype=torch.int32).to(torch.int16).cuda()  # every pattern, NaN among them
    r.q.view(torch.int16)[..., 32:] = bits[..., 32:]
    r.v.view(torch.int16).copy_(bits[:, :2])
    r.call(lib, norm=False)
    assert torch.equal(r.q_out.view(torch.int16)[..., 32:], bits[..., 32:])
    kept = (r.slots >= 0).nonzero()[:, 0]
    assert torch.equal(r.vc.flatten(0, 1)[r.slots[kept].long()].view(torch.int16), r.v[kept].view(torch.int16))


def test_in_place(lib):
    """q_out = q and k_out = k, contiguous: the same bits as beside them."""
    r = Rows(50, 6, 2, 128, 128, packed=False)
    r.call(lib, k_out=True)
    q, k = r.q.clone(), r.k.clone()
    lib.norm_rope_store(q, q, k, r.v, r.positions, lib.rope_turns(r.inv_freq), k_out=k, q_weight=r.qw, k_weight=r.kw)
    torch.cuda.synchronize()
    assert torch.equal(q.view(torch.int16), r.q_out.view(torch.int16))
    assert torch.equal(k.view(torch.int16), r.k_out.view(torch.int16))


def test_overlaps_are_refused(lib):
    r = Rows(8, 4, 4, 64, 64)
    for bad in (dict(q_out=r.all[:, :4].reshape(-1)[:0].new_empty(0)),):
        with pytest.raises(ValueError):
            r.call(lib, **bad)
    flat = torch.zeros(3 * 8 * 4 * 64, dtype=torch.bfloat16, device="cuda")
    part = lambda i: flat[i:i + 8 * 4 * 64].view(8, 4, 64)
    turns = lib.rope_turns(r.inv_freq)
    for q_out, q, k, k_out in ((part(64), part(0), r.k, r.k_out), (part(0), r.q, part(256), r.k_out), (part(0), r.q, r.k, part(8)),
                               (r.q_out, part(0), r.k, part(512)), (r.q_out, r.q, part(0), part(256))):
        with pytest.raises(lib.PkvError, match="INVALID_ARG"):
            lib.norm_rope_store(q_out, q, k, None, r.positions, turns, k_out=k_out)


def test_slots_out_of_range_are_flagged_and_skipped(lib):
    r = Rows(6, 2, 2, 64, 64, skip=0.0)
    r.slots[1], r.slots[4] = r.kc.shape[0] * r.kc.shape[1], -2
    kc = r.kc.clone()
    r.call(lib)
    assert int(r.status.item()) == lib.DEV_BAD_SLOT
    changed = (r.kc != kc).flatten(2).any(2).flatten().nonzero()[:, 0].tolist()
    assert sorted(changed) == sorted(r.slots[[0, 2, 3, 5]].tolist())


def test_no_rows(lib):
    r = Rows(1, 2, 2, 64, 64)
    empty = lambda h: torch.empty(0, h, 64, dtype=torch.bfloat16, device="cuda")
    lib.norm_rope_store(empty(2), empty(2), empty(2), empty(2), r.positions[:0], lib.rope_turns(r.inv_freq), r.kc, r.vc, r.slots[:0])


def test_one_row_of_any_stride(lib):
    """One token: its stride says nothing (torch may give any), the call must not read by it."""
    r = Rows(4, 4, 2, 64, 64)
    q, k, v = (x[2:3] for x in (r.q, r.k, r.v))
    out = torch.empty(1, 4, 64, dtype=torch.bfloat16, device="cuda")
    lib.norm_rope_store(out, q.as_strided(q.shape, (3, 64, 1), q.storage_offset()), k, v, r.positions[2:3], lib.rope_turns(r.inv_freq), r.kc, r.vc,
                        r.slots[2:3], q_weight=r.qw, k_weight=r.kw)
    r.call(lib)
    assert torch.equal(out[0], r.q_out[2])


def test_on_a_stream_and_from_a_graph(lib):
    r = Rows(64, 16, 8, 128, 128)
    turns = lib.rope_turns(r.inv_freq)
    call = lambda stream=None: lib.norm_rope_store(r.q_out, r.q, r.k, r.v, r.positions, turns, r.kc, r.vc, r.slots, q_weight=r.qw, k_weight=r.kw, stream=stream)
    call()
    torch.cuda.synchronize()
    want, keys = r.q_out.clone(), r.kc.clone()
    r.q_out.zero_()
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    call(stream=other)
    other.synchronize()
    assert torch.equal(r.q_out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    r.positions.add_(1)
    graph.replay()
    torch.cuda.synchronize()
    replayed = r.q_out.clone()
    call()
    torch.cuda.synchronize()
    assert torch.equal(r.q_out, replayed) and not torch.equal(replayed, want) and not torch.equal(r.kc, keys)


def test_the_store_is_kv_stores_where_nothing_turns(lib):
    r = Rows(30, 2, 4, 128, 0)
    kc, vc = r.kc.clone(), r.vc.clone()
    r.call(lib, norm=False, positions=r.positions, turns=torch.empty(0, dtype=torch.int64, device="cuda"))
    lib.kv_store(r.k, r.v, kc, vc, r.slots)
    torch.cuda.synchronize()
    assert torch.equal(kc.view(torch.int16), r.kc.view(torch.int16)) and torch.equal(vc.view(torch.int16), r.vc.view(torch.int16))


def test_offsets_past_32_bits(lib):
    """A cache of more than 2^32 values: the last slots of it."""
    NB, block, Hkv, D = (1 << 32) // (512 * 8 * 128) + 2, 512, 8, 128
    kc = torch.zeros(NB, block, Hkv, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    r = Rows(5, 2, Hkv, D, D, skip=0.0)
    last = NB * block
    r.slots.copy_(torch.tensor([last - 1, 0, last - 2, 7, last - 513], dtype=torch.int32))
    r.kc, r.vc = kc, vc
    r.call(lib, k_out=True)
    assert torch.equal(kc.view(-1, Hkv, D)[r.slots.long()], r.k_out)
    assert torch.equal(vc.view(-1, Hkv, D)[r.slots.long()], r.v)


# More than 3 tokens per SM are streamed through shared memory, half a token to a warp at a
# time; more than 64 a whole one.
MANY, FEW, WHOLE = 16 * 152, 400, 64 * 152


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D,R", [(1, 1, 64, 64), (3, 1, 128, 48), (5, 2, 64, 16), (4, 4, 128, 32)])
def test_streamed_rows(lib, Hq, Hkv, D, R, interleaved):
    Rows(MANY + 117, Hq, Hkv, D, R, packed=interleaved).check(lib, norm=R != 16, interleaved=interleaved, amplitude=1.2)


@pytest.mark.parametrize("store,k_out", [(True, True), (False, True)])
def test_streamed_keys_as_a_tensor(lib, store, k_out):
    Rows(MANY + 1, 2, 1, 64, 32, packed=store).check(lib, store=store, k_out=k_out)


@pytest.mark.parametrize("T", [FEW + 100, MANY + 5, WHOLE + 301])
def test_streamed_rows_are_those_of_few(lib, T):
    """The same tokens, streamed and a part of them at a time: the same bits (ordinary head counts, a whole head turned)."""
    r = Rows(T, 16, 8, 128, 128)
    r.call(lib, k_out=True)
    q, k, kc, vc = r.q_out.clone(), r.k_out.clone(), r.kc.clone(), r.vc.clone()
    r.q_out.zero_(), r.k_out.zero_(), r.kc.zero_(), r.vc.zero_()
    turns, T = lib.rope_turns(r.inv_freq), r.q.shape[0]
    for a in range(0, T, FEW):
        b = min(a + FEW, T)
        lib.norm_rope_store(r.q_out[a:b], r.q[a:b], r.k[a:b], r.v[a:b], r.positions[a:b], turns, r.kc, r.vc, r.slots[a:b], k_out=r.k_out[a:b],
                            q_weight=r.qw, k_weight=r.kw)
    torch.cuda.synchronize()
    kept = r.slots[r.slots >= 0].long()
    assert torch.equal(q, r.q_out) and torch.equal(k, r.k_out)
    assert torch.equal(kc.flatten(0, 1)[kept], r.kc.flatten(0, 1)[kept]) and torch.equal(vc.flatten(0, 1)[kept], r.vc.flatten(0, 1)[kept])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D,R,store,k_out", [(1, 1, 64, 64, True, False), (3, 1, 128, 48, True, True), (5, 2, 64, 16, False, True)])
def test_streamed_as_whole_rows(lib, Hq, Hkv, D, R, store, k_out, interleaved):
    Rows(WHOLE + 7, Hq, Hkv, D, R, packed=store).check(lib, store=store, k_out=k_out, interleaved=interleaved)


@pytest.mark.parametrize("T", [FEW + 100, WHOLE + 301])
def test_streamed_on_streams_and_from_a_graph(lib, T):
    """Two calls at a time, and a captured one, replayed on other positions."""
    r = Rows(T, 16, 8, 128, 128)
    turns = lib.rope_turns(r.inv_freq)
    call = lambda out, kc, vc, stream=None: lib.norm_rope_store(out, r.q, r.k, r.v, r.positions, turns, kc, vc, r.slots, q_weight=r.qw, k_weight=r.kw, stream=stream)
    call(r.q_out, r.kc, r.vc)
    sets = [(torch.zeros_like(r.q_out), r.kc.clone().zero_(), r.vc.clone().zero_()) for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        for st, x in zip(streams, sets):
            call(*x, stream=st)
    torch.cuda.synchronize()
    kept = r.slots[r.slots >= 0].long()
    for out, kc, vc in sets:
        assert torch.equal(out, r.q_out)
        assert torch.equal(kc.flatten(0, 1)[kept], r.kc.flatten(0, 1)[kept]) and torch.equal(vc.flatten(0, 1)[kept], r.vc.flatten(0, 1)[kept])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(*sets[0])
    r.positions.add_(1)
    graph.replay()
    call(r.q_out, r.kc, r.vc)
    torch.cuda.synchronize()
    assert torch.equal(sets[0][0], r.q_out) and not torch.equal(sets[1][0], r.q_out)


def test_streamed_in_place(lib):
    r = Rows(MANY + 50, 6, 2, 128, 128, packed=False)
    r.call(lib, k_out=True)
    q, k = r.q.clone(), r.k.clone()
    lib.norm_rope_store(q, q, k, r.v, r.positions, lib.rope_turns(r.inv_freq), k_out=k, q_weight=r.qw, k_weight=r.kw)
    torch.cuda.synchronize()
    assert torch.equal(q.view(torch.int16), r.q_out.view(torch.int16))
    assert torch.equal(k.view(torch.int16), r.k_out.view(torch.int16))


def test_streamed_bits_that_do_not_turn_and_bad_slots(lib):
    r = Rows(MANY + 7, 3, 2, 128, 32, packed=False, skip=0.0)
    bits = torch.randint(-2**15, 2**15, r.q.shape, dtype=torch.int32).to(torch.int16).cuda()
    r.q.view(torch.int16)[..., 32:] = bits[..., 32:]
    r.v.view(torch.int16).copy_(bits[:, :2])
    r.slots[5], r.slots[MANY] = r.kc.shape[0] * r.kc.shape[1], -9
    r.call(lib, norm=False)
    assert torch.equal(r.q_out.view(torch.int16)[..., 32:], bits[..., 32:])
    kept = ((r.slots >= 0) & (r.slots < r.kc.shape[0] * r.kc.shape[1])).nonzero()[:, 0]
    assert torch.equal(r.vc.flatten(0, 1)[r.slots[kept].long()].view(torch.int16), r.v[kept].view(torch.int16))
    assert int(r.status.item()) == lib.DEV_BAD_SLOT


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("Hq,Hkv", [(32, 8), (41, 3), (2, 20)])
def test_streamed_in_halves(lib, Hq, Hkv, interleaved):
    """Rows of a token that leave shared memory room for fewer than twelve warps: most heads of q, few of them, odd numbers."""
    r = Rows(MANY + 9, Hq, Hkv, 128, 64, packed=interleaved, block=256)
    r.call(lib, k_out=True, interleaved=interleaved)
    q, k, kc, vc = r.q_out.clone(), r.k_out.clone(), r.kc.clone(), r.vc.clone()
    r.q_out.zero_(), r.k_out.zero_(), r.kc.zero_(), r.vc.zero_()
    turns, T = lib.rope_turns(r.inv_freq), r.q.shape[0]
    for a in range(0, T, FEW):
        b = min(a + FEW, T)
        lib.norm_rope_store(r.q_out[a:b], r.q[a:b], r.k[a:b], r.v[a:b], r.positions[a:b], turns, r.kc, r.vc, r.slots[a:b], k_out=r.k_out[a:b],
                            q_weight=r.qw, k_weight=r.kw, interleaved=interleaved)
    torch.cuda.synchronize()
    kept = r.slots[r.slots >= 0].long()
    assert torch.equal(q, r.q_out) and torch.equal(k, r.k_out)
    assert torch.equal(kc.flatten(0, 1)[kept], r.kc.flatten(0, 1)[kept]) and torch.equal(vc.flatten(0, 1)[kept], r.vc.flatten(0, 1)[kept])
    # without a store, and in place
    again = r.q.contiguous().clone()
    keys = r.k.contiguous().clone()
    lib.norm_rope_store(again, again, keys, None, r.positions, turns, k_out=keys, q_weight=r.qw, k_weight=r.kw, interleaved=interleaved)
    torch.cuda.synchronize()
    assert torch.equal(again, q) and torch.equal(keys, k)


def test_many_rows_too_wide_to_stream(lib):
    """Rows of a token of which not even halves leave shared memory room for four warps."""
    r = Rows(MANY + 3, 256, 64, 128, 16, packed=False, block=256)
    r.call(lib, norm=True)
    T = r.q.shape[0]
    q = r.q_out.clone()
    turns = lib.rope_turns(r.inv_freq)
    r.q_out.zero_()
    n = FEW
    lib.norm_rope_store(r.q_out[:n], r.q[:n], r.k[:n], r.v[:n], r.positions[:n], turns, r.kc, r.vc, r.slots[:n], q_weight=r.qw, k_weight=r.kw)
    torch.cuda.synchronize()
    assert torch.equal(q[:n], r.q_out[:n])


def test_rows_that_are_no_rows_are_refused(lib):
    """Views whose heads or values are apart, or whose tokens are all the same one."""
    r = Rows(6, 4, 2, 64, 64, packed=False)
    wide = torch.zeros(6, 4, 128, dtype=torch.bfloat16, device="cuda")
    for q in (wide[..., ::2], wide[:, :, :64], r.q[:1].expand(6, 4, 64), r.q.transpose(0, 1).contiguous().transpose(0, 1)):
        with pytest.raises(ValueError, match="rows must be contiguous"):
            r.call(lib, q=q)
    for bad in (dict(k=r.k[:5]), dict(v=r.v[:, :1]), dict(positions=r.positions[:5]), dict(turns=r.positions), dict(slot_mapping=r.slots.long()),
                dict(q_weight=r.qw[:32]), dict(q_out=r.q_out[:, :, :32]), dict(v_cache=r.vc[:1]),
                dict(dev_status=torch.zeros(0, dtype=torch.int32, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            r.call(lib, **bad)
    with pytest.raises(ValueError, match="inconsistent shapes"):
        lib.norm_rope_store(r.q_out, r.q, r.k, None, r.positions, lib.rope_turns(r.inv_freq), k_out=r.k_out[:3])
