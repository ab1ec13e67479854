"""Host checks of plan_step, norm_rope_store and paged_decode_shared_attn (no GPU): what the
library and the binding refuse before any launch, the frequencies, and the oracle of steps."""
import ctypes
import math
import random
from fractions import Fraction

import numpy as np
import pytest
import torch

import paged_kv_cache_241_gb300 as pkv
from oracle import steps

NULL = None
P = ctypes.c_void_p(0x10000)
bf16, i32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def lib():
    return pkv.load()


# ------------------------------------------------------------------- the library's checks

def plan_call(lib, **kw):
    a = dict(new_lens=P, lens=P, borrowed=NULL, tables=P, free=P, num_free=P, new_context=P, new_free=P, slots=P, positions=P, cu_q=P, cu_k=P, S=4,
             rows=10, maxb=8, BS=256, NB=64, capacity=64, st=NULL, stream=NULL)
    a.update(kw)
    return lib.pkv_plan_step(*a.values())


def test_plan_step_rejects_bad_arguments(lib):
    for bad in (dict(S=-1), dict(rows=-1), dict(maxb=0), dict(NB=0), dict(capacity=-1), dict(S=0), dict(BS=0)):
        assert plan_call(lib, **bad) == 1, bad
    for name in ("new_lens", "lens", "tables", "free", "num_free", "new_context", "new_free", "slots", "positions", "cu_q", "cu_k"):
        assert plan_call(lib, **{name: NULL}) == 1, name
    # the lengths after the step in a part of those before it
    at = lambda n: ctypes.c_void_p(0x10000 + 4 * n)
    assert plan_call(lib, new_context=at(1)) == 1 and plan_call(lib, new_context=at(3)) == 1 and plan_call(lib, new_context=at(-2)) == 1
    for bad in (dict(BS=100), dict(BS=32), dict(S=16385), dict(rows=2**31 - 1), dict(capacity=2**31), dict(NB=2**31 // 256), dict(maxb=2**23)):
        assert plan_call(lib, **bad) == 2, bad


def rope_call(lib, **kw):
    a = dict(q_out=ctypes.c_void_p(0x1000000), k_out=NULL, q=ctypes.c_void_p(0x2000000), k=ctypes.c_void_p(0x3000000), v=ctypes.c_void_p(0x4000000),
             kc=P, vc=P, slots=P, positions=P, turns=P, qw=P, kw=P, T=4, Hq=16, Hkv=8, D=128, qs=0, ks=0, vs=0, R=128, inter=0, eps=1e-6, amp=1.0,
             NB=64, BS=256, st=NULL, stream=NULL)
    a.update(kw)
    return lib.pkv_norm_rope_store(*a.values())


def test_norm_rope_store_rejects_bad_arguments(lib):
    odd = ctypes.c_void_p(0x10008)
    nan, inf = float("nan"), float("inf")
    for bad in (dict(T=-1), dict(Hq=0), dict(Hkv=0), dict(D=0), dict(R=-16), dict(R=256), dict(eps=nan), dict(eps=-1e-9), dict(eps=inf), dict(amp=nan),
                dict(amp=inf), dict(qw=NULL), dict(kw=NULL), dict(qs=1000), dict(ks=1000), dict(vs=2044), dict(qs=2052), dict(NB=0), dict(BS=0),
                dict(NB=2**62), dict(kc=NULL), dict(vc=NULL), dict(slots=NULL), dict(kc=NULL, vc=NULL, slots=NULL), dict(q_out=NULL), dict(q=NULL),
                dict(k=NULL), dict(v=NULL), dict(turns=NULL), dict(positions=NULL), dict(q_out=odd), dict(q=odd), dict(kc=odd), dict(qw=odd),
                dict(k_out=odd), dict(T=2**60)):
        assert rope_call(lib, **bad) == 1, bad
    for bad in (dict(D=96, R=64), dict(D=256), dict(R=24), dict(R=8), dict(Hq=1 << 17), dict(Hkv=1 << 17)):
        assert rope_call(lib, **bad) == 2, bad
    assert rope_call(lib, T=0) == 0


def test_norm_rope_store_refuses_overlaps(lib):
    at = lambda base, values: ctypes.c_void_p(base + 2 * values)
    Q, K, V, O, row_q, row_k = 0x2000000, 0x3000000, 0x4000000, 0x1000000, 16 * 128, 8 * 128
    # q_out into q at another place, into k, into v; k_out into q, into k at another place, into v, into q_out
    for bad in (dict(q_out=at(Q, 8)), dict(q_out=at(Q, 4 * row_q - 8)), dict(q_out=at(K, 0)), dict(q_out=at(V, 4 * row_k - 8)),
                dict(q_out=ctypes.c_void_p(Q), qs=row_q + 8), dict(k_out=at(Q, 0)), dict(k_out=at(K, 8)), dict(k_out=at(V, 0)), dict(k_out=at(O, 0))):
        assert rope_call(lib, **bad) == 1, bad


def shared_call(lib, **kw):
    a = dict(out=P, q=P, kc=P, vc=P, bt=P, cl=P, starts=P, shared=P, S=4, N=2, Hq=16, Hkv=8, D=128, BS=256, maxb=8, NB=64, scale=0.1, ws=NULL, wsb=0,
             st=NULL, stream=NULL)
    a.update(kw)
    return lib.pkv_paged_decode_shared_attn(*a.values())


def test_shared_decode_rejects_bad_arguments(lib):
    for bad in (dict(S=-1), dict(N=-1), dict(Hq=12), dict(Hq=0), dict(maxb=0), dict(NB=0), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(scale=3e38), dict(N=0), dict(N=5), dict(out=NULL), dict(q=NULL), dict(kc=NULL), dict(vc=NULL), dict(bt=NULL), dict(cl=NULL),
                dict(starts=NULL), dict(shared=NULL), dict(q=ctypes.c_void_p(0x10008)), dict(out=ctypes.c_void_p(0x10002))):
        assert shared_call(lib, **bad) == 1, bad
    for bad in (dict(D=96), dict(Hq=48, Hkv=3), dict(BS=32), dict(S=8193), dict(maxb=4097), dict(Hq=5000, Hkv=5000)):
        assert shared_call(lib, **bad) == 2, bad
    need = lib.pkv_decode_shared_workspace_size(4, 2, 16, 8, 128)
    for bad in (dict(), dict(ws=P, wsb=need - 1), dict(ws=ctypes.c_void_p(0x10010), wsb=need)):
        assert shared_call(lib, **bad) == 3, bad
    assert shared_call(lib, S=0, N=0) == 0


def test_shared_workspace_size(lib):
    f = lib.pkv_decode_shared_workspace_size
    for bad in ((0, 1, 16, 8, 128), (4, 0, 16, 8, 128), (4, 1, 0, 8, 128), (4, 1, 16, 0, 128), (4, 1, 4, 8, 128), (4, 1, 1 << 17, 8, 128)):
        assert f(*bad) == 0
    assert f(8192, 8192, 64, 8, 128) > f(64, 1, 16, 8, 128) > 0


def test_shared_fault_hook_rejects_bad_arguments(lib):
    assert lib.pkv_test_shared_fault(0, -1, 0) == 1
    assert lib.pkv_test_shared_fault(1000, -2, 0) == 1


# ------------------------------------------------------------------ the binding's checks

def plan_args(S=3, rows=5, wide=2):
    z = lambda *n: torch.zeros(*n, dtype=i32)
    return dict(new_lens=z(S), context_lens=z(S), block_tables=z(S, wide), free_blocks=z(8), num_free=z(1), new_context_lens=z(S), new_num_free=z(1),
                slot_mapping=z(rows), positions=z(rows), cu_seqlens_q=z(S + 1), cu_seqlens_k=z(S + 1), num_blocks=8, block_size=256)


def rope_args(T=3, Hq=4, Hkv=2, D=64):
    z = lambda *n: torch.zeros(*n, dtype=bf16)
    return dict(q_out=z(T, Hq, D), q=z(T, Hq, D), k=z(T, Hkv, D), v=z(T, Hkv, D), positions=torch.zeros(T, dtype=i32),
                turns=torch.zeros(D // 2, dtype=torch.int64), k_cache=z(4, 256, Hkv, D), v_cache=z(4, 256, Hkv, D), slot_mapping=torch.zeros(T, dtype=i32))


def shared_args(S=2, Hq=4, Hkv=2, D=64):
    z = lambda *n: torch.zeros(*n, dtype=bf16)
    n = lambda *x: torch.zeros(*x, dtype=i32)
    return dict(out=z(S, Hq, D), q=z(S, Hq, D), k_cache=z(4, 256, Hkv, D), v_cache=z(4, 256, Hkv, D), block_tables=n(S, 2), context_lens=n(S),
                group_starts=n(2), shared_blocks=n(1), scale=0.1, workspace=torch.zeros(1 << 20, dtype=torch.uint8))


@pytest.mark.parametrize("call,args", [("plan_step", plan_args), ("norm_rope_store", rope_args), ("paged_decode_shared_attn", shared_args)])
def test_host_tensors_and_wrong_dtypes_are_refused(call, args):
    f = getattr(pkv, call)
    with pytest.raises(ValueError, match="CUDA"):
        f(**args())
    a = args()
    for name, t in a.items():
        if torch.is_tensor(t):
            with pytest.raises((TypeError, ValueError)):
                f(**{**a, name: t.double()})
    # (the first one that is looked at: its dtype before its device)
    first = "q" if call == "norm_rope_store" else next(iter(a))
    with pytest.raises(TypeError, match=first):
        f(**{**a, first: a[first].double()})


@pytest.mark.parametrize("call,args", [("plan_step", plan_args), ("norm_rope_store", rope_args), ("paged_decode_shared_attn", shared_args)])
def test_tensors_without_storage_and_no_tensors_are_refused(call, args):
    f = getattr(pkv, call)
    a = args()
    for name, t in a.items():
        if torch.is_tensor(t):
            for other in (t.to("meta"), torch.zeros(2).to_sparse(), t.tolist(), "x", 7):
                with pytest.raises((TypeError, ValueError, AttributeError)):
                    f(**{**a, name: other})


def test_the_bindings_module_is_for_one_torch():
    pkv.load()
    with pytest.raises(ImportError, match="built for torch"):
        pkv._call.bind("0.1", 1, 2, 3)
    assert pkv._call.bind(torch.__version__, *[ctypes.cast(getattr(pkv.load(), "pkv_" + n), ctypes.c_void_p).value for n in
                                                ("plan_step", "norm_rope_store", "paged_decode_shared_attn")]) is None


def test_parts_that_go_together():
    a = rope_args()
    for missing in ("k_cache", "v_cache", "slot_mapping"):
        with pytest.raises(ValueError, match="go together"):
            pkv.norm_rope_store(**{**a, missing: None})
    with pytest.raises(ValueError, match="go together"):
        pkv.norm_rope_store(**a, q_weight=torch.ones(64, dtype=bf16))


# ---------------------------------------------------------------------- the frequencies

def test_turns_are_fractions_of_a_turn():
    f = [1.0, 0.5, 1e-4, 10000.0 ** (-62 / 64), 0.0, -1.0, 2 * math.pi, 6.5]
    turns = pkv.rope_turns(f, "cpu").tolist()
    for x, t in zip(f, turns):
        want = x / (2 * math.pi)  # (to 2^-53 of itself, as the library takes it)
        off = (Fraction(t % 2**64, 2**64) - Fraction(want)) % 1
        assert min(off, 1 - off) <= Fraction(2, 2**53) * max(1, abs(Fraction(want)))
    # angles of far positions, from the integers: within position * 2^-54 turns
    for pos in (1, 12345, 1 << 20, 2**31 - 1, -7):
        for x, t in zip(f[:4], turns):
            turn = Fraction((pos * t) % 2**64, 2**64)
            want = Fraction(pos) * Fraction(x) / Fraction(2 * math.pi)
            off = (turn - want) % 1
            assert min(off, 1 - off) <= abs(pos) * Fraction(1, 2**50)


def test_turns_refuse_what_is_no_frequency():
    for bad in ([float("nan")], [float("inf")], [2e6], [1.0, -3e6]):
        with pytest.raises(pkv.PkvError, match="INVALID_ARG"):
            pkv.rope_turns(bad, "cpu")
    with pytest.raises(ValueError):
        pkv.rope_turns([[1.0]], "cpu")
    assert pkv.rope_turns([], "cpu").shape == (0,)


# ---------------------------------------------------------------------------- the oracle

def test_oracle_step_against_the_block_manager():
    """Random lives of sequences: the oracle's lengths, numbers of blocks and offsets are the host allocator's."""
    rng, BS, NB, S = random.Random(4), 64, 60, 6
    bm = pkv.BlockManager(NB, BS)
    tables, lens, stack = [[-1] * 12 for _ in range(S)], [0] * S, list(range(NB))
    free = NB
    for step in range(60):
        new = [-1 if L and rng.random() < 0.1 else rng.choice([0, 1, 1, rng.randint(1, 90)]) for L in lens]
        new = [n if L + n <= 12 * BS else 0 for L, n in zip(lens, new)]
        rows = sum(max(n, 0) for n in new)
        got, status = steps.plan_step(new, lens, tables, stack, free, rows, NB, BS)
        if status:
            assert status == steps.NO_BLOCKS
        for s in range(S):  # (the ends first)
            if new[s] == -1:
                bm.free(s)
        for s in range(S):
            grown = got["new_context_lens"][s] - lens[s]
            if new[s] > 0 and grown:
                if lens[s] == 0:
                    bm.allocate(s, [1000 * step + s] * grown)  # (no two alike: nothing is found)
                else:
                    for _ in range(grown):
                        bm.append(s, rng.randrange(1 << 30))
        tables, lens, stack, free = got["block_tables"], got["new_context_lens"], got["free_blocks"], got["new_num_free"][0]
        assert free == bm.num_free_blocks
        held = []
        for s in range(S):
            if lens[s]:
                assert bm.num_tokens(s) == lens[s]
                theirs = bm.block_table(s, 12)
                assert [b >= 0 for b in theirs] == [i * BS < lens[s] for i in range(12)]
                held += tables[s][: -(-lens[s] // BS)]
        assert len(set(held + stack[:free])) == NB and len(held) + free == NB  # no block twice, none lost


def test_oracle_rotation_keeps_lengths_and_composes():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 2, 16))
    f = [1.0, 0.3, 0.01, 0.7]
    for inter in (False, True):
        y = steps.norm_rope(x, [0, 5, -9], f, interleaved=inter)
        assert np.allclose(y[0], x[0]) and np.allclose(y[..., 8:], x[..., 8:])
        assert np.allclose((y**2).sum(-1), (x**2).sum(-1))
        again = steps.norm_rope(y, [0, -5, 9], f, interleaved=inter)
        assert np.allclose(again, x)
        # a query and a key turned by their positions: the product depends on the distance alone
        a, b = steps.norm_rope(x, [3, 8, 20], f, interleaved=inter), steps.norm_rope(x, [103, 108, 120], f, interleaved=inter)
        assert np.allclose(np.einsum("hd,hd->h", a[0], a[1]), np.einsum("hd,hd->h", b[0], b[1]))
    n = steps.norm_rope(x, [0, 0, 0], f, weight=np.full(16, 2.0), eps=0.0)
    assert np.allclose((n**2).mean(-1), 4.0)


def test_the_shared_decode_takes_tensor_memory_after_the_wait_for_the_kernel_before():
    """Read as text: the attention is a programmatic dependent, of whatever precedes the call where it plans by itself.  Were it to
    take all of tensor memory before it waits, a kernel before it that has yet to allocate its own on the same SM would wait for it,
    and it for that kernel's end."""
    import os
    import re

    text = open(os.path.join(os.path.dirname(pkv.__file__), "csrc", "decode_shared.cu")).read()
    text = re.sub(r"//[^\n]*", "", text)
    kernel = text.split("shared_attn_kernel(", 1)[1]
    assert kernel.index("griddepcontrol.wait") < kernel.index("prefixes<D>(")
    assert "tmem_alloc(" not in kernel.split("shared_join_kernel", 1)[0]  # (it is in prefixes, called behind the wait)
    assert text.count("tmem_alloc(") == 1 and "tmem_alloc(" in text.split("void prefixes(", 1)[1]
