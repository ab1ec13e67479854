"""CPU checks of the key-weight and eviction calls: the oracle's own pins, the
library's and the binding's refusals (nothing reaches a GPU), the block manager."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_241_gb300 as pkv
import workloads as wl
from test_abi import lib  # noqa: F401  (fixture: the built library, no GPU)

NULL, P = None, ctypes.c_void_p(0x10000)


# ------------------------------------------------------------------- the oracle

def test_weights_of_a_step_sum_to_the_group():
    b = wl.build_batch("w", "decode", 3, [4, 299], [1, 1], 4, 2, 64)
    kc, _ = oracle.kv_store(b.k_cache, b.v_cache, b.k, b.v, b.slot_mapping)
    before = np.ones((b.num_blocks, 2, 256))
    after, brought = oracle.decode_weights(before, b.q, kc, b.block_tables, b.context_lens, b.scale)
    # each of the two query heads of a kv head hands out weights that sum to one
    assert np.allclose(brought.sum((0, 2)), 2 * b.num_seqs, atol=1e-12)
    newest = b.slot_mapping
    assert np.allclose(after[newest // 256, :, newest % 256], brought[newest // 256, :, newest % 256])
    assert np.allclose((after - brought).sum(), before.sum() - 2 * b.num_seqs)


def test_a_chunk_of_one_query_is_a_decode_step():
    b = wl.build_batch("w", "decode", 4, [6, 130], [1, 1], 4, 2, 64, block_size=64)
    kc, _ = oracle.kv_store(b.k_cache, b.v_cache, b.k, b.v, b.slot_mapping)
    before = np.random.default_rng(0).random((b.num_blocks, 2, 64))
    one, _ = oracle.decode_weights(before, b.q, kc, b.block_tables, b.context_lens, b.scale)
    for window in (1, 5):
        two, _ = oracle.prefill_weights(before, b.q, kc, b.block_tables, b.cu_seqlens_q, b.cu_seqlens_k, window, b.scale)
        assert np.allclose(one, two, atol=1e-14)


def test_evict_map_by_hand():
    w = [5.0, 0.0, 3.0, 1.0, 4.0, 2.0, 9.0, 9.0]
    assert oracle.evict_map(w, 8, 5, 2).tolist() == [0, 4, 2, 6, 7]   # kept 0, 2, 4; 4 fills place 1
    assert oracle.evict_map(w, 8, 8, 2).tolist() == list(range(8))    # nothing to do
    assert oracle.evict_map(w, 3, 5, 2).tolist() == [0, 1, 2, -1, -1]
    assert oracle.evict_map([1.0] * 6, 6, 3, 0).tolist() == [0, 1, 2]  # ties: the lowest positions
    assert oracle.evict_map([float("nan"), 0.0, -1.0, 7.0], 4, 2, 1).tolist() == [1, 3]
    assert oracle.evict_map(w, 8, 3, 3).tolist() == [5, 6, 7]         # only the recent


# ----------------------------------------------------- refusals of the C entries

def decode_call(lib, **kw):  # noqa: F811
    a = dict(out=P, kw=P, q=P, nk=NULL, nv=NULL, sm=NULL, kc=P, vc=P, bt=P, cl=P, S=4, Hq=16, Hkv=8,
             D=128, BS=256, maxb=8, NB=64, mtb=32, scale=0.1, ws=NULL, wsb=0, st=NULL, stream=NULL)
    a.update(kw)
    return lib.pkv_paged_decode_weights_attn(*a.values())


def test_decode_weights_rejects_bad_arguments(lib):  # noqa: F811
    assert decode_call(lib, Hq=12) == 1
    assert decode_call(lib, D=96) == 2
    assert decode_call(lib, Hq=48, Hkv=3) == 2
    assert decode_call(lib, BS=100) == 2
    assert decode_call(lib, S=20000) == 2
    for bad in (float("nan"), float("inf"), -float("inf")):
        assert decode_call(lib, S=0, scale=bad) == 1
    assert decode_call(lib, S=0) == 0
    for name in ("out", "kw", "q", "kc", "vc", "bt", "cl"):
        assert decode_call(lib, **{name: NULL}) == 1, name
    for name in ("out", "q", "kc", "vc"):
        assert decode_call(lib, **{name: ctypes.c_void_p(0x10008)}) == 1, name
    assert decode_call(lib, kw=ctypes.c_void_p(0x10002)) == 1
    assert decode_call(lib, nk=P) == 1 and decode_call(lib, nk=P, nv=P) == 1  # the store's three go together
    assert decode_call(lib, nk=P, nv=ctypes.c_void_p(0x10008), sm=P) == 1
    need = lib.pkv_decode_weights_workspace_size(4, 16, 8, 128, 256, 32)
    assert need > 0
    assert decode_call(lib) == 3 and decode_call(lib, ws=P, wsb=need - 1) == 3
    assert decode_call(lib, ws=ctypes.c_void_p(0x10010), wsb=need) == 3
    assert decode_call(lib, ws=P, wsb=1 << 40, mtb=1 << 62) == 1  # a workspace that cannot be addressed


def test_weights_workspace_sizes(lib):  # noqa: F811
    f = lib.pkv_decode_weights_workspace_size
    assert f(0, 16, 8, 128, 256, 8) == 0 and f(4, 16, 8, 128, 256, -1) == 0
    assert f(4, 16, 8, 128, 256, 1 << 62) == 0 and f(4, 1 << 20, 8, 128, 256, 8) == 0
    # it holds at least every block's logits
    for mtb in (0, 1, 7, 4000, 1 << 20):
        assert f(4, 16, 8, 128, 256, mtb) >= mtb * 16 * 256 * 4
    g = lib.pkv_prefill_weights_workspace_size
    assert g(0, 10, 10, 5, 16, 8, 4, 256) == 0 and g(2, 10, 10, 0, 16, 8, 4, 256) == 0
    assert g(2, 20, 10, 5, 16, 8, 4, 256) >= 2 * 5 * 16 * 4
    assert g(1 << 30, (1 << 31) - 1, (1 << 31) - 1, (1 << 31) - 1, 1 << 30, 1, 1 << 30, 512) == 0


def prompt_call(lib, **kw):  # noqa: F811
    a = dict(kw=P, q=P, kc=P, bt=P, cq=P, ck=P, S=2, T=100, mq=64, window=32, Hq=16, Hkv=8, D=128,
             BS=256, maxb=4, NB=16, scale=0.1, ws=NULL, wsb=0, st=NULL, stream=NULL)
    a.update(kw)
    return lib.pkv_paged_prefill_weights(*a.values())


def test_prefill_weights_rejects_bad_arguments(lib):  # noqa: F811
    assert prompt_call(lib, Hq=10, Hkv=4) == 1
    assert prompt_call(lib, D=80) == 2
    assert prompt_call(lib, BS=32) == 2
    assert prompt_call(lib, Hq=32, Hkv=2) == 2
    assert prompt_call(lib, T=-1) == 1
    assert prompt_call(lib, window=0) == 1 and prompt_call(lib, window=-3) == 1
    for bad in (float("nan"), float("inf"), -float("inf")):
        assert prompt_call(lib, T=0, scale=bad) == 1
    assert prompt_call(lib, T=0) == 0 and prompt_call(lib, S=0) == 0
    assert prompt_call(lib, T=1 << 31) == 2
    for name in ("kw", "q", "kc", "bt", "cq", "ck"):
        assert prompt_call(lib, **{name: NULL}) == 1, name
    assert prompt_call(lib, q=ctypes.c_void_p(0x10008)) == 1
    assert prompt_call(lib, kw=ctypes.c_void_p(0x10002)) == 1
    need = lib.pkv_prefill_weights_workspace_size(2, 100, 64, 32, 16, 8, 4, 256)
    assert prompt_call(lib) == 3 and prompt_call(lib, ws=P, wsb=need - 1) == 3
    assert prompt_call(lib, ws=ctypes.c_void_p(0x10010), wsb=need) == 3


def evict_call(lib, **kw):  # noqa: F811
    a = dict(kc=P, vc=P, kw=P, bt=P, cl=P, S=4, Hkv=8, D=128, BS=256, maxb=8, NB=64, budget=1024,
             recent=32, kept=P, nl=ctypes.c_void_p(0x20000), st=NULL, stream=NULL)
    a.update(kw)
    return lib.pkv_kv_evict(*a.values())


def test_evict_rejects_bad_arguments(lib):  # noqa: F811
    assert evict_call(lib, budget=0) == 1 and evict_call(lib, budget=-1) == 1
    assert evict_call(lib, recent=-1) == 1 and evict_call(lib, recent=1025) == 1
    assert evict_call(lib, D=96) == 2
    assert evict_call(lib, BS=100) == 2
    assert evict_call(lib, maxb=4097) == 2                 # more than 2^20 places
    assert evict_call(lib, budget=(1 << 20) + 1) == 2
    assert evict_call(lib, S=0) == 0
    for name in ("kc", "vc", "kw", "bt", "cl", "kept", "nl"):
        assert evict_call(lib, **{name: NULL}) == 1, name
    assert evict_call(lib, kc=ctypes.c_void_p(0x10008)) == 1
    assert evict_call(lib, kw=ctypes.c_void_p(0x10002)) == 1
    assert evict_call(lib, nl=P) == 1                      # new_lens over context_lens


# -------------------------------------------------------- refusals of the binding

def test_binding_refuses_host_tensors_dtypes_and_shapes():
    bf16, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    S, Hq, Hkv, D, NB, BS = 2, 4, 2, 64, 8, 256
    kc, kw = torch.zeros(NB, BS, Hkv, D, dtype=bf16), torch.zeros(NB, Hkv, BS)
    bt, cl, ws = torch.zeros(S, 2, dtype=i32), torch.ones(S, dtype=i32), torch.zeros(64, dtype=torch.uint8)
    q = torch.zeros(S, Hq, D, dtype=bf16)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_decode_weights_attn(q.clone(), kw, q, kc, kc.clone(), bt, cl, 0.1, ws, 4)
    with pytest.raises(ValueError, match="go together"):
        pkv.paged_decode_weights_attn(q.clone(), kw, q, kc, kc.clone(), bt, cl, 0.1, ws, 4, k=q)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_prefill_weights(kw, q, kc, bt, cl, cl, 2, 4, 0.1, ws)
    with pytest.raises(TypeError, match="q"):
        pkv.paged_prefill_weights(kw, q.float(), kc, bt, cl, cl, 2, 4, 0.1, ws)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.kv_evict(kc, kc.clone(), kw, bt, cl, 4, 1, torch.zeros(S, Hkv, 4, dtype=i32), cl.clone())
    with pytest.raises(TypeError, match="k_cache"):
        pkv.kv_evict(kc.to(f32), kc.clone(), kw, bt, cl, 4, 1, torch.zeros(S, Hkv, 4, dtype=i32), cl.clone())


# ------------------------------------------------------------- the block manager

def test_manager_evict_releases_blocks_and_forgets_content(lib):  # noqa: F811
    bm = pkv.BlockManager(12, 4)
    prompt = list(range(100, 118))                          # 18 tokens, 5 blocks
    assert bm.allocate(1, prompt) == 0
    table = bm.block_table(1, 6).copy()
    bm.evict(1, 18)                                        # nothing to cut
    bm.evict(1, 40)
    assert bm.num_tokens(1) == 18 and bm.num_free_blocks == 7
    bm.evict(1, 6)
    assert bm.num_tokens(1) == 6 and bm.num_free_blocks == 10
    assert bm.block_table(1, 6).tolist() == table[:2].tolist() + [-1] * 4
    assert [bm.ref_count(b) for b in table[:5]] == [1, 1, 0, 0, 0]
    # the rewritten blocks are found by nobody any more
    assert bm.allocate(2, prompt) == 0
    assert not set(bm.block_table(2, 5).tolist()) & set(table[:2].tolist())
    bm.free(2)
    # growth goes on from the new length; the blocks that fill up are not keyed
    for t in range(10):
        bm.append(1, 500 + t)
    assert bm.num_tokens(1) == 16 and len(set(bm.block_table(1, 4).tolist())) == 4
    assert bm.slots(1, 6, 3).tolist() == [int(table[1]) * 4 + 2, int(table[1]) * 4 + 3, int(bm.block_table(1, 4)[2]) * 4]
    mine = set(bm.block_table(1, 4).tolist())
    assert bm.allocate(3, [500 + t for t in range(2, 6)] + [1]) == 0
    assert not set(bm.block_table(3, 2).tolist()) & mine
    bm.free(1)
    bm.free(3)
    assert bm.num_free_blocks == 12


def test_manager_refuses_to_evict_a_shared_prefix(lib):  # noqa: F811
    bm = pkv.BlockManager(16, 4)
    prompt = list(range(20))
    bm.allocate(1, prompt)
    assert bm.allocate(2, prompt[:8] + [77] * 6) == 8       # two blocks shared
    before = bm.block_table(1, 5).tolist()
    with pytest.raises(pkv.PkvError, match="UNSUPPORTED"):
        bm.evict(1, 12)
    assert bm.block_table(1, 5).tolist() == before and bm.num_tokens(1) == 20
    bm.free(2)
    bm.evict(1, 12)
    assert bm.num_tokens(1) == 12
    with pytest.raises(pkv.PkvError, match="INVALID"):
        bm.evict(1, 0)
    with pytest.raises(pkv.PkvError, match="INVALID"):
        bm.evict(9, 4)


def test_manager_evict_may_release_shared_tail_blocks(lib):  # noqa: F811
    # Only the blocks that eviction rewrites must be the sequence's own.
    bm = pkv.BlockManager(16, 4)
    bm.allocate(1, list(range(16)))
    bm.allocate(2, list(range(16)) + [5])
    with pytest.raises(pkv.PkvError):
        bm.evict(2, 4)
    assert [bm.ref_count(int(b)) for b in bm.block_table(2, 5)] == [2, 2, 2, 2, 1]


def test_int_arguments_do_not_wrap():
    # 2**32 + 5 must not reach the library as 5
    assert pkv._c_int32((1 << 32) + 5) == 0x7FFFFFFF and pkv._c_int32(-(1 << 32) + 5) == -1
    assert pkv._c_int32(7) == 7 and pkv._c_int32(0) == 0
