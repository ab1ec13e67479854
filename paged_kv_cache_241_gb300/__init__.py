"""Paged KV-cache attention for GB300 (sm_103a): Python binding of libpkv.

A thin ctypes layer over the C ABI declared in include/pkv.h.  It only
marshals arguments (torch tensors -> device pointers and sizes, the current
CUDA stream) and raises on a non-OK status; every step of the computation runs
in the library's CUDA kernels.  There is no CPU fallback: if the shared library
has not been built, `load()` raises.

    import paged_kv_cache_241_gb300 as pkv
    pkv.kv_store(k, v, k_cache, v_cache, slot_mapping)
    pkv.paged_decode_attn(out, q, k_cache, v_cache, block_tables, context_lens,
                          scale, workspace, max_total_blocks)
    pkv.paged_prefill_attn(out, q, k_cache, v_cache, block_tables, cu_q, cu_k,
                           max_seqlen_q, scale)   # workspace: one per stream, cached
    # a bounded cache: collect the weight each key receives, keep the heaviest
    pkv.paged_prefill_weights(key_weights, q, k_cache, block_tables, cu_q, cu_k,
                              max_seqlen_q, window, scale, prompt_workspace)
    pkv.paged_decode_weights_attn(out, key_weights, q, k_cache, v_cache, block_tables,
                                  context_lens, scale, workspace, max_total_blocks)
    pkv.kv_evict(k_cache, v_cache, key_weights, block_tables, context_lens, budget,
                 recent, kept, new_lens)
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpkv.so")

PKV_OK = 0
STATUS_NAMES = {0: "PKV_OK", 1: "PKV_ERR_INVALID_ARG", 2: "PKV_ERR_UNSUPPORTED",
                3: "PKV_ERR_WORKSPACE", 4: "PKV_ERR_CUDA", 5: "PKV_ERR_OUT_OF_BLOCKS"}
PKV_ERR_OUT_OF_BLOCKS = 5
DEV_BAD_SLOT = 0x1
DEV_BAD_BLOCK = 0x2
DEV_BAD_CONTEXT = 0x4
DEV_TIMEOUT = 0x8
DEV_WORKSPACE = 0x10
DEV_BAD_SEQLEN = 0x20

# Exported symbols and their ctypes signatures (must match include/pkv.h).
_c_int, _c_i64, _c_sz, _c_f, _p = (ctypes.c_int, ctypes.c_int64, ctypes.c_size_t,
                                   ctypes.c_float, ctypes.c_void_p)
SIGNATURES = {
    "pkv_status_string": (ctypes.c_char_p, [_c_int]),
    "pkv_abi_version": (_c_int, []),
    "pkv_kv_store": (_c_int, [_p, _p, _p, _p, _p, _c_i64, _c_int, _c_int, _c_i64, _c_i64, _c_i64,
                              _c_int, _p, _p]),
    "pkv_decode_workspace_size": (_c_sz, [_c_int, _c_int, _c_int, _c_int, _c_i64]),
    "pkv_paged_decode_attn": (_c_int, [_p, _p, _p, _p, _p, _p, _c_int, _c_int, _c_int, _c_int,
                                       _c_int, _c_int, _c_i64, _c_i64, _c_f, _p, _c_sz, _p, _p]),
    "pkv_paged_decode_store_attn": (_c_int, [_p, _p, _p, _p, _p, _p, _p, _p, _p, _c_int, _c_int,
                                             _c_int, _c_int, _c_int, _c_int, _c_i64, _c_i64, _c_f,
                                             _p, _c_sz, _p, _p]),
    "pkv_paged_decode_attn_noalloc": (_c_int, [_p, _p, _p, _p, _p, _p, _c_int, _c_int, _c_int,
                                               _c_int, _c_int, _c_int, _c_i64, _c_i64, _c_f, _p,
                                               _p]),
    "pkv_paged_prefill_attn": (_c_int, [_p, _p, _p, _p, _p, _p, _p, _c_int, _c_i64, _c_int,
                                        _c_int, _c_int, _c_int, _c_int, _c_int, _c_i64, _c_f, _p,
                                        _c_sz, _p, _p]),
    "pkv_prefill_workspace_size": (_c_sz, []),
    "pkv_test_decode_fault": (_c_int, [_c_i64, _c_int]),
    "pkv_decode_weights_workspace_size": (_c_sz, [_c_int, _c_int, _c_int, _c_int, _c_int, _c_i64]),
    "pkv_paged_decode_weights_attn": (_c_int, [_p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _c_int,
                                               _c_int, _c_int, _c_int, _c_int, _c_int, _c_i64,
                                               _c_i64, _c_f, _p, _c_sz, _p, _p]),
    "pkv_prefill_weights_workspace_size": (_c_sz, [_c_int, _c_i64, _c_int, _c_int, _c_int, _c_int,
                                                   _c_int, _c_int]),
    "pkv_paged_prefill_weights": (_c_int, [_p, _p, _p, _p, _p, _p, _c_int, _c_i64, _c_int, _c_int,
                                           _c_int, _c_int, _c_int, _c_int, _c_int, _c_i64, _c_f,
                                           _p, _c_sz, _p, _p]),
    "pkv_test_prompt_fault": (_c_int, [_c_i64, _c_int, _c_int]),
    "pkv_kv_evict": (_c_int, [_p, _p, _p, _p, _p, _c_int, _c_int, _c_int, _c_int, _c_int, _c_i64,
                              _c_int, _c_int, _p, _p, _p, _p]),
    "pkv_w4a16_dequant": (_c_int, [_p, _p, _p, _c_i64, _c_i64, _c_int, _p]),
    "pkv_bm_create": (_p, [_c_int, _c_int]),
    "pkv_bm_destroy": (None, [_p]),
    "pkv_bm_num_free_blocks": (_c_int, [_p]),
    "pkv_bm_allocate": (_c_int, [_p, _c_i64, _p, _c_int, ctypes.POINTER(_c_int)]),
    "pkv_bm_append": (_c_int, [_p, _c_i64, ctypes.c_int32]),
    "pkv_bm_free": (_c_int, [_p, _c_i64]),
    "pkv_bm_evict": (_c_int, [_p, _c_i64, _c_int]),
    "pkv_bm_num_tokens": (_c_int, [_p, _c_i64]),
    "pkv_bm_block_table": (_c_int, [_p, _c_i64, _p, _c_int]),
    "pkv_bm_slots": (_c_int, [_p, _c_i64, _c_int, _c_int, _p]),
    "pkv_bm_ref_count": (_c_int, [_p, _c_int]),
}

_lib = None


class PkvError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what} failed: {STATUS_NAMES.get(status, status)}")
        self.status = status


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libpkv.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it with `python -m paged_kv_cache_241_gb300.build` "
            "(the CUDA library is required; there is no fallback)")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(status: int, what: str) -> None:
    if status != PKV_OK:
        raise PkvError(status, what)


def _stream(stream) -> int:
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return int(getattr(stream, "cuda_stream", stream))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need(t, dtype, name, ndim=None):
    import torch

    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name}: expected {ndim} dims, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t


def kv_store(k, v, k_cache, v_cache, slot_mapping, dev_status=None, stream=None) -> None:
    """Write new K/V rows k/v [T, Hkv, D] (bf16; rows may be strided by a
    token stride) into k_cache/v_cache [NB, BS, Hkv, D] at slot_mapping [T]."""
    import torch

    lib = load()
    _need(k_cache, torch.bfloat16, "k_cache", 4)
    _need(v_cache, torch.bfloat16, "v_cache", 4)
    _need(slot_mapping, torch.int32, "slot_mapping", 1)
    NB, BS, Hkv, D = k_cache.shape
    for name, t in (("k", k), ("v", v)):
        if t.dtype != torch.bfloat16 or not t.is_cuda or t.dim() != 3:
            raise ValueError(f"{name}: expected a CUDA bf16 [T, Hkv, D] tensor")
        if t.stride(2) != 1 or t.stride(1) != D or tuple(t.shape[1:]) != (Hkv, D):
            raise ValueError(f"{name}: rows must be contiguous [Hkv, D] = {(Hkv, D)}")
    st = lib.pkv_kv_store(_ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache), _ptr(slot_mapping),
                          k.shape[0], Hkv, D, k.stride(0), v.stride(0), NB, BS,
                          _ptr(dev_status), _stream(stream))
    _check(st, "pkv_kv_store")


def decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, max_total_blocks) -> int:
    return int(load().pkv_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                max_total_blocks))


def decode_workspace(num_seqs, num_q_heads, num_kv_heads, head_dim, max_total_blocks,
                     device="cuda"):
    """Allocate a zero-filled decode workspace (uint8, 256-byte aligned by torch)."""
    import torch

    n = decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, max_total_blocks)
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=device)


def paged_decode_attn(out, q, k_cache, v_cache, block_tables, context_lens, scale, workspace,
                      max_total_blocks, dev_status=None, stream=None) -> None:
    """out/q [S, Hq, D] bf16; block_tables [S, max_blocks] int32; context_lens [S] int32."""
    import torch

    lib = load()
    _need(out, torch.bfloat16, "out", 3)
    _need(q, torch.bfloat16, "q", 3)
    _need(k_cache, torch.bfloat16, "k_cache", 4)
    _need(v_cache, torch.bfloat16, "v_cache", 4)
    _need(block_tables, torch.int32, "block_tables", 2)
    _need(context_lens, torch.int32, "context_lens", 1)
    S, Hq, D = q.shape
    NB, BS, Hkv, Dc = k_cache.shape
    if Dc != D or tuple(out.shape) != (S, Hq, D) or block_tables.shape[0] != S or \
            context_lens.shape[0] != S or tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError("paged_decode_attn: inconsistent shapes")
    st = lib.pkv_paged_decode_attn(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
        _ptr(context_lens), S, Hq, Hkv, D, BS, block_tables.shape[1], NB, int(max_total_blocks),
        float(scale), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _ptr(dev_status), _stream(stream))
    _check(st, "pkv_paged_decode_attn")


def paged_decode_store_attn(out, q, k, v, slot_mapping, k_cache, v_cache, block_tables,
                            context_lens, scale, workspace, max_total_blocks, dev_status=None,
                            stream=None) -> None:
    """One decode step: store k/v [S, Hkv, D] (row s = the newest token of
    sequence s) at slot_mapping [S] and attend, fused (see include/pkv.h)."""
    import torch

    lib = load()
    for name, t, dt, nd in (("out", out, torch.bfloat16, 3), ("q", q, torch.bfloat16, 3),
                            ("k", k, torch.bfloat16, 3), ("v", v, torch.bfloat16, 3),
                            ("slot_mapping", slot_mapping, torch.int32, 1),
                            ("k_cache", k_cache, torch.bfloat16, 4),
                            ("v_cache", v_cache, torch.bfloat16, 4),
                            ("block_tables", block_tables, torch.int32, 2),
                            ("context_lens", context_lens, torch.int32, 1)):
        _need(t, dt, name, nd)
    S, Hq, D = q.shape
    NB, BS, Hkv, _ = k_cache.shape
    if tuple(k.shape) != (S, Hkv, D) or tuple(v.shape) != (S, Hkv, D) or \
            slot_mapping.shape[0] != S or tuple(out.shape) != (S, Hq, D):
        raise ValueError("paged_decode_store_attn: inconsistent shapes")
    st = lib.pkv_paged_decode_store_attn(
        _ptr(out), _ptr(q), _ptr(k), _ptr(v), _ptr(slot_mapping), _ptr(k_cache), _ptr(v_cache),
        _ptr(block_tables), _ptr(context_lens), S, Hq, Hkv, D, BS, block_tables.shape[1], NB,
        int(max_total_blocks), float(scale), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(dev_status), _stream(stream))
    _check(st, "pkv_paged_decode_store_attn")


def paged_decode_attn_noalloc(out, q, k_cache, v_cache, block_tables, context_lens, scale,
                              max_total_blocks, dev_status=None, stream=None) -> None:
    """paged_decode_attn for callers that cannot allocate a workspace: the
    scratch is a fixed 16 MiB array inside the library (see include/pkv.h).
    Calls that overlap on the GPU must not be issued: they share that array."""
    import torch

    lib = load()
    for name, t, dt, nd in (("out", out, torch.bfloat16, 3), ("q", q, torch.bfloat16, 3),
                            ("k_cache", k_cache, torch.bfloat16, 4),
                            ("v_cache", v_cache, torch.bfloat16, 4),
                            ("block_tables", block_tables, torch.int32, 2),
                            ("context_lens", context_lens, torch.int32, 1)):
        _need(t, dt, name, nd)
    S, Hq, D = q.shape
    NB, BS, Hkv, _ = k_cache.shape
    st = lib.pkv_paged_decode_attn_noalloc(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
        _ptr(context_lens), S, Hq, Hkv, D, BS, block_tables.shape[1], NB, int(max_total_blocks),
        float(scale), _ptr(dev_status), _stream(stream))
    _check(st, "pkv_paged_decode_attn_noalloc")


def test_decode_fault(wait_limit_ns: int, withhold_tile: int) -> None:
    """TEST ONLY: shorten the decode kernels' wait limit on the current device
    and make every decode CTA skip loading its tile number `withhold_tile`
    (-1: none), so that a decode call times out and reports PKV_DEV_TIMEOUT.
    Restore with test_decode_fault(10**9, -1)."""
    _check(load().pkv_test_decode_fault(int(wait_limit_ns), int(withhold_tile)),
           "test_decode_fault")


def prefill_workspace(device="cuda"):
    """A zero-filled prefill workspace (the work counter the kernel's CTAs
    share; every call leaves it zeroed).  Calls that may overlap on the GPU
    need workspaces of their own."""
    import torch

    n = int(load().pkv_prefill_workspace_size())
    return torch.zeros(n, dtype=torch.uint8, device=device)


_prefill_ws = {}


def _default_prefill_workspace(device, stream):
    # One workspace per (device, stream): calls on one stream are serialised.
    key = (device.index, _stream(stream))
    ws = _prefill_ws.get(key)
    if ws is None:
        ws = _prefill_ws[key] = prefill_workspace(device)
    return ws


def paged_prefill_attn(out, q, k_cache, v_cache, block_tables, cu_seqlens_q, cu_seqlens_k,
                       max_seqlen_q, scale, workspace=None, dev_status=None, stream=None) -> None:
    """out/q [T, Hq, D] bf16 packed by cu_seqlens_q; keys from the paged cache.
    workspace: from prefill_workspace(); by default one cached per stream."""
    import torch

    lib = load()
    _need(out, torch.bfloat16, "out", 3)
    _need(q, torch.bfloat16, "q", 3)
    _need(k_cache, torch.bfloat16, "k_cache", 4)
    _need(v_cache, torch.bfloat16, "v_cache", 4)
    _need(block_tables, torch.int32, "block_tables", 2)
    _need(cu_seqlens_q, torch.int32, "cu_seqlens_q", 1)
    _need(cu_seqlens_k, torch.int32, "cu_seqlens_k", 1)
    T, Hq, D = q.shape
    NB, BS, Hkv, Dc = k_cache.shape
    S = cu_seqlens_q.shape[0] - 1
    if Dc != D or tuple(out.shape) != (T, Hq, D) or block_tables.shape[0] != S or \
            cu_seqlens_k.shape[0] != S + 1 or tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError("paged_prefill_attn: inconsistent shapes")
    if workspace is None:
        workspace = _default_prefill_workspace(q.device, stream)
    st = lib.pkv_paged_prefill_attn(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(cu_seqlens_q),
        _ptr(cu_seqlens_k), S, T, int(max_seqlen_q), Hq, Hkv, D, BS, block_tables.shape[1], NB,
        float(scale), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _ptr(dev_status), _stream(stream))
    _check(st, "pkv_paged_prefill_attn")


def _check_args(what, key_weights, k_cache, args, dev_status):
    """The checks of the key-weight calls: every tensor's dtype, rank, layout
    and device (all on the current one: the library launches there), and
    key_weights' shape.  args: (name, tensor or None, dtype, rank).  Says what is
    wrong, if anything is; the calls ask _plain first."""
    import torch

    dev = _device_of(k_cache)
    for name, t, dtype, ndim in args:
        if t is not None and (t.dtype is not dtype or t.get_device() != dev or dev < 0 or
                              t.dim() != ndim or not t.is_contiguous()):
            _need(t, dtype, name, ndim)
            raise ValueError(f"{what}: {name} is not on the current CUDA device")
    if dev_status is not None and (dev_status.dtype is not torch.int32 or
                                   dev_status.get_device() != dev or dev_status.numel() < 1):
        raise ValueError(f"{what}: dev_status must be an int32 tensor on the current CUDA device")
    NB, BS, Hkv, _ = k_cache.shape
    if key_weights.shape != (NB, Hkv, BS):
        raise ValueError(f"key_weights: expected [num_blocks, Hkv, block_size] = {(NB, Hkv, BS)}")


def _plain(dev, dtype, *tensors) -> bool:
    """Whether all are contiguous, of dtype and on device dev (a few microseconds a
    call are mostly such checks: no names, no objects)."""
    for t in tensors:
        if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
            return False
    return dev >= 0


def _plain_status(dev, dev_status) -> bool:
    import torch

    return dev_status is None or _plain(dev, torch.int32, dev_status) and dev_status.numel() > 0


def _device_of(k_cache) -> int:
    import torch

    return torch.cuda.current_device() if k_cache.is_cuda else -1


def _raw_stream(stream, dev) -> int:
    import torch

    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return int(getattr(stream, "cuda_stream", stream))


def _addr(t):
    return None if t is None else t.data_ptr()


def _workspace(n, what, device):
    import torch

    if n == 0:
        raise ValueError(f"{what}: no workspace for these sizes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def decode_weights_workspace(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                             max_total_blocks, device="cuda"):
    """Allocate a workspace for paged_decode_weights_attn."""
    ints = map(_c_int32, (num_seqs, num_q_heads, num_kv_heads, head_dim, block_size))
    n = int(load().pkv_decode_weights_workspace_size(*ints, _c_int64(max_total_blocks)))
    return _workspace(n, "decode_weights_workspace", device)


def paged_decode_weights_attn(out, key_weights, q, k_cache, v_cache, block_tables, context_lens,
                              scale, workspace, max_total_blocks, k=None, v=None,
                              slot_mapping=None, dev_status=None, stream=None) -> None:
    """paged_decode_attn (with k, v [S, Hkv, D] and slot_mapping [S]:
    paged_decode_store_attn) that also adds the weight each key received to
    key_weights [NB, Hkv, BS] (fp32) and sets the newest key's."""
    import torch

    lib = load()
    if not (k is None) == (v is None) == (slot_mapping is None):
        raise ValueError("paged_decode_weights_attn: k, v and slot_mapping go together")
    bf16, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    dev = _device_of(k_cache)
    q_shape, cache_shape, table_shape = q.shape, k_cache.shape, block_tables.shape
    if not (_plain_status(dev, dev_status) and _plain(dev, bf16, out, q, k_cache, v_cache) and
            _plain(dev, i32, block_tables, context_lens) and _plain(dev, f32, key_weights) and
            _plain(dev, torch.uint8, workspace) and
            (k is None or _plain(dev, bf16, k, v) and _plain(dev, i32, slot_mapping)) and
            len(q_shape) == 3 and len(cache_shape) == 4 and len(table_shape) == 2):
        _check_args("paged_decode_weights_attn", key_weights, k_cache, (
            ("out", out, bf16, 3), ("q", q, bf16, 3), ("k", k, bf16, 3), ("v", v, bf16, 3),
            ("slot_mapping", slot_mapping, i32, 1), ("k_cache", k_cache, bf16, 4),
            ("v_cache", v_cache, bf16, 4), ("block_tables", block_tables, i32, 2),
            ("context_lens", context_lens, i32, 1), ("workspace", workspace, torch.uint8, 1),
            ("key_weights", key_weights, f32, 3)), dev_status)
    S, Hq, D = q_shape
    NB, BS, Hkv, Dc = cache_shape
    if Dc != D or out.shape != q_shape or table_shape[0] != S or context_lens.shape != (S,) or \
            v_cache.shape != cache_shape or key_weights.shape != (NB, Hkv, BS):
        raise ValueError("paged_decode_weights_attn: inconsistent shapes")
    if k is not None and (k.shape != (S, Hkv, D) or v.shape != (S, Hkv, D) or
                          slot_mapping.shape != (S,)):
        raise ValueError("paged_decode_weights_attn: inconsistent shapes of the new tokens")
    st = lib.pkv_paged_decode_weights_attn(
        out.data_ptr(), key_weights.data_ptr(), q.data_ptr(), _addr(k), _addr(v),
        _addr(slot_mapping), k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(),
        context_lens.data_ptr(), S, Hq, Hkv, D, BS, table_shape[1], NB,
        _c_int64(max_total_blocks), float(scale), workspace.data_ptr(), workspace.numel(),
        _addr(dev_status), _raw_stream(stream, dev))
    _check(st, "pkv_paged_decode_weights_attn")


def prefill_weights_workspace(num_seqs, total_q, max_seqlen_q, window, num_q_heads, num_kv_heads,
                              max_blocks_per_seq, block_size, device="cuda"):
    """Allocate a zero-filled workspace for paged_prefill_weights (filled on the
    current stream: calls on another one wait for it)."""
    ints = map(_c_int32, (max_seqlen_q, window, num_q_heads, num_kv_heads, max_blocks_per_seq,
                          block_size))
    n = int(load().pkv_prefill_weights_workspace_size(_c_int32(num_seqs), _c_int64(total_q),
                                                      *ints))
    return _workspace(n, "prefill_weights_workspace", device)


def _c_int32(x) -> int:
    """An int argument as the library sees it: what does not fit stays too large
    or becomes -1 (refused there), instead of wrapping around."""
    return max(-1, min(int(x), 0x7FFFFFFF))


def _c_int64(x) -> int:
    """The same for an int64 argument."""
    return max(-1, min(int(x), 0x7FFFFFFFFFFFFFFF))


def paged_prefill_weights(key_weights, q, k_cache, block_tables, cu_seqlens_q, cu_seqlens_k,
                          max_seqlen_q, window, scale, workspace, dev_status=None,
                          stream=None) -> None:
    """Adds to key_weights [NB, Hkv, BS] (fp32) the weight that the last
    `window` queries of each prompt chunk give to the keys cached before it,
    and sets the sums of the chunk's own keys (arguments as for
    paged_prefill_attn, beside which it is called)."""
    import torch

    lib = load()
    bf16, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    dev = _device_of(k_cache)
    q_shape, cache_shape, table_shape = q.shape, k_cache.shape, block_tables.shape
    if not (_plain_status(dev, dev_status) and _plain(dev, bf16, q, k_cache) and
            _plain(dev, i32, block_tables, cu_seqlens_q, cu_seqlens_k) and
            _plain(dev, f32, key_weights) and _plain(dev, torch.uint8, workspace) and
            len(q_shape) == 3 and len(cache_shape) == 4 and len(table_shape) == 2):
        _check_args("paged_prefill_weights", key_weights, k_cache, (
            ("q", q, bf16, 3), ("k_cache", k_cache, bf16, 4),
            ("block_tables", block_tables, i32, 2), ("cu_seqlens_q", cu_seqlens_q, i32, 1),
            ("cu_seqlens_k", cu_seqlens_k, i32, 1), ("workspace", workspace, torch.uint8, 1),
            ("key_weights", key_weights, f32, 3)), dev_status)
    T, Hq, D = q_shape
    NB, BS, Hkv, Dc = cache_shape
    S = table_shape[0]
    if Dc != D or cu_seqlens_q.shape != (S + 1,) or cu_seqlens_k.shape != (S + 1,) or \
            key_weights.shape != (NB, Hkv, BS):
        raise ValueError("paged_prefill_weights: inconsistent shapes")
    st = lib.pkv_paged_prefill_weights(
        key_weights.data_ptr(), q.data_ptr(), k_cache.data_ptr(), block_tables.data_ptr(),
        cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), S, T, _c_int32(max_seqlen_q),
        _c_int32(window), Hq, Hkv, D, BS, table_shape[1], NB, float(scale),
        workspace.data_ptr(), workspace.numel(), _addr(dev_status), _raw_stream(stream, dev))
    _check(st, "pkv_paged_prefill_weights")


def test_prompt_fault(wait_limit_ns: int, which_pass: int, loading_ctas: int) -> None:
    """TEST ONLY: shorten the wait limit of paged_prefill_weights on the current
    device and let only the first `loading_ctas` CTAs of its first or second pass load
    their tiles (-1: all).  Restore with test_prompt_fault(10**9, 1, -1)."""
    _check(load().pkv_test_prompt_fault(int(wait_limit_ns), int(which_pass), int(loading_ctas)),
           "test_prompt_fault")


def kv_evict(k_cache, v_cache, key_weights, block_tables, context_lens, budget, recent, kept,
             new_lens, dev_status=None, stream=None) -> None:
    """Shortens every sequence longer than `budget` to its last `recent` tokens
    and, per kv head, the heaviest others by key_weights, in place.
    kept [S, Hkv, budget] int32: the old position of what is now at each place;
    new_lens [S] int32: the new context lengths (see include/pkv.h)."""
    import torch

    lib = load()
    bf16, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    dev = _device_of(k_cache)
    cache_shape, table_shape = k_cache.shape, block_tables.shape
    if not (_plain_status(dev, dev_status) and _plain(dev, bf16, k_cache, v_cache) and
            _plain(dev, i32, block_tables, context_lens, kept, new_lens) and
            _plain(dev, f32, key_weights) and len(cache_shape) == 4 and len(table_shape) == 2):
        _check_args("kv_evict", key_weights, k_cache, (
            ("k_cache", k_cache, bf16, 4), ("v_cache", v_cache, bf16, 4),
            ("block_tables", block_tables, i32, 2), ("context_lens", context_lens, i32, 1),
            ("kept", kept, i32, 3), ("new_lens", new_lens, i32, 1),
            ("key_weights", key_weights, f32, 3)), dev_status)
    NB, BS, Hkv, D = cache_shape
    S = table_shape[0]
    if v_cache.shape != cache_shape or context_lens.shape != (S,) or new_lens.shape != (S,) or \
            kept.shape != (S, Hkv, int(budget)) or key_weights.shape != (NB, Hkv, BS):
        raise ValueError("kv_evict: inconsistent shapes")
    st = lib.pkv_kv_evict(k_cache.data_ptr(), v_cache.data_ptr(), key_weights.data_ptr(),
                          block_tables.data_ptr(), context_lens.data_ptr(), S, Hkv, D, BS,
                          table_shape[1], NB, _c_int32(budget), _c_int32(recent),
                          kept.data_ptr(), new_lens.data_ptr(), _addr(dev_status), _raw_stream(stream, dev))
    _check(st, "pkv_kv_evict")


def w4a16_dequant(out, packed, scales, group_size=128, stream=None) -> None:
    """out [N, K] bf16 <- packed [N, K/8] int32 (eight 4-bit values per word,
    lowest nibble first, value = nibble - 8) times scales [N, K/128] bf16."""
    import torch

    lib = load()
    _need(out, torch.bfloat16, "out", 2)
    _need(packed, torch.int32, "packed", 2)
    _need(scales, torch.bfloat16, "scales", 2)
    N, K = out.shape
    if tuple(packed.shape) != (N, K // 8) or tuple(scales.shape) != (N, K // group_size):
        raise ValueError("w4a16_dequant: inconsistent shapes")
    st = lib.pkv_w4a16_dequant(_ptr(out), _ptr(packed), _ptr(scales), N, K, int(group_size),
                               _stream(stream))
    _check(st, "pkv_w4a16_dequant")


class BlockManager:
    """Host allocator of the cache's blocks with reference counts and
    hash-chained prefix sharing (the library's pkv_bm_* calls; no GPU work).

        bm = BlockManager(num_blocks, block_size=256)
        cached = bm.allocate(seq_id, prompt_tokens)   # leading tokens already in reused blocks
        slots = bm.slots(seq_id, cached, len(prompt_tokens) - cached)
        row = bm.block_table(seq_id, max_blocks)
        bm.append(seq_id, token); bm.free(seq_id)
    """

    def __init__(self, num_blocks: int, block_size: int = 256):
        self._lib = load()
        self._h = self._lib.pkv_bm_create(int(num_blocks), int(block_size))
        if not self._h:
            raise ValueError("BlockManager: bad sizes or out of host memory")
        self.num_blocks, self.block_size = int(num_blocks), int(block_size)

    def close(self):
        if getattr(self, "_h", None):
            self._lib.pkv_bm_destroy(self._h)
            self._h = None

    def __del__(self):
        self.close()

    @property
    def num_free_blocks(self) -> int:
        return int(self._lib.pkv_bm_num_free_blocks(self._h))

    def allocate(self, seq_id: int, tokens) -> int:
        import numpy as np

        t = np.ascontiguousarray(tokens, dtype=np.int32)
        cached = ctypes.c_int(0)
        _check(self._lib.pkv_bm_allocate(self._h, int(seq_id), t.ctypes.data, int(t.size),
                                         ctypes.byref(cached)), "pkv_bm_allocate")
        return int(cached.value)

    def append(self, seq_id: int, token: int) -> None:
        _check(self._lib.pkv_bm_append(self._h, int(seq_id), int(token)), "pkv_bm_append")

    def free(self, seq_id: int) -> None:
        _check(self._lib.pkv_bm_free(self._h, int(seq_id)), "pkv_bm_free")

    def evict(self, seq_id: int, keep_tokens: int) -> None:
        """The sequence is cut to its first keep_tokens places by kv_evict on
        its table as it was before this call; raises, changing nothing, when
        another sequence shares one of the blocks that eviction would rewrite."""
        _check(self._lib.pkv_bm_evict(self._h, int(seq_id), _c_int32(keep_tokens)), "pkv_bm_evict")

    def num_tokens(self, seq_id: int) -> int:
        return int(self._lib.pkv_bm_num_tokens(self._h, int(seq_id)))

    def block_table(self, seq_id: int, max_blocks: int):
        import numpy as np

        out = np.empty(int(max_blocks), dtype=np.int32)
        n = self._lib.pkv_bm_block_table(self._h, int(seq_id), out.ctypes.data, int(max_blocks))
        if n < 0:
            raise KeyError(seq_id)
        return out

    def slots(self, seq_id: int, first: int, count: int):
        import numpy as np

        out = np.empty(int(count), dtype=np.int32)
        _check(self._lib.pkv_bm_slots(self._h, int(seq_id), int(first), int(count),
                                      out.ctypes.data), "pkv_bm_slots")
        return out

    def ref_count(self, block: int) -> int:
        return int(self._lib.pkv_bm_ref_count(self._h, int(block)))
