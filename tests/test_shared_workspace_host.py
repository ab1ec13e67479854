"""Sizes of paged_decode_shared_attn's workspace at the ends of what its arguments can say (no GPU)."""
import pytest

import paged_kv_cache_241_gb300 as pkv

MOST = 2**31 - 1


def test_batches_that_no_call_takes_have_no_size():
    """(Their bytes would not fit 64 bits: some came out small, or below the bytes of fewer sequences.)"""
    f = pkv.load().pkv_decode_shared_workspace_size
    for S, Hq, D in ((MOST, 1 << 16, 1 << 16), (1 << 30, 1 << 16, 1 << 14), (MOST, 16, 128), (8193, 16, 128)):
        assert f(S, 1, Hq, 1, D) == 0, S
    with pytest.raises(ValueError, match="no workspace"):
        pkv.decode_shared_workspace(MOST, 1, 1 << 16, 1, 1 << 16)


def test_sizes_of_batches_grow_with_them():
    f = pkv.load().pkv_decode_shared_workspace_size
    for Hq, Hkv, D in ((1 << 16, 1, 1 << 16), (16, 8, 128), (4, 4, 64)):
        sizes = [f(S, N, Hq, Hkv, D) for S, N in ((1, 1), (2, 2), (100, 7), (8192, 1), (8192, 8192), (8192, MOST))]
        assert sizes == sorted(sizes) and sizes[0] > 0
        assert sizes[3] > 8192 * Hq * D * 8  # (fp32 of every row, twice: tails and first parts)
