"""CPU checks of the key-weight, eviction and block-manager calls beside
test_key_weights_host: nothing here reaches a GPU."""
import pytest

import paged_kv_cache_241_gb300 as pkv
from test_abi import lib  # noqa: F401  (fixture: the built library, no GPU)
from test_key_weights_host import decode_call, prompt_call


def test_prompt_fault_hook_rejects_bad_arguments(lib):  # noqa: F811
    # checked before any device call
    assert lib.pkv_test_prompt_fault(0, 1, -1) == 1
    assert lib.pkv_test_prompt_fault(1000, 0, -1) == 1 and lib.pkv_test_prompt_fault(1000, 3, -1) == 1
    assert lib.pkv_test_prompt_fault(1000, 2, -2) == 1


# ------------------------------------------------- ints that the library has no room for

def test_manager_evict_does_not_wrap(lib):  # noqa: F811
    bm = pkv.BlockManager(12, 4)
    bm.allocate(1, list(range(18)))
    bm.evict(1, (1 << 32) + 5)                              # far more than it has: nothing to cut
    assert bm.num_tokens(1) == 18
    for bad in (0, -1, -(1 << 32) + 5):
        with pytest.raises(pkv.PkvError, match="INVALID"):
            bm.evict(1, bad)
    assert bm.num_tokens(1) == 18


def test_workspaces_do_not_wrap(lib):  # noqa: F811
    """A size that does not fit is as large as fits, or refused: never a small one."""
    big = 1 << 32
    sizes = dict(num_seqs=4, total_q=100, max_seqlen_q=50, window=1 << 20, num_q_heads=16, num_kv_heads=8,
                 max_blocks_per_seq=4, block_size=256)
    # more queries a sequence than the call has: each counted once, as with 100
    whole = pkv.prefill_weights_workspace(**dict(sizes, max_seqlen_q=100), device="cpu").numel()
    assert pkv.prefill_weights_workspace(**dict(sizes, max_seqlen_q=big + 5), device="cpu").numel() == whole
    # more sequences than queries: a row of statistics for each query
    rows = 100 * 16 * 4
    assert rows <= pkv.prefill_weights_workspace(**dict(sizes, num_seqs=big + 4), device="meta").numel() < rows + (2 << 20)
    for name in ("total_q", "num_q_heads", "num_kv_heads", "max_blocks_per_seq", "block_size"):
        for wrapped in (big + sizes[name], (1 << 64) + sizes[name]):
            with pytest.raises(ValueError, match="no workspace"):
                pkv.prefill_weights_workspace(**dict(sizes, **{name: wrapped}), device="meta")
    sizes = dict(num_seqs=4, num_q_heads=16, num_kv_heads=8, head_dim=128, block_size=256, max_total_blocks=32)
    for name in ("num_q_heads", "num_kv_heads", "head_dim", "block_size", "max_total_blocks"):
        with pytest.raises(ValueError, match="no workspace"):
            pkv.decode_weights_workspace(**dict(sizes, **{name: (1 << 64) + sizes[name]}), device="meta")
    assert pkv.decode_weights_workspace(**dict(sizes, num_seqs=big + 4), device="meta").numel() > 1 << 40


# ------------------------------------------------------------------ buffers that overlap

def test_evict_rejects_buffers_that_overlap(lib):  # noqa: F811
    base = dict(kc=1 << 40, vc=1 << 41, kw=1 << 42, bt=1 << 43, cl=1 << 44, S=4, Hkv=8, D=128, BS=256, maxb=8, NB=64,
                budget=1024, recent=32, kept=1 << 45, nl=1 << 46, st=None, stream=None)
    cache = 64 * 256 * 8 * 128 * 2
    # (refused before any launch: there is no GPU here, and what is not refused fails to launch)
    for kw in (dict(vc=base["kc"]), dict(vc=base["kc"] + cache - 16), dict(vc=base["kc"] - cache + 16),
               dict(vc=base["kc"] + 16, NB=1 << 62), dict(vc=base["kc"] + 16, NB=(1 << 63) - 1),
               dict(nl=base["cl"]), dict(nl=base["cl"] + 12), dict(nl=base["cl"] - 12)):
        assert lib.pkv_kv_evict(*dict(base, **kw).values()) == 1, kw


# ----------------------------------------------------------------------- the scale

def test_scales_that_overflow_in_base_two_are_refused(lib):  # noqa: F811
    # (checked before the batch's size: S = 0 and T = 0 launch nothing)
    for scale in (3.0e38, -3.0e38, 2.4e38):                 # times log2(e): past 3.4e38
        assert decode_call(lib, S=0, scale=scale) == 1
        assert prompt_call(lib, T=0, scale=scale) == 1
    for scale in (2.3e38, -2.3e38, 0.0):
        assert decode_call(lib, S=0, scale=scale) == 0
        assert prompt_call(lib, T=0, scale=scale) == 0
