"""Host checks of norm_rope_store's test hook (no GPU)."""
import paged_kv_cache_241_gb300 as pkv


def test_rope_fault_hook_rejects_bad_arguments():
    lib = pkv.load()
    assert lib.pkv_test_rope_fault(0, -1) == 1
    assert lib.pkv_test_rope_fault(1000, -2) == 1
