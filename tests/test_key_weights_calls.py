"""CPU checks of the key-weight, eviction and block-manager calls beside
test_key_weights_host: nothing here reaches a GPU."""
from test_abi import lib  # noqa: F401  (fixture: the built library, no GPU)


def test_prompt_fault_hook_rejects_bad_arguments(lib):  # noqa: F811
    # checked before any device call
    assert lib.pkv_test_prompt_fault(0, 1, -1) == 1
    assert lib.pkv_test_prompt_fault(1000, 0, -1) == 1 and lib.pkv_test_prompt_fault(1000, 3, -1) == 1
    assert lib.pkv_test_prompt_fault(1000, 2, -2) == 1
