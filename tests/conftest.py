import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built library")
    config.addinivalue_line("markers", "by_choice: decode over shared prefixes shares them only where it pays")


@pytest.fixture(scope="session")
def lib():
    """The CUDA library through its Python binding; fails loudly when missing."""
    import torch

    if not torch.cuda.is_available():
        pytest.fail("GPU test collected on a machine without a GPU; run with -m 'not gpu'")
    import paged_kv_cache_241_gb300 as pkv

    pkv.load()  # raises if the shared library was not built
    return pkv
