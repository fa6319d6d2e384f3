import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")
    config.addinivalue_line("markers", "slow: CPU test that takes more than a few seconds")


@pytest.fixture(scope="module", autouse=True)
def _fresh_scratch(request):
    """GPU modules start without the memory that the library kept for the streams of other modules:
    torch hands the same 32 streams out in turn."""
    if request.node.get_closest_marker("gpu") is not None:
        import torch

        import submanifold_sparse_convolution_amd as sc

        if torch.cuda.is_available():
            torch.cuda.synchronize()
            sc.subm_release_cached_memory()
    yield
