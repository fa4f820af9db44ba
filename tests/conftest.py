import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built library")


@pytest.fixture(autouse=True)
def _decoded_pages_of_one_test():
    """The Server of test_gpu_packed_flow keeps decoded pages under its id, in a default argument. An id comes back once its
    owner is gone, so nothing of it is carried from one test to the next."""
    yield
    for name, module in list(sys.modules.items()):
        if name.endswith("test_gpu_packed_flow"):
            module.Server.values.__defaults__[0].clear()


@pytest.fixture(scope="session")
def orc():
    import oracle
    oracle.build()
    return oracle


@pytest.fixture(scope="session")
def kap():
    """The CUDA library through its Python binding; GPU tests only."""
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import selected_kv_sparse_gb300 as k
    k.load()
    return k
