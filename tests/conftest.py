import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (GB300, sm_103a)")
    config.addinivalue_line("markers", "slow: long-running CPU test")


@pytest.fixture(scope="session")
def orc():
    import oracle
    oracle.build()
    return oracle


@pytest.fixture(scope="module", autouse=True)
def operators_status(request):
    """After each file of the operators' GPU tests: no kernel's bounded wait gave up.  (A wait that
    did leaves outputs unwritten, which a test that does not compare them all would not see.)"""
    if not request.module.__name__.split(".")[-1].startswith("test_gpu_ops_"):
        yield
        return
    import torch
    from bit_exact_fp8_gb300 import _lib
    if torch.cuda.is_available():
        _lib.emu_ops_device_status(reset=True)
    yield
    if torch.cuda.is_available():
        assert _lib.emu_ops_device_status() == 0
