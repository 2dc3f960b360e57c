import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)
HERE = os.path.dirname(os.path.abspath(__file__))
if HERE not in sys.path:
    sys.path.insert(0, HERE)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built library")


@pytest.fixture(scope="session")
def orc():
    import oracle
    return oracle.default()


# The refusal tests pass addresses that are nobody's, and of the accepted calls
# among them expect that no device is there to launch on: on one they would fault it.
NO_DEVICE = ("test_abi.py", "test_block_ops_cpu.py", "test_logprob_stats_cpu.py", "test_train_ops_cpu.py")


def pytest_runtest_setup(item):
    if item.path.name in NO_DEVICE and "lib" in getattr(item, "fixturenames", ()):
        import torch
        if torch.cuda.is_available():
            pytest.skip("calls with fake addresses, for a machine without a GPU")
