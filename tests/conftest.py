import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA device (B200, sm_100a)")
    config.addinivalue_line("markers", "slow: full-size workload (minutes)")


@pytest.fixture(scope="session")
def cuda_dev():
    import torch

    if not torch.cuda.is_available():
        pytest.fail("this test needs a CUDA device")
    return torch.device("cuda:0")


@pytest.hookimpl(tryfirst=True)
def pytest_runtest_setup(item):
    """The bounded-wait tests load the test-only library as they find it: it is brought up to
    date with the sources first (an error where that cannot be done)."""
    if "dbg" in getattr(item, "fixturenames", ()):
        from top_sparse_attention_02_b200 import build

        build.ensure(debug=True)
