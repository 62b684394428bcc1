import os
import sys

import pytest

# The oracle's products run on numpy's threads and its conversions on torch's, in
# turn, and torch's spin for the next one while numpy's want the cores: one layer
# of the "small" model takes 1.6 s on 16 cores with them spinning, 0.3 s without.
# Read when torch is first imported, here and in the tests' child processes.
os.environ.setdefault("OMP_WAIT_POLICY", "passive")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA device (B200, sm_100a)")
    config.addinivalue_line("markers", "slow: long-running CPU test")


@pytest.fixture(scope="session")
def cuda_available():
    import torch
    return torch.cuda.is_available()
