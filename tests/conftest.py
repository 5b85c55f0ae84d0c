import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


@pytest.fixture(scope="session", autouse=True)
def built():
    """librat.so and _binding.so of these sources, whichever tests are asked for."""
    from recurrence_augmented_dilated_gated_b200 import build

    build.build()


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA device (a B200) and the built library")
    config.addinivalue_line("markers", "slow: large sizes; still runs in the gpu suite")
