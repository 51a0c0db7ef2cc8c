import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built library")


# Holds a wrong value: it expects infinity where h exceeds fp16's range, for sums that are finite in Y's type
# (test_projection_f16 has their exact values).  Last, so that a run that stops at a failure has run the others.
HOLDS_A_WRONG_VALUE = ("test_gpu_adapters.py::test_infinite_in_16_bits_is_not_nan",)


def pytest_collection_modifyitems(items):
    items.sort(key=lambda item: item.nodeid.endswith(HOLDS_A_WRONG_VALUE))
