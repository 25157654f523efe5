import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line(
        "markers", "gpu: needs a CUDA GPU (GB300, sm_103a) and the built libflce.so")
    config.addinivalue_line(
        "markers", "slow: full-size parity case (minutes of host fp64 work)")


# Hand made-up addresses to the library and count on the missing device to end the call: on a GPU
# the kernels would use them.
WITHOUT_DEVICE = ("test_operators_host.py::test_grad_overlaps",)


def pytest_collection_modifyitems(config, items):
    try:
        import torch
        has_gpu = torch.cuda.is_available()
    except Exception:  # pragma: no cover
        has_gpu = False
    if has_gpu:
        skip = pytest.mark.skip(reason="passes made-up addresses, for machines without a GPU")
        for item in items:
            if item.nodeid.endswith(WITHOUT_DEVICE):
                item.add_marker(skip)
        return
    skip = pytest.mark.skip(reason="no CUDA device in this process")
    for item in items:
        if "gpu" in item.keywords:
            item.add_marker(skip)
