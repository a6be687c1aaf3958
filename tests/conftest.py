import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    # The exponentials of torch's first large double-precision logsumexp may be of reduced
    # accuracy (1e-9) in the part of one thread: on x86 they are MKL's, and its first use
    # by two threads at once was seen to give one of them another variant (14 of 100
    # runs, the same 32 of 64 rows and values each time, right when computed again).  A
    # first use by one thread comes before them all.
    try:
        import torch
        torch.logsumexp(torch.zeros(8, dtype=torch.float64), -1)
    except ImportError:
        pass
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built library")
    config.addinivalue_line("markers", "slow: full-size workloads (minutes)")


def pytest_collection_modifyitems(config, items):
    try:
        import torch
        has_gpu = torch.cuda.is_available()
    except Exception:
        has_gpu = False
    if has_gpu:
        return
    skip = pytest.mark.skip(reason="no CUDA device")
    for item in items:
        if "gpu" in item.keywords:
            item.add_marker(skip)
