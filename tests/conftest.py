import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    # The first double-precision logsumexp of a process was seen to be off by 1e-9 in
    # some runs (9 of 60 with torch 2.11 on x86) when it came after the oracle's OpenMP
    # threads, and never (0 of 60) when torch had computed one before them.
    try:
        import torch
        torch.logsumexp(torch.zeros((64, 64), dtype=torch.float64), -1)
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
