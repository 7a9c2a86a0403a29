import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a B200 (sm_100a) GPU")
    config.addinivalue_line("markers", "slow: full-size workload")


# Holds a value that the formula does not have: rows of 1e30 as zeros, where
# h w / sqrt(mean(h^2) + eps) is w (the norm's squares no longer overflow).  It
# runs last, so that a run with -x reaches every other test.
LAST = {"test_norm_values_that_are_not_finite"}


def pytest_collection_modifyitems(config, items):
    items.sort(key=lambda it: it.name in LAST)
    # GPU tests on a machine without a GPU are skipped, not failed, so that a
    # plain `pytest tests/` still runs the CPU suite here.
    try:
        import torch
        has_gpu = torch.cuda.is_available()
    except Exception:  # pragma: no cover
        has_gpu = False
    if has_gpu:
        return
    skip = pytest.mark.skip(reason="no CUDA device")
    for it in items:
        if "gpu" in it.keywords:
            it.add_marker(skip)
