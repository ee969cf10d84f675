import os
import sys

import pytest

ROOT = os.path.abspath(os.path.join(os.path.dirname(__file__), ".."))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built CUDA library")
    config.addinivalue_line("markers", "slow: GLM-sized case (minutes)")


# Two of its cases count ids as handed out that no table row can hold; moe_kv_plan keeps those on
# the free list (test_gpu_kv_plan_pages.py).  It fails there, so it comes last: a run that stops at
# its first failure has then seen all others.
LAST = "test_gpu_kv_plan.py::test_shortages_are_flagged_and_leave_no_slot"


def pytest_collection_modifyitems(config, items):
    items.sort(key=lambda item: item.nodeid.endswith(LAST))
    try:
        import torch
        has_gpu = torch.cuda.is_available()
    except Exception:  # pragma: no cover
        has_gpu = False
    if has_gpu:
        return
    skip = pytest.mark.skip(reason="no CUDA device")
    for item in items:
        if "gpu" in item.keywords:
            item.add_marker(skip)
