import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (GB300, sm_103a)")
    config.addinivalue_line("markers", "slow: takes more than a few seconds")


# Tests that hold a wrong value: they stay as they are, run, and have to fail on it.
WRONG_VALUE = {
    "test_gpu_cache_shrinking.py::test_mxfp4_append_and_read[":
        "expects zeros of MXFP4 blocks with scale byte 0, whose values are code * 2^-127 by the format "
        "(and in oracle/mxfp4.py); test_mxfp4_append_and_read_of_every_scale has the same inputs",
}


def pytest_collection_modifyitems(config, items):
    for item in items:
        for name, why in WRONG_VALUE.items():
            if name in item.nodeid:
                item.add_marker(pytest.mark.xfail(reason=why, raises=AssertionError, strict=True))
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


def load_golden(name):
    """key = value fixtures under tests/golden (comments after '#')."""
    out = {}
    with open(os.path.join(ROOT, "tests", "golden", name)) as f:
        for line in f:
            line = line.split("#", 1)[0].strip()
            if not line:
                continue
            k, v = (s.strip() for s in line.split("=", 1))
            out[k] = v
    return out
