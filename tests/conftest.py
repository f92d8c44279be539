import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")


# Tests that hold a wrong value: they stay as they are and have to fail.
WRONG = {
    f"test_gpu_routed.py::test_against_64_bits[{case}]":
        "sets the expected d_topk_w of a weight of 0 to 0; out = residual + sum w y has the gradient <dout, y> in w whatever w is "
        "(test_gpu_routed_weights.py)"
    for case in ("60-100-68-5-3-0.7", "300-128-96-8-2-1.0")}


def pytest_collection_modifyitems(items):
    for item in items:
        reason = WRONG.get(item.nodeid.rsplit("/", 1)[-1])
        if reason:
            item.add_marker(pytest.mark.xfail(reason=reason, raises=AssertionError, strict=True))
