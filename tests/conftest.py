import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")


# Cases whose expected value is wrong, kept as they are and expected to fail.
# test_select_infinite_bounds: its reference takes a bound's share of the score
# as max(q, 0) hi + min(q, 0) lo.  With lo = hi = infinity one factor is 0 and
# the share NaN, so the page ranks last; the header's definition is
# max(q lo, q hi), which is infinite there, and the page ranks first.
# test_gpu_select_infinite.py tests the definition.
WRONG_VALUES = {"test_gpu_select_pages.py::test_select_infinite_bounds[inf]",
                "test_gpu_select_pages.py::test_select_infinite_bounds[-inf]"}


def pytest_collection_modifyitems(items):
    for item in items:
        if item.nodeid.split("/")[-1] in WRONG_VALUES:
            item.add_marker(pytest.mark.xfail(strict=True, reason="expects 0 * inf = NaN where the score is infinite"))
