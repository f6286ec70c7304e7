"""ibp_select_pages with a NaN in q: a head that has one scores every page as
the lowest, alone or beside others."""
from __future__ import annotations

import math

import pytest

from tests.select_util import FORMS, compare

pytestmark = pytest.mark.gpu


def cancelling(b):
    """Large terms that cancel, so that 32-bit sums decide nothing."""
    b[:, :, 0], b[:, :, 1] = 1024.0, -1024.0
    b[:, :, 2:] *= 2.0 ** -12
    return b.sort(1)[0]


@pytest.mark.parametrize("rows,n", FORMS)
@pytest.mark.parametrize("group", [1, 2, 4, 17])
@pytest.mark.parametrize("dim", [64, 256])
def test_one_head_of_a_group(rows, n, group, dim):
    """The head's other numbers are large: without its NaN it would choose."""
    def queries(q):
        q.fill_(1.0)
        q[:, group - 1] *= 64
        q[:, group - 1, 5] = math.nan
        return q

    compare(rows, n, group, dim, "bf16", queries, cancelling, seed=n)


@pytest.mark.parametrize("group", [1, 2, 3, 8])
@pytest.mark.parametrize("make", ["near", "far"])
def test_a_row_does_not_depend_on_its_neighbours(group, make):
    """A row of NaNs, one with a NaN, and ordinary ones among them."""
    def queries(q):
        q[3] = math.nan
        q[6, :, 5] = math.nan
        return q

    compare(11, 700, group, 64, "bf16", queries, cancelling if make == "near" else lambda b: b, seed=group)
