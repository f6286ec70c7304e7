"""ibp_select_pages where 32-bit products underflow: the scores are sums in 64
bits, rounded to 32 bits once, numbers below the normal range included."""
from __future__ import annotations

import pytest

from tests.select_util import FORMS, compare

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,n", FORMS)
@pytest.mark.parametrize("q_scale,b_scale", [(1e-20, 1e-20), (1e-19, 3e-24), (1e-2, 1e-38), (1e30, 1e-39), (1e-39, 1e30),
                                             (1e-22, 1e-20), (1e-22, 1e-22), (1e-23, 3e-22), (1.0, 0.0), (0.0, 1.0)])
def test_tiny_products(rows, n, q_scale, b_scale):
    """Scores of 1e-39 down to 1e-43 (below the normal range of 32 bits, the
    last a few hundred of its steps), products of numbers below the normal range
    of bf16 with large ones, and zeros."""
    compare(rows, n, 2, 64, "bf16", lambda q: (q.double() * q_scale).to(q.dtype),
            lambda b: (b.double() * b_scale).to(b.dtype), seed=n)


@pytest.mark.parametrize("rows,n", FORMS)
def test_tiny_products_beside_zeros(rows, n):
    """Most pages have no score at all, a few one below the normal range."""
    def few(b):
        keep = b[::37].double() * 1e-20
        b.zero_()
        b[::37] = keep.to(b.dtype)
        return b

    compare(rows, n, 1, 128, "bf16", lambda q: (q.double() * 1e-20).to(q.dtype), few, seed=n)
