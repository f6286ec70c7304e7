"""ibp_select_pages over bounds that are infinite, as a page's with an
overflowed key are: the score is by its definition, max(q lo, q hi) of each
number, so an infinite bound that q does not use changes nothing, and one that
it does puts the page first."""
from __future__ import annotations

import math

import pytest
import torch

from lossless_tensor_compression_ibp_amd import ibp
from tests.kv_util import Pool, values
from tests.select_util import FORMS, compare, select

pytestmark = pytest.mark.gpu

INFINITE = {"lo": (-math.inf, None), "hi": (None, math.inf), "lo and hi": (-math.inf, math.inf),
            "both above": (math.inf, math.inf), "both below": (-math.inf, -math.inf)}


@pytest.mark.parametrize("rows,n", FORMS)
@pytest.mark.parametrize("sign", [1, -1, 0])
@pytest.mark.parametrize("which", INFINITE)
def test_infinite_bounds(rows, n, sign, which):
    """Every 17th page has an infinite bound in one dim; sign: of q there (0:
    a head of each)."""
    lo, hi = INFINITE[which]

    def some(b):
        if lo is not None:
            b[::17, 0, 9] = lo
        if hi is not None:
            b[::17, 1, 9] = hi
        return b

    def queries(q):
        q[:, :, 9] = q[:, :, 9].abs() + 0.1
        if sign <= 0:
            q[:, 1:, 9] *= -1
        if sign < 0:
            q[:, :1, 9] *= -1
        return q

    compare(rows, n, 2, 64, "fp16", queries, some, seed=n)


@pytest.mark.parametrize("rows,n", FORMS)
@pytest.mark.parametrize("group", [1, 4, 17])
def test_infinite_bounds_in_several_dims(rows, n, group):
    """Sums of +infinity and -infinity, and zeros of q: NaN, ranked last."""
    def some(b):
        b[::7, 0, 3], b[::5, 1, 4], b[::11, :, 100] = -math.inf, math.inf, -math.inf
        return b

    def queries(q):
        q[:, 0, 3] = 0
        return q

    compare(rows, n, group, 128, "bf16", queries, some, seed=group, kv_heads=2)


@pytest.mark.parametrize("dim", [64, 256])
def test_a_page_with_an_overflowed_key_is_found(dim):
    """From the pages: one key overflowed, and the queries point its way."""
    x = values(400, 16, dim, torch.float16, dim)
    x[123, 7, 5] = math.inf
    x[200, 3, 6] = -math.inf
    p = Pool(x, None)
    b = torch.zeros(400, 2, dim, dtype=torch.float16, device="cuda")
    ibp.ibp_page_bounds(p.pages, torch.arange(400, device="cuda"), None, b)
    q = torch.randn(1, 1, dim, device="cuda").half()
    q[:, :, 5], q[:, :, 6] = 1, -1
    t = torch.arange(400, device="cuda").reshape(1, 1, 400).contiguous()
    got = select(q, b, t, [6400], [0], 16, 2, 0, 0)
    assert got.flatten().tolist() == [123, 200]
