"""Errors in the pool of values: latched on its own handle, and on the keys',
which stands for the whole call."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from lossless_tensor_compression_ibp_amd import ibp
from tests.kv_util import Pool, values

pytestmark = pytest.mark.gpu

T, D = 16, 128


def run(kp, vp, rows, kt=None, vt=None, sparse=False):
    n = kp.n
    t = torch.arange(n, device="cuda").reshape(1, 1, n).contiguous()
    kt, vt = t if kt is None else kt, t if vt is None else vt
    q = torch.randn(rows, 2, D, device="cuda").bfloat16()
    out = torch.empty_like(q)
    lens = torch.full((rows if sparse else 1,), n * T, dtype=torch.int32, device="cuda")
    if sparse:
        blocks = torch.arange(n, dtype=torch.int32, device="cuda").expand(rows, 1, n).contiguous()
        ibp.ibp_sparse_attention(kp.pages, vp.pages, q, kt, vt, lens, blocks, out, scale=0.1,
                                 row_seq=torch.zeros(rows, dtype=torch.int32, device="cuda"))
        return
    new = torch.zeros(rows, 1, D, dtype=torch.bfloat16, device="cuda")
    ibp.ibp_tree_attention(kp.pages, vp.pages, q, kt, vt, lens, torch.tensor([0, rows], dtype=torch.int32, device="cuda"),
                           new, new, torch.zeros(rows, 1, dtype=torch.int64, device="cuda"), out, scale=0.1, max_new=rows)


def pools():
    return Pool(values(9, T, D, torch.bfloat16, 1)), Pool(values(9, T, D, torch.bfloat16, 2))


def break_record(p):
    """One record's participation bits cleared: as long as its page and longer,
    which no record is."""
    i = int(np.flatnonzero(p.compressed())[0])
    p.slots[i] = 0


@pytest.mark.parametrize("rows,sparse", [(1, False), (40, False), (2, True)])
def test_corrupt_records(rows, sparse):
    kp, vp = pools()
    run(kp, vp, rows, sparse=sparse)
    assert (kp.check(), vp.check()) == (ibp.IBP_OK, ibp.IBP_OK)
    break_record(vp)
    run(kp, vp, rows, sparse=sparse)
    assert (vp.check(), kp.check()) == (ibp.IBP_ERR_CORRUPT, ibp.IBP_ERR_CORRUPT)
    assert (vp.check(), kp.check()) == (ibp.IBP_OK, ibp.IBP_OK)
    kp, vp = pools()
    break_record(kp)
    run(kp, vp, rows, sparse=sparse)
    assert (vp.check(), kp.check()) == (ibp.IBP_OK, ibp.IBP_ERR_CORRUPT)


@pytest.mark.parametrize("rows,sparse", [(1, False), (40, False), (2, True)])
def test_ids_out_of_range(rows, sparse):
    kp, vp = pools()
    t = torch.arange(9, device="cuda").reshape(1, 1, 9).contiguous()
    t[0, 0, 4] = 9
    run(kp, vp, rows, vt=t, sparse=sparse)
    assert (vp.check(), kp.check()) == (ibp.IBP_ERR_RANGE, ibp.IBP_ERR_RANGE)
    run(kp, vp, rows, kt=t, sparse=sparse)
    assert (vp.check(), kp.check()) == (ibp.IBP_OK, ibp.IBP_ERR_RANGE)
