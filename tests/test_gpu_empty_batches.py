"""Calls without rows: an empty batch is done, whatever its tables hold."""
from __future__ import annotations

import pytest
import torch

from lossless_tensor_compression_ibp_amd import ibp
from tests.kv_util import Pool, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seqs,width", [(0, 4), (0, 0), (2, 0), (2, 4)])
def test_no_rows(seqs, width):
    D = 64
    p = Pool(values(9, 16, D, torch.bfloat16, 1))
    q, new = torch.empty(0, 4, D, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 2, D, dtype=torch.bfloat16, device="cuda")
    t = torch.zeros(seqs, 2, width, dtype=torch.int64, device="cuda")
    lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    ibp.ibp_tree_attention(p.pages, p.pages, q, t, t, lens, torch.zeros(seqs + 1, dtype=torch.int32, device="cuda"), new,
                           new, torch.empty(0, 1, dtype=torch.int64, device="cuda"), q, scale=1.0, max_new=1)
    blocks = torch.empty(0, 2, 3, dtype=torch.int32, device="cuda")
    ibp.ibp_sparse_attention(p.pages, p.pages, q, t, t, none, blocks, q, scale=1.0, row_seq=none)
    bounds = torch.zeros(9, 2, D, dtype=torch.bfloat16, device="cuda")
    ibp.ibp_select_pages(q, bounds, t, none, blocks, meta=p.meta, page_tokens=16, row_seq=none)
    assert p.check() == ibp.IBP_OK


def test_rows_without_sequences_or_blocks_are_refused():
    D = 64
    p = Pool(values(9, 16, D, torch.bfloat16, 1))
    q = torch.zeros(1, 4, D, dtype=torch.bfloat16, device="cuda")
    i32 = torch.zeros(1, dtype=torch.int32, device="cuda")
    blocks = torch.zeros(1, 2, 3, dtype=torch.int32, device="cuda")
    for seqs, width in ((0, 4), (1, 0)):
        t = torch.zeros(seqs, 2, width, dtype=torch.int64, device="cuda")
        with pytest.raises(ibp.IBPError) as e:
            ibp.ibp_sparse_attention(p.pages, p.pages, q, t, t, i32, blocks, torch.empty_like(q), scale=1.0, row_seq=i32)
        assert e.value.status == ibp.IBP_ERR_INVALID_ARG
