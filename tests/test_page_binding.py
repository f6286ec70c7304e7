"""The page operators' refusals that need no GPU: the binding's checks of
types, shapes and sizes, and the C entries' checks of handles."""
from __future__ import annotations

import pytest
import torch

from lossless_tensor_compression_ibp_amd import ibp

T, D = 16, 128
L = T * D * 2


def _meta(tensor_bytes=L):
    return ibp.Meta(None, tensor_bytes, 32)


def _slots(n, nbytes=L):
    return torch.zeros(n * nbytes, dtype=torch.uint8)


def _bm(n):
    return torch.zeros((n + 31) // 32, dtype=torch.int32)


def test_pool_of_pages():
    with pytest.raises(ValueError, match="slots"):
        ibp.Pages(_meta(), _slots(9), 10, _bm(10))
    with pytest.raises(ValueError, match="bitmask"):
        ibp.Pages(_meta(), _slots(40), 40, _bm(32))
    with pytest.raises(ValueError, match="closed"):
        ibp.Pages(_meta(), _slots(4), 4, _bm(4))._as_parameter_


def _attention(**kw):
    rows, heads, kv, seqs, blocks = 3, 4, 2, 2, 5
    p = ibp.Pages(_meta(), _slots(8), 8, _bm(8))
    a = dict(k=p, v=p, q=torch.zeros(rows, heads, D, dtype=torch.bfloat16),
             k_table=torch.zeros(seqs, kv, blocks, dtype=torch.int64),
             v_table=torch.zeros(seqs, kv, blocks, dtype=torch.int64), lens=torch.zeros(seqs, dtype=torch.int32),
             new_rows=torch.zeros(seqs + 1, dtype=torch.int32), k_new=torch.zeros(rows, kv, D, dtype=torch.bfloat16),
             v_new=torch.zeros(rows, kv, D, dtype=torch.bfloat16), mask=torch.zeros(rows, 1, dtype=torch.int64),
             out=torch.zeros(rows, heads, D, dtype=torch.bfloat16), lse=torch.zeros(rows, heads))
    a.update(kw)
    return a


@pytest.mark.parametrize("kw", [
    dict(q=torch.zeros(3, 4, D)), dict(q=torch.zeros(3, D, 4, dtype=torch.bfloat16).transpose(1, 2)),
    dict(k_table=torch.zeros(2, 2, 5, dtype=torch.int32)), dict(k_table=torch.zeros(2, 10, dtype=torch.int64)),
    dict(v_table=torch.zeros(2, 2, 4, dtype=torch.int64)), dict(lens=torch.zeros(1, dtype=torch.int32)),
    dict(lens=torch.zeros(2, dtype=torch.int64)), dict(new_rows=torch.zeros(2, dtype=torch.int32)),
    dict(k_new=torch.zeros(3, 2, D, dtype=torch.float16)), dict(k_new=torch.zeros(3, 4, D, dtype=torch.bfloat16)),
    dict(v_new=torch.zeros(3, 4, D, dtype=torch.bfloat16)[:, ::2]), dict(mask=torch.zeros(3, dtype=torch.int64)),
    dict(mask=torch.zeros(2, 1, dtype=torch.int64)), dict(mask=torch.zeros(3, 1, dtype=torch.int32)),
    dict(out=torch.zeros(3, 4, D)), dict(out=torch.zeros(2, 4, D, dtype=torch.bfloat16)), dict(lse=torch.zeros(3, 3)),
])
def test_tree_attention_refuses(kw):
    with pytest.raises(ValueError):
        ibp.ibp_tree_attention(*_attention(**kw).values(), scale=1.0, max_new=1)


@pytest.mark.parametrize("kw", [
    dict(blocks=torch.zeros(3, 2, 4, dtype=torch.int64)), dict(blocks=torch.zeros(3, 4, dtype=torch.int32)),
    dict(blocks=torch.zeros(2, 2, 4, dtype=torch.int32)), dict(lens=torch.zeros(2, dtype=torch.int32)),
    dict(row_seq=torch.zeros(2, dtype=torch.int32)), dict(row_seq=torch.zeros(3, dtype=torch.int64)),
    dict(row_seq=None),
])
def test_sparse_attention_and_selection_refuse(kw):
    a = _attention()
    args = dict(lens=torch.zeros(3, dtype=torch.int32), blocks=torch.zeros(3, 2, 4, dtype=torch.int32),
                row_seq=torch.zeros(3, dtype=torch.int32))
    args.update(kw)
    with pytest.raises(ValueError):
        ibp.ibp_sparse_attention(a["k"], a["v"], a["q"], a["k_table"], a["v_table"], args["lens"], args["blocks"],
                                 a["out"], scale=1.0, row_seq=args["row_seq"])
    with pytest.raises(ValueError):
        ibp.ibp_select_pages(a["q"], torch.zeros(8, 2, D, dtype=torch.bfloat16), a["k_table"], args["lens"],
                             args["blocks"], meta=_meta(), page_tokens=T, row_seq=args["row_seq"])


def test_bounds_refuse():
    p = ibp.Pages(_meta(), _slots(8), 8, _bm(8))
    ids = torch.zeros(4, dtype=torch.int64)
    for b in (torch.zeros(8, 2, D), torch.zeros(7, 2, D, dtype=torch.bfloat16), torch.zeros(8, 3, D, dtype=torch.bfloat16)):
        with pytest.raises(ValueError, match="bounds"):
            ibp.ibp_page_bounds(p, ids, None, b)
    b = torch.zeros(8, 2, D, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="ids"):
        ibp.ibp_page_bounds(p, ids.int(), None, b)
    with pytest.raises(ValueError, match="tokens"):
        ibp.ibp_page_bounds(p, ids, torch.zeros(3, dtype=torch.int32), b)


def test_page_moves_refuse():
    m, s, bm, ids = _meta(), _slots(8), _bm(8), torch.zeros(4, dtype=torch.int64)
    refs, table = torch.zeros(8, dtype=torch.int32), torch.zeros(2, 2, 3, dtype=torch.int64)
    lens = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="dst_ids"):
        ibp.ibp_pages_copy(m, s, 8, bm, ids, s, 8, bm, ids[:3])
    with pytest.raises(ValueError, match="src_ids"):
        ibp.ibp_pages_copy(m, s, 8, bm, ids.int(), s, 8, bm, ids)
    with pytest.raises(ValueError, match="dst_slots"):
        ibp.ibp_pages_copy(m, s, 8, bm, ids, s, 9, bm, ids)
    with pytest.raises(ValueError, match="refs"):
        ibp.ibp_pages_alloc(m, refs, 9, ids)
    with pytest.raises(ValueError, match="children"):
        ibp.ibp_pages_fork(m, s, 8, bm, refs, table, lens, ids, ids[:3], page_tokens=T)
    with pytest.raises(ValueError, match="lens"):
        ibp.ibp_pages_fork(m, s, 8, bm, refs, table, lens[:1], ids, ids, page_tokens=T)
    with pytest.raises(ValueError, match="table"):
        ibp.ibp_pages_free(m, refs, 8, table.int(), ids)
    with pytest.raises(ValueError, match="map"):
        ibp.ibp_pages_compact(m, s, 8, bm, refs, ids, ids)
    with pytest.raises(ValueError, match="n_live"):
        ibp.ibp_pages_compact(m, s, 8, bm, refs, torch.zeros(8, dtype=torch.int64), refs)
    with pytest.raises(ValueError, match="workspace"):
        ibp.ibp_pages_alloc(m, refs, 8, ids, workspace=torch.zeros(4, dtype=torch.uint8))


def test_c_entries_refuse_null_handles():
    f = ibp.lib()
    bad = ibp.IBP_ERR_INVALID_ARG
    assert f.ibp_pages_copy(None, None, 0, None, None, None, 0, None, None, 1, None) == bad
    assert f.ibp_pages_alloc(None, None, 1, None, 1, None, 0, None) == bad
    assert f.ibp_pages_fork(None, None, 1, None, None, None, 1, 1, 1, None, 16, None, None, 1, None, 0, None) == bad
    assert f.ibp_pages_free(None, None, 1, None, 1, 1, 1, None, 1, None) == bad
    assert f.ibp_pages_compact(None, None, 1, None, None, None, None, None, 0, None, 0, None) == bad
    assert f.ibp_page_bounds(None, 0, 128, None, None, 1, None, None) == bad
    assert f.ibp_select_pages(None, None, None, None, 1, None, None, None, 0, 0, None, 1, None, 0, None) == bad
    assert f.ibp_tree_attention(None, None, None, *[None] * 8, 1, None, None, None, 0, None) == bad
    assert f.ibp_sparse_attention(None, None, None, *[None] * 6, 1, None, None, None, 0, None) == bad
    a = ibp.ibp_attention()
    assert f.ibp_tree_attention_workspace(None) == 0 and f.ibp_sparse_attention_workspace(None, 1) == 0
    assert f.ibp_tree_attention_workspace(a) == 0 and f.ibp_select_pages_workspace(None) == 0


def test_workspaces_grow_with_the_split():
    a = ibp.ibp_attention(dtype=0, head_dim=128, page_tokens=16, n_q_heads=8, n_kv_heads=2, n_rows=3, n_seqs=1,
                          table_blocks=4096, max_len=65536, max_new=1)
    f = ibp.lib()
    assert f.ibp_tree_attention_workspace(a) > 0
    a.max_len = 40
    assert f.ibp_tree_attention_workspace(a) == 0  # one part: nothing to join
    assert f.ibp_sparse_attention_workspace(a, 2) == 0
    assert f.ibp_select_pages_workspace(a) >= 4 * 3 * 2 * 4096
    assert ibp.ibp_pages_workspace(100, 500) >= 8 * 500
