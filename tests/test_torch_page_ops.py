"""torch.ops.ibp.* over pages: schemas and fake kernels on the CPU, and the run of
them together against the binding on the GPU."""
from __future__ import annotations

import numpy as np
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from lossless_tensor_compression_ibp_amd import torch_ops


def test_page_ops_are_registered_with_their_schemas():
    for name, mutated in (("pages_copy", {"dst_slots", "dst_bitmask"}), ("page_bounds", {"bounds"}),
                          ("select_pages", set()), ("sparse_attention", set()), ("tree_attention", set())):
        schema = getattr(torch.ops.ibp, name).default._schema
        got = {a.name for a in schema.arguments if a.alias_info is not None and a.alias_info.is_write}
        assert got == mutated, schema


def test_fake_page_ops_give_the_output_shapes():
    with FakeTensorMode(allow_non_fake_inputs=False):
        def t(*shape, dtype=torch.int64):
            return torch.empty(shape, dtype=dtype, device="cuda")
        slots, bm = t(64, 4096, dtype=torch.uint8), t(2, dtype=torch.int32)
        q, table = t(6, 16, 128, dtype=torch.bfloat16), t(3, 4, 9)
        new = t(6, 4, 128, dtype=torch.bfloat16)
        i32 = t(6, dtype=torch.int32)
        blocks = torch.ops.ibp.select_pages(1, q, t(64, 2, 128, dtype=torch.bfloat16), table, i32, 5, 16, row_seq=i32)
        out, lse = torch.ops.ibp.sparse_attention(1, slots, bm, 1, slots, bm, q, table, table, i32, blocks, 0.1,
                                                  row_seq=i32)
        o2, l2 = torch.ops.ibp.tree_attention(1, slots, bm, 1, slots, bm, q, table, table, i32, i32, new, new, t(6, 1),
                                              0.1, 2)
    assert tuple(blocks.shape) == (6, 4, 5) and blocks.dtype == torch.int32
    for o, l in ((out, lse), (o2, l2)):
        assert tuple(o.shape) == (6, 16, 128) and o.dtype == torch.bfloat16
        assert tuple(l.shape) == (6, 16) and l.dtype == torch.float32


@pytest.mark.gpu
def test_page_ops_match_the_binding_on_the_gpu():
    """Pages moved to another pool, bounded, selected and attended to through
    the operators: every result equal to the binding's, bit for bit."""
    from lossless_tensor_compression_ibp_amd import ibp
    from tests.kv_util import Pool, pages_needed, table, values

    lens, heads, page, dim, group = [200, 77, 16], 2, 16, 128, 4
    n = pages_needed(lens, heads, page) + 3
    k = Pool(values(n, page, dim, torch.bfloat16, 1))
    v = Pool(values(n, page, dim, torch.bfloat16, 2))
    kt, vt = table(lens, heads, page, n, 3), table(lens, heads, page, n, 4)
    kk, vk = torch_ops.register(k.meta), torch_ops.register(v.meta)
    g = torch.Generator(device="cuda").manual_seed(5)
    q = torch.randn(3, heads * group, dim, device="cuda", generator=g).bfloat16()
    len_t = torch.tensor(lens, dtype=torch.int32, device="cuda")

    # pages of keys to another pool, in another order
    order = torch.from_numpy(np.random.default_rng(6).permutation(n)).cuda()
    slots2, bm2 = torch.zeros_like(k.slots), torch.zeros_like(k.bitmask)
    ids = torch.arange(n, device="cuda")
    torch.ops.ibp.pages_copy(kk, k.slots, k.bitmask, ids, slots2, bm2, order)
    kt2 = torch.where(kt >= 0, order[kt.clamp(min=0)], kt)
    assert torch.equal(torch.ops.ibp.gather_decompress(kk, slots2, bm2, order),
                       torch.ops.ibp.gather_decompress(kk, k.slots, k.bitmask, ids))

    bounds = torch.zeros(n, 2, dim, dtype=torch.bfloat16, device="cuda")
    bounds2 = torch.zeros_like(bounds)
    torch.ops.ibp.page_bounds(kk, slots2, bm2, order, None, bounds2)
    ibp.ibp_page_bounds(k.pages, ids, None, bounds)
    assert torch.equal(bounds2[order], bounds)

    blocks = torch.ops.ibp.select_pages(kk, q, bounds2, kt2, len_t, 4, page, 1, 1)
    want = torch.empty_like(blocks)
    ibp.ibp_select_pages(q, bounds, kt, len_t, want, meta=k.meta, page_tokens=page, keep_first=1, keep_last=1)
    assert torch.equal(blocks, want)

    out, lse = torch.ops.ibp.sparse_attention(kk, slots2, bm2, vk, v.slots, v.bitmask, q, kt2, vt, len_t, blocks,
                                              dim ** -0.5)
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    ibp.ibp_sparse_attention(k.pages, v.pages, q, kt, vt, len_t, want, o2, l2, scale=dim ** -0.5)
    assert torch.equal(out, o2) and torch.equal(lse, l2)

    new = torch.randn(3, heads, dim, device="cuda", generator=g).bfloat16()
    rows = torch.tensor([0, 1, 1, 2], dtype=torch.int32, device="cuda")  # row 2 belongs to no sequence
    mask = torch.ones(3, 1, dtype=torch.int64, device="cuda")
    tree = (kk, slots2, bm2, vk, v.slots, v.bitmask, q, kt2, vt, len_t, rows, new, new, mask, dim ** -0.5, 1)
    out, lse = torch.ops.ibp.tree_attention(*tree)
    o2, l2 = torch.zeros_like(out), torch.full_like(lse, -torch.inf)
    ibp.ibp_tree_attention(k.pages, v.pages, q, kt, vt, len_t, rows, new, new, mask, o2, l2, scale=dim ** -0.5,
                           max_new=1)
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    assert not out[2].any() and bool((lse[2] == -torch.inf).all())
    torch_ops.check(kk)
    torch_ops.check(vk)
    for op, args in ((torch.ops.ibp.tree_attention, tree),
                     (torch.ops.ibp.select_pages, (kk, q, bounds2, kt2, len_t, 4, page, 1, 1)),
                     (torch.ops.ibp.page_bounds, (kk, slots2, bm2, order, None, bounds2))):
        torch.library.opcheck(op.default, args, test_utils=("test_schema", "test_faketensor"))
    torch_ops.release(kk)
    torch_ops.release(vk)
