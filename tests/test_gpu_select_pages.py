"""ibp_page_bounds, ibp_select_pages and ibp_sparse_attention against their
definitions, and the operators run together as a cache uses them."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from lossless_tensor_compression_ibp_amd import ibp
from tests.kv_util import DT, Pool, assert_close, attend64, context, pages_needed, table, values

pytestmark = pytest.mark.gpu


# --- bounds --------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dim,page", [(64, 16), (64, 32), (64, 64), (128, 16), (128, 32), (256, 16), (256, 4)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("fmt", [None, (32, None), (32, "page"), (128, "page")])
def test_bounds(dim, page, dtype, fmt):
    x = values(300, page, dim, DT[dtype], dim + page)
    if fmt and fmt[1] == "page":
        fmt = (fmt[0], page * dim * 16)
    p = Pool(x, fmt)
    ids = torch.randperm(300, device="cuda")[:201].contiguous()
    ids[7] = -1
    tokens = (torch.arange(201, device="cuda", dtype=torch.int32) % (page + 1)).contiguous()
    b = torch.full((300, 2, dim), 7.0, dtype=x.dtype, device="cuda")
    want = b.clone()
    ibp.ibp_page_bounds(p.pages, ids, tokens, b)
    assert p.check() == ibp.IBP_OK
    for i, n in zip(ids.tolist(), tokens.tolist()):
        if i >= 0 and n:
            want[i, 0], want[i, 1] = x[i, :n].amin(0), x[i, :n].amax(0)
    assert torch.equal(b, want)
    ibp.ibp_page_bounds(p.pages, torch.arange(300, device="cuda"), None, b)
    assert torch.equal(b[:, 0], x.amin(1)) and torch.equal(b[:, 1], x.amax(1))


def test_bounds_pass_on_nan_and_infinity():
    x = values(4, 16, 128, torch.bfloat16, 1)
    x[0, 3, 5], x[1, 15, 0], x[2, 0, 127], x[2, 9, 127] = math.nan, math.inf, -math.inf, math.nan
    p = Pool(x, None)
    b = torch.zeros(4, 2, 128, dtype=x.dtype, device="cuda")
    ibp.ibp_page_bounds(p.pages, torch.arange(4, device="cuda"), None, b)
    want = torch.stack([x.amin(1), x.amax(1)], 1)
    assert torch.equal(torch.isnan(b), torch.isnan(want))
    ok = ~torch.isnan(want)
    assert torch.equal(b[ok], want[ok])


@pytest.mark.parametrize("runs", [3, 4, 5, 7, 8])
def test_bounds_with_large_tables(runs):
    """Tables of 1,024 words from just below to just above what a launch's LDS
    holds."""
    page, dim, n = 32, 128, 200
    L = page * dim * 2
    bits = np.uint32(sum(1 << b for b in (1, 5, 9, 13, 17, 21, 25)[:runs - 1]))
    mask = np.full(L // 4 // 2, bits, np.uint32)
    mask[77] = 0
    x = values(n, page, dim, torch.bfloat16, runs)
    words = x.view(torch.int32).reshape(n, -1)
    keep = torch.from_numpy((~np.tile(mask, 2)).view(np.int32)).cuda()
    words[::2] &= keep
    p = Pool(x, None)
    p.meta = ibp.ibp_meta_create(L, 32, 4 * L, mask, np.zeros_like(mask))
    assert ibp.ibp_meta_get_info(p.meta)["max_runs"] == runs
    ibp.ibp_compress(p.meta, x.view(torch.uint8).reshape(n, L), n, p.slots, p.bitmask)
    p.pages = ibp.Pages(p.meta, p.slots, n, p.bitmask)
    assert p.compressed().any()
    b = torch.zeros(n, 2, dim, dtype=x.dtype, device="cuda")
    ibp.ibp_page_bounds(p.pages, torch.arange(n, device="cuda"), None, b)
    assert p.check() == ibp.IBP_OK
    assert torch.equal(b[:, 0], x.amin(1)) and torch.equal(b[:, 1], x.amax(1))


def test_bounds_errors():
    p = Pool(values(8, 16, 64, torch.bfloat16, 1))
    b = torch.zeros(8, 2, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (8, -2, 1 << 40):
        ibp.ibp_page_bounds(p.pages, torch.tensor([bad, 1], device="cuda"), None, b)
        assert p.check() == ibp.IBP_ERR_RANGE
    with pytest.raises(ibp.IBPError) as e:
        ibp.ibp_page_bounds(p.pages, torch.arange(8, device="cuda"), None,
                            torch.zeros(8, 2, 96, dtype=torch.bfloat16, device="cuda"))
    assert e.value.status == ibp.IBP_ERR_UNSUPPORTED


# --- selection -----------------------------------------------------------------------------------------------
def chosen(q, bounds, ids, n, top, first, last):
    """Blocks of one (row, head): q (heads, dim); 64-bit sums rounded to 32."""
    if n <= top:
        return list(range(n)) + [-1] * (top - n)
    b = bounds[torch.as_tensor(ids[:n], device="cuda")].double()
    qd = q.double()
    s = (qd.clamp(min=0)[:, None] * b[None, :, 1] + qd.clamp(max=0)[:, None] * b[None, :, 0]).sum(-1).float()
    s = torch.where(torch.isnan(s), torch.full_like(s, -math.inf), s).amax(0).cpu().numpy()
    forced = np.zeros(n, bool)
    forced[:first] = True
    if last:
        forced[-last:] = True
    order = np.lexsort((np.arange(n), -s, ~forced))[:top]
    return sorted(order.tolist())


def select_case(lens, seqs, heads, kv_heads, dim, page, top, first, last, dtype="bf16", seed=0, row_seq=None,
                make=None, q=None, width=None):
    dt = DT[dtype]
    need = pages_needed(seqs, kv_heads, page) + 3
    bounds = torch.randn(need, 2, dim, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)).to(dt)
    bounds = bounds.sort(1)[0].contiguous()
    if make:
        bounds = make(bounds)
    t = table(seqs, kv_heads, page, need, seed, width)
    rows = len(lens)
    if q is None:
        q = torch.randn(rows, heads, dim, device="cuda", generator=torch.Generator("cuda").manual_seed(seed + 1)).to(dt)
    meta = Pool(values(2, page, dim, dt, 0)).meta
    blocks = torch.full((rows, kv_heads, top), -7, dtype=torch.int32, device="cuda")
    rs = None if row_seq is None else torch.tensor(row_seq, dtype=torch.int32, device="cuda")
    ibp.ibp_select_pages(q, bounds, t, torch.tensor(lens, dtype=torch.int32, device="cuda"), blocks, meta=meta,
                         page_tokens=page, keep_first=first, keep_last=last, row_seq=rs)
    assert ibp.ibp_check(meta) == ibp.IBP_OK
    G = heads // kv_heads
    got, tn = blocks.cpu().numpy(), t.cpu().numpy()
    for r in range(rows):
        for h in range(kv_heads):
            s = r if row_seq is None else row_seq[r]
            want = chosen(q[r, h * G:(h + 1) * G], bounds, tn[s, h], -(-lens[r] // page), top, first, last)
            assert got[r, h].tolist() == want, (r, h)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_select(dim, dtype):
    page = 16
    lens = [1, 16, 17, 500, 1000, 3001, 0]
    select_case(lens, lens, 8, 2, dim, page, 12, 1, 2, dtype, seed=dim)


@pytest.mark.parametrize("group", [1, 3, 5, 7, 8, 9, 16, 17, 40])
def test_select_groups(group):
    select_case([900, 64, 700], [900, 64, 700], 2 * group, 2, 64, 16, 7, 0, 1, seed=group)


@pytest.mark.parametrize("top,first,last", [(1, 0, 0), (1, 1, 0), (2, 1, 1), (5, 0, 5), (30, 3, 4), (64, 0, 0),
                                            (300, 1, 1)])
def test_select_counts(top, first, last):
    select_case([1600, 977, 33], [1600, 977, 33], 4, 2, 64, 16, top, first, last, seed=top)


def test_select_rows_of_several_sequences():
    """Rows of one tile that belong to different sequences, in any order."""
    seqs = [400, 1300, 90]
    row_seq = [1, 1, 0, 2, 1, 0, 1, 1, 2, 0, 1]
    lens = [1300, 1299, 400, 90, 700, 17, 1, 1300, 50, 399, 1030]
    select_case(lens, seqs, 4, 2, 128, 16, 9, 1, 2, seed=5, row_seq=row_seq)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 2, 4, 7, 16])
@pytest.mark.parametrize("mixed", [False, True])
def test_select_many_rows_of_a_sequence(dim, group, mixed):
    """Rows that share their pages' bounds: blocks of rows of one sequence, and
    rows of two in any order, with lengths from nothing to all of it."""
    seqs = [3300, 1500]
    rng = np.random.default_rng(dim + group)
    row_seq = rng.integers(0, 2, 37).tolist() if mixed else [0] * 24 + [1] * 13
    lens = [int(rng.integers(0, seqs[s] + 1)) for s in row_seq]
    lens[0], lens[5], lens[36] = seqs[row_seq[0]], 0, 1
    select_case(lens, seqs, 2 * group, 2, dim, 16, 11, 1, 2, seed=dim, row_seq=row_seq)


def test_select_ties_go_to_the_lower_block():
    def same(b):
        return b[:1].expand_as(b).contiguous()

    def coarse(b):
        return b.float().round().clamp(-1, 1).to(b.dtype).contiguous()

    lens = [2000, 1999]
    select_case(lens, lens, 4, 2, 64, 16, 20, 1, 2, make=same, seed=1)
    q = torch.randint(-1, 2, (2, 4, 64), device="cuda").to(torch.bfloat16)
    select_case(lens, lens, 4, 2, 64, 16, 20, 1, 2, make=coarse, q=q, seed=2)
    select_case(lens, lens, 4, 2, 64, 16, 20, 0, 0, q=torch.zeros(2, 4, 64, device="cuda", dtype=torch.bfloat16))


def test_select_near_scores_are_summed_in_64_bits():
    """Scores that 32-bit sums cannot tell apart: large terms that cancel."""
    def close(b):
        b = b.clone()
        b[:, :, 0], b[:, :, 1] = 1024.0, -1024.0
        b[:, :, 2:] *= 2.0 ** -12
        return b.sort(1)[0].contiguous()

    q = torch.ones(2, 4, 128, device="cuda", dtype=torch.bfloat16)
    select_case([4000, 3333], [4000, 3333], 4, 2, 128, 16, 25, 1, 2, make=close, q=q, seed=3)


@pytest.mark.parametrize("rows", [2, 9])
@pytest.mark.parametrize("n", [300, 2000, 9000])
def test_select_sums_that_overflow_32_bits(rows, n):
    """Products of 2e38 that cancel: 32-bit sums are infinite or NaN where those
    of 64 bits are not; and scores that are infinite in both."""
    def large(b):
        b = b * 1e17
        b[:, :, 0], b[:, :, 1], b[:, :, 2], b[:, :, 3] = 2e19, 1.5e19, -2e19, -1.5e19
        b[::len(b) // 12, 1, 9] = 3e38  # times q: more than 32 bits hold
        return b

    q = torch.ones(rows, 2, 64, device="cuda", dtype=torch.bfloat16) * 1e19
    q[:, 1] *= 0.5
    select_case([16 * n - 1] * rows, [16 * n] * 2, 2, 1, 64, 16, 40, 1, 2, make=large, q=q, seed=n,
                row_seq=[i % 2 for i in range(rows)])


@pytest.mark.parametrize("bad", [math.inf, -math.inf])
def test_select_infinite_bounds(bad):
    def some(b):
        b = b.clone()
        b[::3, :, 3] = bad
        return b

    select_case([1600, 900], [1600, 900], 4, 1, 64, 16, 60, 0, 1, make=some, seed=8)


def test_select_nan_ranks_last():
    def some(b):
        b = b.clone()
        b[::5, 0, 3] = math.nan
        b[::5, 1, 3] = math.nan
        return b

    select_case([1600], [1600], 4, 1, 64, 16, 30, 0, 1, make=some, seed=4)


def test_select_long_row():
    n = 60001
    select_case([n * 16 - 3], [n * 16], 2, 1, 64, 16, 200, 1, 2, seed=6)


def test_select_errors_and_refusals():
    meta = Pool(values(2, 16, 64, torch.bfloat16, 0)).meta
    q = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    b = torch.zeros(50, 2, 64, dtype=torch.bfloat16, device="cuda")
    t = torch.arange(40, device="cuda").reshape(2, 1, 20).contiguous()
    out = torch.full((2, 1, 4), -7, dtype=torch.int32, device="cuda")

    def call(lens, table=t, row_seq=None, **kw):
        ibp.ibp_select_pages(q, b, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), out, meta=meta,
                             page_tokens=kw.pop("page_tokens", 16), row_seq=row_seq, **kw)
        return ibp.ibp_check(meta)

    assert call([320, 100]) == ibp.IBP_OK
    assert call([321, 100]) == ibp.IBP_ERR_RANGE  # more than the table holds
    assert call([-1, 100]) == ibp.IBP_ERR_RANGE
    assert call([320, 100], row_seq=torch.tensor([0, 2], dtype=torch.int32, device="cuda")) == ibp.IBP_ERR_RANGE
    wrong = t.clone()
    wrong[0, 0, 3] = 50
    assert call([320, 100], wrong) == ibp.IBP_ERR_RANGE
    for kw in (dict(keep_first=3, keep_last=2), dict(page_tokens=12)):
        with pytest.raises(ibp.IBPError):
            call([320, 100], **kw)
    with pytest.raises(ValueError):
        ibp.ibp_select_pages(q, b[:, :, :32], t, torch.zeros(2, dtype=torch.int32, device="cuda"), out, meta=meta,
                             page_tokens=16)


# --- sparse attention ----------------------------------------------------------------------------------------
class Sparse:
    def __init__(self, lens, heads, kv_heads, dim, page, lists, dtype="bf16", fmt=(32, None), seed=0, seqs=None,
                 row_seq=None, pinned=False):
        dt = DT[dtype]
        self.seqs = seqs or lens
        n = pages_needed(self.seqs, kv_heads, page) + 2
        self.k = Pool(values(n, page, dim, dt, seed + 1), fmt, pinned)
        self.v = Pool(values(n, page, dim, dt, seed + 2), fmt, pinned)
        self.kt, self.vt = table(self.seqs, kv_heads, page, n, seed), table(self.seqs, kv_heads, page, n, seed + 9)
        self.lens, self.page, self.row_seq = lens, page, row_seq
        g = torch.Generator("cuda").manual_seed(seed)
        self.q = torch.randn(len(lens), heads, dim, device="cuda", generator=g).to(dt)
        self.blocks = lists(self)
        self.scale = dim ** -0.5

    def call(self, **kw):
        out = torch.empty_like(self.q)
        lse = torch.empty(self.q.shape[:2], dtype=torch.float32, device="cuda")
        rs = None if self.row_seq is None else torch.tensor(self.row_seq, dtype=torch.int32, device="cuda")
        ibp.ibp_sparse_attention(self.k.pages, self.v.pages, self.q, self.kt, self.vt,
                                 torch.tensor(self.lens, dtype=torch.int32, device="cuda"), self.blocks, out, lse,
                                 scale=self.scale, row_seq=rs, **kw)
        return out, lse

    def want(self):
        R, H, D = self.q.shape
        HK = self.kt.shape[1]
        G, T = H // HK, self.page
        shape = (R, H, D)
        out, tol = (torch.zeros(shape, dtype=torch.float64, device="cuda") for _ in range(2))
        lse, ltol = (torch.zeros(shape[:2], dtype=torch.float64, device="cuda") for _ in range(2))
        bl = self.blocks.cpu().numpy()
        for r in range(R):
            s = r if self.row_seq is None else self.row_seq[r]
            for h in range(HK):
                at = [b * T + i for b in bl[r, h] if b >= 0 for i in range(T) if b * T + i < self.lens[r]]
                at = torch.tensor(at, dtype=torch.long, device="cuda")
                full = self.kt.shape[2] * T
                k, v = context(self.k, self.kt[s, h], full)[at], context(self.v, self.vt[s, h], full)[at]
                for i in range(h * G, h * G + G):
                    seen = torch.ones(at.numel(), dtype=torch.bool, device="cuda")
                    out[r, i], lse[r, i], tol[r, i], ltol[r, i] = attend64(self.q[r, i], k, v, seen, self.scale)
        return out, lse, tol, ltol

    def compare(self, label):
        print(f"[sparse] {label}", flush=True)
        out, lse = self.call()
        assert self.k.check() == ibp.IBP_OK
        o, l, tol, ltol = self.want()
        assert_close(out, o, tol, f"{label} out")
        assert_close(lse, l, ltol, f"{label} lse")


def random_lists(top, seed=0):
    def make(c):
        rng = np.random.default_rng(seed)
        HK = c.kt.shape[1]
        out = np.full((len(c.lens), HK, top), -1, np.int32)
        for r, n in enumerate(c.lens):
            nb = -(-n // c.page)
            for h in range(HK):
                k = int(rng.integers(0, min(top, nb) + 1)) if r % 2 else min(top, nb)
                out[r, h, :k] = np.sort(rng.choice(nb, k, replace=False)) if nb else []
        return torch.from_numpy(out).cuda()

    return make


@pytest.mark.parametrize("dim,page", [(64, 16), (64, 32), (64, 64), (128, 16), (128, 32), (256, 16)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_sparse_attention(dim, page, dtype):
    Sparse([1, 900, 0, 333, page], 6, 2, dim, page, random_lists(9), dtype, seed=dim + page).compare(f"{dim}x{page}")


@pytest.mark.parametrize("group", [1, 7, 16, 17, 33])
@pytest.mark.parametrize("fmt", [None, (32, 32768)])
def test_sparse_groups(group, fmt):
    Sparse([700, 64], 2 * group, 2, 128, 16, random_lists(5), fmt=fmt, seed=group).compare(f"group {group} {fmt}")


def test_sparse_lists_in_any_order_with_gaps_and_repeats():
    def lists(c):
        b = torch.full((2, 1, 70), -1, dtype=torch.int32, device="cuda")
        b[0, 0, :8] = torch.tensor([5, -1, 0, 5, 31, -1, 2, 40])  # 31 holds the end, 40 lies behind it
        b[1, 0, 60:] = 3
        return b

    c = Sparse([500, 64], 4, 1, 128, 16, lists, seed=3)
    c.compare("order")


def test_sparse_split_and_rows_of_sequences():
    row_seq = [0, 1, 1, 0, 1]
    lens = [9000, 40, 3000, 8999, 2500]
    Sparse(lens, 4, 1, 128, 16, random_lists(400), seed=4, seqs=[9000, 3000], row_seq=row_seq).compare("split")


def test_sparse_pinned_pool():
    Sparse([900, 100], 4, 2, 128, 16, random_lists(9), seed=5, pinned=True).compare("pinned")


def test_sparse_stale_numbers():
    c = Sparse([19, 33], 4, 2, 128, 16, random_lists(4), fmt=None, seed=6)
    want = c.want()
    for pool, t in ((c.k, c.kt), (c.v, c.vt)):
        x = pool.slots.view(torch.bfloat16).reshape(pool.x.shape)
        for s, n in enumerate(c.lens):
            for h in range(2):
                x[t[s, h, n // 16], n % 16:] = math.nan
    out, lse = c.call()
    assert_close(out, want[0], want[2], "stale out")


def test_sparse_captured():
    c = Sparse([5000, 700], 4, 2, 128, 16, random_lists(100), seed=7)
    s = torch.cuda.Stream()
    want, _ = c.call()
    rs = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:2], dtype=torch.float32, device="cuda")
    bounds = torch.stack([c.k.x.amin(1), c.k.x.amax(1)], 1).contiguous()
    blocks = torch.empty_like(c.blocks)

    def step():
        ibp.ibp_select_pages(c.q, bounds, c.kt, rs, blocks, meta=c.k.meta, page_tokens=16, keep_last=1, stream=s)
        ibp.ibp_sparse_attention(c.k.pages, c.v.pages, c.q, c.kt, c.vt, rs, blocks, out, lse, scale=c.scale, stream=s)

    torch.cuda.synchronize()
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    q0 = c.q.clone()
    for i in range(4):
        c.q.copy_(q0.roll(i, 0))
        torch.cuda.synchronize()
        step()
        torch.cuda.synchronize()
        eager = out.clone(), blocks.clone()
        out.zero_()
        blocks.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager[0]) and torch.equal(blocks, eager[1])


# --- together ------------------------------------------------------------------------------------------------
def test_a_cache_from_prefill_to_sparse_decoding():
    """Pages encoded by the codec, moved to a pinned pool and back, summarised,
    selected and read; forked, freed and compacted in between."""
    HK, G, D, T = 2, 4, 128, 16
    lens = [1000, 333]
    n = 400
    kx, vx = values(n, T, D, torch.bfloat16, 1), values(n, T, D, torch.bfloat16, 2)
    k, v = Pool(kx), Pool(vx)
    assert k.compressed().any()
    used = pages_needed(lens, HK, T)
    t = table(lens, HK, T, used + 20, 3)  # slots are shared by both tables: one id names a page in both pools
    full = torch.full((4, HK, t.shape[2]), -1, dtype=torch.int64, device="cuda")
    full[:2] = t
    refs = torch.zeros(n, dtype=torch.int32, device="cuda")
    refs[full[full >= 0]] = 1
    len_t = torch.tensor(lens + [0, 0], dtype=torch.int32, device="cuda")
    q = torch.randn(4, HK * G, D, device="cuda").to(torch.bfloat16)

    def attend(kp, vp, tab, ln, sparse):
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float32, device="cuda")
        if not sparse:
            new = torch.zeros(4, HK, D, dtype=torch.bfloat16, device="cuda")
            ibp.ibp_tree_attention(kp, vp, q, tab, tab, ln, torch.arange(5, dtype=torch.int32, device="cuda"), new,
                                   new, torch.zeros(4, 1, dtype=torch.int64, device="cuda"), out, lse, scale=0.1,
                                   max_new=1)
            return out, None
        bounds = torch.zeros(n, 2, D, dtype=torch.bfloat16, device="cuda")
        ids = tab[tab >= 0]
        ibp.ibp_page_bounds(kp, ids, None, bounds)
        blocks = torch.empty(4, HK, sparse, dtype=torch.int32, device="cuda")
        ibp.ibp_select_pages(q, bounds, tab, ln, blocks, meta=k.meta, page_tokens=T, keep_last=1)
        ibp.ibp_sparse_attention(kp, vp, q, tab, tab, ln, blocks, out, lse, scale=0.1)
        return out, blocks

    dense, _ = attend(k.pages, v.pages, full, len_t, 0)
    every, blocks = attend(k.pages, v.pages, full, len_t, full.shape[2])
    # all pages selected: the same sums in another order
    assert (dense.float() - every.float()).abs().max() <= 2.0 ** -6 * dense.float().abs().max()
    few, blocks = attend(k.pages, v.pages, full, len_t, 8)
    # the selected pages, gathered by the codec, are the pages that were stored
    picked = full[0, 0, blocks[0, 0].long()].contiguous()
    got = torch.empty(8, k.L, dtype=torch.uint8, device="cuda")
    ibp.ibp_gather_decompress(k.meta, k.slots, n, k.bitmask, picked, got)
    assert torch.equal(got.view(torch.bfloat16).reshape(8, T, D), kx[picked])
    # to pinned memory at the compressed size, read from there
    far = {}
    for name, p in (("k", k), ("v", v)):
        host = torch.zeros(n, p.L, dtype=torch.uint8).pin_memory()
        bm = torch.zeros_like(p.bitmask)
        ids = torch.arange(n, device="cuda")
        ibp.ibp_pages_copy(p.meta, p.slots, n, p.bitmask, ids, host, n, bm, ids)
        torch.cuda.synchronize()
        far[name] = ibp.Pages(p.meta, host, n, bm)
    away, _ = attend(far["k"], far["v"], full, len_t, 8)
    assert torch.equal(away, few)
    # forks share pages and read the same; the copied tail is the child's own.
    # Both pools hand out the same slots, so one table serves both.
    parents, children = torch.tensor([0, 1], device="cuda"), torch.tensor([3, 2], device="cuda")
    refs_v, table_v = refs.clone(), full.clone()
    for p, rc, tb in ((k, refs, full), (v, refs_v, table_v)):
        ibp.ibp_pages_fork(p.meta, p.slots, n, p.bitmask, rc, tb, len_t, parents, children, page_tokens=T)
    assert torch.equal(full, table_v) and torch.equal(refs, refs_v)
    len_t[children] = len_t[parents]
    q[children] = q[parents]
    forked, _ = attend(k.pages, v.pages, full, len_t, 8)
    assert torch.equal(forked[children], forked[parents]) and torch.equal(forked[:2], few[:2])
    # parents leave, the pool is compacted, the children read the same
    for p, rc, tb in ((k, refs, full), (v, refs_v, table_v)):
        ibp.ibp_pages_free(p.meta, rc, n, tb, parents)
        m, live = torch.empty(n, dtype=torch.int64, device="cuda"), torch.empty(1, dtype=torch.int64, device="cuda")
        ibp.ibp_pages_compact(p.meta, p.slots, n, p.bitmask, rc, m, live, table=tb)
    assert int(live) == int((refs > 0).sum()) and bool((refs[:int(live)] > 0).all())
    assert int(full.max()) < int(live)
    len_t[parents] = 0
    after, _ = attend(k.pages, v.pages, full, len_t, 8)
    assert torch.equal(after[children], forked[children])
    assert k.check() == ibp.IBP_OK and v.check() == ibp.IBP_OK
