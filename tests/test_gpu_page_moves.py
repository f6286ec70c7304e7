"""ibp_pages_copy, _alloc, _fork, _free and _compact against a plain model of
slots, bits, counts and tables: every byte of the pools is compared."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from lossless_tensor_compression_ibp_amd import ibp

pytestmark = pytest.mark.gpu

FORMATS = [(512, 32, 4096), (1024, 1024, 8192), (1536, 32, 384), (2048, 32, 32), (4096, 32, 32768), (4096, 64, 2048),
           (6144, 32, 1024), (8192, 128, 65536), (8192, 32, 2048)]


class Slots:
    """n slots of an L-byte format, half of them compressible."""

    def __init__(self, n, L, W, M, seed=0, pinned=False):
        rng = np.random.default_rng(seed)
        x = rng.normal(size=(n, L // 4)).astype(np.float32)
        x[::2] = np.abs(x[::2]) * 0.1
        x[rng.random(x.shape) < 0.3] = 0
        raw = torch.from_numpy(x.view(np.uint8).reshape(n, L)).cuda()
        self.n, self.L = n, L
        self.meta = ibp.ibp_build_metadata(raw[::2].contiguous(), (n + 1) // 2, L, W, M, 0.9)
        self.slots = torch.full((n, L), 0xAB, dtype=torch.uint8, device="cuda")
        self.bm = torch.zeros((n + 31) // 32, dtype=torch.int32, device="cuda")
        st = torch.zeros(n, dtype=torch.int64, device="cuda")
        ibp.ibp_compress(self.meta, raw, n, self.slots, self.bm, st)
        torch.cuda.synchronize()
        self.stored = st.cpu().numpy()
        if pinned:
            host = torch.empty((n, L), dtype=torch.uint8, pin_memory=True)
            host.copy_(self.slots)
            self.slots = host

    def bytes(self):
        return self.slots.cpu().numpy().copy()

    def bits(self):
        return np.unpackbits(self.bm.cpu().numpy().view(np.uint8), bitorder="little").copy()

    def check(self):
        return ibp.ibp_check(self.meta)


def ids_of(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int64)).cuda()


@pytest.mark.parametrize("L,W,M", FORMATS)
@pytest.mark.parametrize("where", ["hbm", "to_pinned", "from_pinned"])
def test_copy(L, W, M, where):
    rng = np.random.default_rng(L + W)
    print(f"[copy] {L} {W} {M} {where}", flush=True)
    a = Slots(200, L, W, M, pinned=where == "from_pinned")
    assert (a.stored < L).any()
    dst = torch.full((150, L), 0x5C, dtype=torch.uint8)
    dst = dst.pin_memory() if where == "to_pinned" else dst.cuda()
    dbm = torch.full((5,), -1, dtype=torch.int32, device="cuda")
    src, to = rng.integers(0, 200, 77), rng.permutation(150)[:77]
    src[5], to[9] = -1, -1
    want, bits, sb, ss = dst.cpu().numpy().copy(), np.ones(160, np.uint8), a.bits(), a.bytes()
    for s, d in zip(src, to):
        if s >= 0 and d >= 0:
            want[d, :a.stored[s]] = ss[s, :a.stored[s]]
            bits[d] = sb[s]
    ibp.ibp_pages_copy(a.meta, a.slots, 200, a.bm, ids_of(src), dst, 150, dbm, ids_of(to))
    torch.cuda.synchronize()
    assert a.check() == ibp.IBP_OK
    np.testing.assert_array_equal(dst.cpu().numpy(), want)
    np.testing.assert_array_equal(np.unpackbits(dbm.cpu().numpy().view(np.uint8), bitorder="little"), bits)


def test_copy_short_first_read():
    """The rest of a record is read after its header."""
    a = Slots(64, 4096, 32, 32768)
    ibp.ibp_meta_set_first_read(a.meta, 256)
    dst, bm = torch.zeros_like(a.slots), torch.zeros_like(a.bm)
    ibp.ibp_pages_copy(a.meta, a.slots, 64, a.bm, ids_of(np.arange(64)), dst, 64, bm, ids_of(np.arange(64)))
    d, s = dst.cpu().numpy(), a.bytes()
    for i in range(64):
        k = a.stored[i]
        assert np.array_equal(d[i, :k], s[i, :k]) and not d[i, k:].any()
    assert torch.equal(bm, a.bm)


def test_copy_within_a_pool_and_errors():
    a = Slots(100, 512, 32, 4096)
    before, bits = a.bytes(), a.bits()
    src, to = np.arange(0, 50), np.arange(99, 49, -1)
    for s, d in zip(src, to):
        before[d, :a.stored[s]] = before[s, :a.stored[s]]
        bits[d] = bits[s]
    ibp.ibp_pages_copy(a.meta, a.slots, 100, a.bm, ids_of(src), a.slots, 100, a.bm, ids_of(to))
    np.testing.assert_array_equal(a.bytes(), before)
    np.testing.assert_array_equal(a.bits(), bits)
    for s, d in ((100, 0), (0, 100), (-2, 0), (0, -5), (1 << 40, 0)):
        ibp.ibp_pages_copy(a.meta, a.slots, 100, a.bm, ids_of([s]), a.slots, 100, a.bm, ids_of([d]))
        assert a.check() == ibp.IBP_ERR_RANGE
    np.testing.assert_array_equal(a.bytes(), before)
    # a slot that is marked as a record but holds none: copied whole, latched
    b = Slots(4, 512, 32, 4096)
    b.slots.zero_()
    b.slots[0, 100] = 7
    b.bm.fill_(1)
    out, bm = torch.full_like(b.slots, 9), torch.zeros_like(b.bm)
    ibp.ibp_pages_copy(b.meta, b.slots, 4, b.bm, ids_of([0]), out, 4, bm, ids_of([2]))
    assert b.check() == ibp.IBP_ERR_CORRUPT
    assert torch.equal(out[2], b.slots[0])


def test_copy_refusals():
    a = Slots(10, 512, 32, 4096)
    i = ids_of([0])
    with pytest.raises(ibp.IBPError) as e:  # pageable memory
        ibp.ibp_pages_copy(a.meta, torch.zeros(10, 512, dtype=torch.uint8), 10, a.bm, i, a.slots, 10, a.bm, i)
    assert e.value.status == ibp.IBP_ERR_INVALID_ARG
    with pytest.raises(ibp.IBPError) as e:  # pools that overlap in part
        ibp.ibp_pages_copy(a.meta, a.slots, 9, a.bm, i, a.slots[1:], 9, a.bm, i)
    assert e.value.status == ibp.IBP_ERR_INVALID_ARG
    odd = torch.zeros(10 * 512 + 8, dtype=torch.uint8, device="cuda")[8:]
    with pytest.raises(ibp.IBPError) as e:  # slots not on 16 bytes
        ibp.ibp_pages_copy(a.meta, odd, 10, a.bm, i, a.slots, 10, a.bm, i)
    assert e.value.status == ibp.IBP_ERR_UNSUPPORTED
    big = ibp.ibp_meta_create(16384, 32, 32, np.zeros(1, np.uint32), np.zeros(1, np.uint32))
    s = torch.zeros(4, 16384, dtype=torch.uint8, device="cuda")
    with pytest.raises(ibp.IBPError) as e:
        ibp.ibp_pages_copy(big, s, 4, a.bm, i, s.clone(), 4, a.bm, i)
    assert e.value.status == ibp.IBP_ERR_UNSUPPORTED


@pytest.mark.parametrize("n_slots", [1, 31, 4096, 4097, 50001])
@pytest.mark.parametrize("share", [0.0, 0.3, 1.0])
def test_alloc(n_slots, share):
    meta = Slots(2, 512, 32, 4096).meta
    rng = np.random.default_rng(n_slots)
    refs = (rng.random(n_slots) < share).astype(np.int32) * 3
    free = np.flatnonzero(refs == 0)
    for n in sorted({1, max(1, free.size // 2), max(1, free.size), free.size + 5}):
        r = torch.from_numpy(refs.copy()).cuda()
        ids = torch.full((n,), -9, dtype=torch.int64, device="cuda")
        ibp.ibp_pages_alloc(meta, r, n_slots, ids)
        k = min(n, free.size)
        want = np.concatenate([free[:k], np.full(n - k, -1)])
        np.testing.assert_array_equal(ids.cpu().numpy(), want)
        after = refs.copy()
        after[free[:k]] = 1
        np.testing.assert_array_equal(r.cpu().numpy(), after)
        assert ibp.ibp_check(meta) == (ibp.IBP_OK if n <= free.size else ibp.IBP_ERR_NOMEM)


def fork_model(slots, bits, stored, refs, table, lens, parents, children, T):
    """The definition, pair by pair; slots and bits change in place."""
    free = list(np.flatnonzero(refs == 0))
    at = 0
    new = table.copy()
    for p, c in zip(parents, children):
        full, tail = divmod(int(lens[p]), T)
        for h in range(table.shape[1]):
            row = np.full(table.shape[2], -1, np.int64)
            row[:full] = table[p, h, :full]
            np.add.at(refs, row[:full], 1)
            if tail:
                if at < len(free):
                    o, w = int(table[p, h, full]), int(free[at])
                    slots[w, :stored[o]] = slots[o, :stored[o]]
                    bits[w] = bits[o]
                    refs[w] = 1
                    row[full] = w
                at += 1
            new[c, h] = row
    return new


@pytest.mark.parametrize("room", [1000, 3])
def test_fork_and_free(room):
    T, H, B, L = 16, 3, 9, 2048
    rng = np.random.default_rng(room)
    a = Slots(7 * H * B + room, L, 32, 32)
    n = a.n
    lens = np.array([B * T, 1, 17, 0, 16, B * T - 1, 40, 0, 0, 0, 0, 0, 0], np.int32)
    table = np.full((13, H, B), -1, np.int64)
    order = iter(rng.permutation(7 * H * B))
    refs = np.zeros(n, np.int32)
    for s in range(7):
        for h in range(H):
            for b in range(-(-int(lens[s]) // T)):
                table[s, h, b] = next(order)
                refs[table[s, h, b]] = 1
    if room == 3:  # all but three slots are taken
        refs[refs == 0] = 5
        refs[-3:] = 0
    parents, children = np.array([5, 0, 2, 2, 3, 1]), np.array([12, 7, 9, 8, 10, 11])
    slots, bits, r0 = a.bytes(), a.bits(), refs.copy()
    want = fork_model(slots, bits, a.stored, refs, table, lens, parents, children, T)
    g_refs, g_table = torch.from_numpy(r0).cuda(), torch.from_numpy(table.copy()).cuda()
    ibp.ibp_pages_fork(a.meta, a.slots, n, a.bm, g_refs, g_table, torch.from_numpy(lens).cuda(), ids_of(parents),
                       ids_of(children), page_tokens=T)
    assert a.check() == (ibp.IBP_OK if room == 1000 else ibp.IBP_ERR_NOMEM)
    np.testing.assert_array_equal(g_table.cpu().numpy(), want)
    np.testing.assert_array_equal(g_refs.cpu().numpy(), refs)
    np.testing.assert_array_equal(a.bytes(), slots)
    np.testing.assert_array_equal(a.bits(), bits)
    # freeing: a sequence given twice counts once
    gone = np.array([12, 0, 7, 12])
    ibp.ibp_pages_free(a.meta, g_refs, n, g_table, ids_of(gone))
    for s in sorted(set(gone.tolist())):
        ids = want[s][want[s] >= 0]
        np.subtract.at(refs, ids, 1)
        want[s] = -1
    assert a.check() == ibp.IBP_OK
    np.testing.assert_array_equal(g_refs.cpu().numpy(), refs)
    np.testing.assert_array_equal(g_table.cpu().numpy(), want)


def test_fork_and_free_errors():
    a = Slots(50, 512, 32, 4096)
    refs = torch.ones(50, dtype=torch.int32, device="cuda")
    refs[40:] = 0
    table = torch.arange(24, device="cuda").reshape(4, 2, 3).contiguous()
    lens = torch.tensor([10, 12, 13, -1], dtype=torch.int32, device="cuda")
    keep = table.clone()
    for p, c in ((0, 4), (-1, 1), (2, 1), (3, 1), (1, 1)):  # no such row, more than its row holds, itself
        ibp.ibp_pages_fork(a.meta, a.slots, 50, a.bm, refs, table, lens, ids_of([p]), ids_of([c]), page_tokens=4)
        assert a.check() == ibp.IBP_ERR_RANGE
        assert torch.equal(table, keep)
    refs.zero_()
    ibp.ibp_pages_free(a.meta, refs, 50, table, ids_of([1]))
    assert a.check() == ibp.IBP_ERR_CORRUPT and not refs.any()
    ibp.ibp_pages_free(a.meta, refs, 50, table, ids_of([7]))
    assert a.check() == ibp.IBP_ERR_RANGE


@pytest.mark.parametrize("n_slots,share", [(1, 0.0), (1, 1.0), (33, 0.5), (4096, 0.9), (5000, 0.02), (9001, 0.5),
                                           (300, 1.0), (300, 0.0)])
def test_compact(n_slots, share):
    a = Slots(n_slots, 1024, 1024, 8192)
    rng = np.random.default_rng(n_slots)
    refs = (rng.random(n_slots) < share).astype(np.int32) * rng.integers(1, 4, n_slots).astype(np.int32)
    live = np.flatnonzero(refs)
    table = np.concatenate([rng.permutation(live), [-1, -1]]).astype(np.int64)
    slots, bits = a.bytes(), a.bits()
    m = np.where(refs > 0, np.arange(n_slots), -1)
    holes = [i for i in range(live.size) if refs[i] == 0]
    movers = [i for i in range(n_slots - 1, live.size - 1, -1) if refs[i] > 0]
    want_refs = refs.copy()
    for d, s in zip(holes, movers):
        slots[d, :a.stored[s]] = slots[s, :a.stored[s]]
        bits[d] = bits[s]
        m[s] = d
        want_refs[d], want_refs[s] = refs[s], 0
    assert len(holes) == len(movers)
    g_refs, g_table = torch.from_numpy(refs).cuda(), torch.from_numpy(table).cuda()
    g_map = torch.empty(n_slots, dtype=torch.int64, device="cuda")
    n_live = torch.empty(1, dtype=torch.int64, device="cuda")
    ibp.ibp_pages_compact(a.meta, a.slots, n_slots, a.bm, g_refs, g_map, n_live, table=g_table)
    assert a.check() == ibp.IBP_OK
    assert int(n_live) == live.size
    np.testing.assert_array_equal(g_map.cpu().numpy(), m)
    np.testing.assert_array_equal(g_refs.cpu().numpy(), want_refs)
    np.testing.assert_array_equal(g_table.cpu().numpy(), np.where(table >= 0, m[table], -1))
    np.testing.assert_array_equal(a.bytes(), slots)
    np.testing.assert_array_equal(a.bits(), bits)


def test_captured_fork_free_and_compact():
    """A beam step captured once and replayed, eager steps between."""
    T, H, B = 16, 2, 4
    a = Slots(64, 2048, 32, 32)
    table0 = np.full((4, H, B), -1, np.int64)
    table0[0] = np.arange(40, 40 + H * B).reshape(H, B)
    table0[1, :, :2] = np.arange(20, 24).reshape(H, 2)
    lens = torch.tensor([B * T - 3, 2 * T, 0, 0], dtype=torch.int32, device="cuda")
    refs0 = np.zeros(64, np.int32)
    refs0[table0[table0 >= 0]] = 1
    table, refs = torch.from_numpy(table0).cuda(), torch.from_numpy(refs0).cuda()
    m, live = torch.empty(64, dtype=torch.int64, device="cuda"), torch.empty(1, dtype=torch.int64, device="cuda")
    parents, children = ids_of([0, 1]), ids_of([2, 3])
    start = a.slots.clone(), a.bm.clone()
    s = torch.cuda.Stream()

    def step():
        ibp.ibp_pages_fork(a.meta, a.slots, 64, a.bm, refs, table, lens, parents, children, page_tokens=T, stream=s)
        ibp.ibp_pages_free(a.meta, refs, 64, table, parents[:1], stream=s)
        ibp.ibp_pages_compact(a.meta, a.slots, 64, a.bm, refs, m, live, table=table, stream=s)

    def reset():
        table.copy_(torch.from_numpy(table0))
        refs.copy_(torch.from_numpy(refs0))
        a.slots.copy_(start[0])
        a.bm.copy_(start[1])
        m.zero_()
        torch.cuda.synchronize()

    torch.cuda.synchronize()
    step()
    torch.cuda.synchronize()
    reset()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    for _ in range(3):
        reset()
        step()
        torch.cuda.synchronize()
        eager = [t.clone() for t in (a.slots, a.bm, refs, table, m, live)]
        reset()
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip(eager, (a.slots, a.bm, refs, table, m, live)):
            assert torch.equal(x, y)
    assert a.check() == ibp.IBP_OK


@pytest.mark.parametrize("n_slots", [4095, 32768, 32769, 65536, 65537, 131079])
@pytest.mark.parametrize("at", ["front", "back", "spread"])
def test_fork_and_compact_of_large_pools(n_slots, at):
    """Pools on both sides of the sizes up to which free slots are counted and
    listed in one launch; the counts start 4 bytes past an aligned address."""
    T, H, B, L = 16, 2, 2, 512
    rng = np.random.default_rng(n_slots)
    a = Slots(n_slots, L, 32, 4096)
    free = {"front": np.arange(6), "back": np.arange(n_slots - 6, n_slots),
            "spread": np.sort(rng.choice(n_slots, 6, replace=False))}[at]
    refs = np.ones(n_slots, np.int32)
    refs[free] = 0
    taken = rng.choice(np.flatnonzero(refs), 2 * H * B, replace=False)
    table = np.full((4, H, B), -1, np.int64)
    table[:2] = taken.reshape(2, H, B)
    lens = np.array([2 * T - 1, T + 5, 0, 0], np.int32)
    slots, bits, want_refs = a.bytes(), a.bits(), refs.copy()
    want = fork_model(slots, bits, a.stored, want_refs, table, lens, [0, 1], [3, 2], T)
    g_refs = torch.zeros(n_slots + 1, dtype=torch.int32, device="cuda")[1:]
    g_refs.copy_(torch.from_numpy(refs))
    g_table = torch.from_numpy(table.copy()).cuda()
    ibp.ibp_pages_fork(a.meta, a.slots, n_slots, a.bm, g_refs, g_table, torch.from_numpy(lens).cuda(), ids_of([0, 1]),
                       ids_of([3, 2]), page_tokens=T)
    assert a.check() == ibp.IBP_OK
    np.testing.assert_array_equal(g_table.cpu().numpy(), want)
    np.testing.assert_array_equal(g_refs.cpu().numpy(), want_refs)
    np.testing.assert_array_equal(a.bytes(), slots)
    np.testing.assert_array_equal(a.bits(), bits)
    # two free slots are left: the live pages behind them move into them
    m = torch.empty(n_slots, dtype=torch.int64, device="cuda")
    live = torch.empty(1, dtype=torch.int64, device="cuda")
    ibp.ibp_pages_compact(a.meta, a.slots, n_slots, a.bm, g_refs, m, live, table=g_table)
    assert a.check() == ibp.IBP_OK and int(live) == n_slots - 2
    new = np.where(want_refs > 0, np.arange(n_slots), -1)
    holes = [i for i in np.flatnonzero(want_refs == 0) if i < n_slots - 2]
    movers = [i for i in (n_slots - 1, n_slots - 2) if want_refs[i] > 0]
    assert len(holes) == len(movers)
    for d, s in zip(holes, movers):
        new[s] = d
        want_refs[d], want_refs[s] = want_refs[s], 0
    np.testing.assert_array_equal(m.cpu().numpy(), new)
    np.testing.assert_array_equal(g_refs.cpu().numpy(), want_refs)
    np.testing.assert_array_equal(g_table.cpu().numpy(), np.where(want >= 0, new[want], -1))
