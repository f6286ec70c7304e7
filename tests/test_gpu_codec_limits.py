"""Rows that are not a multiple of 16 bytes take a wave each, of which one
launch holds fewer than 2^26 (the runtime takes larger numbers of threads
modulo 2^32): more rows take several launches."""
from __future__ import annotations

import pytest
import torch

from lossless_tensor_compression_ibp_amd import ibp

pytestmark = pytest.mark.gpu

L, N = 20, 2 ** 26 + 37


def test_rows_of_20_bytes():
    i = torch.arange(N, dtype=torch.int32, device="cuda")
    words = torch.stack([(i >> 9 * j) & 511 for j in (0, 1, 2)] + [i & 255, i & 127], 1)
    words[5::11] = ~words[5::11]  # rows that stay raw among records
    raw = words.view(torch.uint8)
    meta = ibp.ibp_build_metadata(raw, 1024, L, 32, 32, 0.9)
    slots, bm = torch.full_like(raw, 7), torch.zeros((N + 31) // 32, dtype=torch.int32, device="cuda")
    stored = torch.zeros(N, dtype=torch.int64, device="cuda")
    ibp.ibp_compress(meta, raw, N, slots, bm, stored)
    # the last rows by themselves are stored alike
    first = (N - 1000) // 32 * 32
    n = N - first
    tail, tbm = torch.full_like(raw[first:], 7), torch.zeros((n + 31) // 32, dtype=torch.int32, device="cuda")
    tstored = torch.zeros(n, dtype=torch.int64, device="cuda")
    ibp.ibp_compress(meta, raw[first:].contiguous(), n, tail, tbm, tstored)
    assert torch.equal(slots[first:], tail) and torch.equal(bm[first // 32:], tbm) and torch.equal(stored[first:], tstored)
    assert bool((tstored < L).any()) and bool((tstored == L).any())
    out = torch.full_like(raw, 9)
    ibp.ibp_decompress(meta, slots, bm, N, out)
    assert ibp.ibp_check(meta) == ibp.IBP_OK and torch.equal(out, raw)
    ids = torch.randint(0, N, (N,), device="cuda")
    out.fill_(9)
    ibp.ibp_gather_decompress(meta, slots, N, bm, ids, out)
    assert ibp.ibp_check(meta) == ibp.IBP_OK
    for at in range(0, N, 1 << 24):
        assert torch.equal(out[at:at + (1 << 24)], raw[ids[at:at + (1 << 24)]])
