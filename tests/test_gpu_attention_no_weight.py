"""Rows whose every key has a score of minus infinity: zeros, and a log-sum-exp
of minus infinity, whatever the values are."""
from __future__ import annotations

import math

import pytest
import torch

from lossless_tensor_compression_ibp_amd import ibp
from tests.kv_util import DT, Pool, values

pytestmark = pytest.mark.gpu

T, D = 16, 128


def setting(n, dtype, odd):
    """Keys that give -infinity to any q with a positive first number; values of
    which some are `odd`."""
    k, v = values(n, T, D, DT[dtype], 1), values(n, T, D, DT[dtype], 2)
    k[:, :, 0] = -math.inf
    v[::3, ::5, 7] = odd
    return Pool(k, None), Pool(v, None)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("odd", [1.0, math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("tokens", [0, 50, 6000])
@pytest.mark.parametrize("rows", [1, 40])
def test_tree(rows, tokens, odd, dtype):
    """Contexts of one part and of several; the drafted keys alike."""
    n = max(1, -(-tokens // T))
    kp, vp = setting(n, dtype, odd)
    t = torch.arange(n, device="cuda").reshape(1, 1, n).contiguous()
    q = torch.randn(rows, 4, D, device="cuda").to(DT[dtype])
    q[:, :, 0] = 1.0
    k_new, v_new = (torch.randn(rows, 1, D, device="cuda").to(DT[dtype]) for _ in range(2))
    k_new[:, :, 0] = -math.inf
    v_new[:, :, 9] = odd
    mask = torch.full((rows, 1), -1, dtype=torch.int64, device="cuda")
    ends = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    out, lse = torch.full_like(q, 3.0), torch.zeros(rows, 4, device="cuda")
    ibp.ibp_tree_attention(kp.pages, vp.pages, q, t, t, torch.tensor([tokens], dtype=torch.int32, device="cuda"), ends,
                           k_new, v_new, mask, out, lse, scale=0.1, max_len=tokens, max_new=rows)
    assert kp.check() == ibp.IBP_OK
    assert torch.equal(out, torch.zeros_like(out)) and bool((lse == -math.inf).all())


@pytest.mark.parametrize("odd", [math.inf, math.nan])
def test_rows_beside_others(odd):
    """One row with a weight, the others without: each by itself."""
    kp, vp = setting(3, "bf16", 1.0)
    t = torch.arange(3, device="cuda").reshape(1, 1, 3).contiguous()
    q = torch.randn(3, 2, D, device="cuda").bfloat16()
    q[:, :, 0] = 1.0
    k_new, v_new = (torch.randn(3, 1, D, device="cuda").bfloat16() for _ in range(2))
    k_new[:2, :, 0] = -math.inf
    v_new[:, :, 9] = odd
    mask = torch.tensor([[1], [3], [4]], dtype=torch.int64, device="cuda")
    ends = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(3, 2, device="cuda")
    ibp.ibp_tree_attention(kp.pages, vp.pages, q, t, t, torch.zeros(1, dtype=torch.int32, device="cuda"), ends, k_new,
                           v_new, mask, out, lse, scale=0.1, max_new=3)
    assert not out[:2].any() and bool((lse[:2] == -math.inf).all())
    want = v_new[2, 0].expand(2, D)
    got = out[2]
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    ok = ~torch.isnan(want)
    assert torch.equal(got[ok], want[ok]) and bool(torch.isfinite(lse[2]).all())


@pytest.mark.parametrize("odd", [math.inf, math.nan])
@pytest.mark.parametrize("top", [5, 400])
def test_sparse(top, odd):
    kp, vp = setting(400, "bf16", odd)
    t = torch.arange(400, device="cuda").reshape(1, 1, 400).contiguous()
    q = torch.randn(1, 4, D, device="cuda").bfloat16()
    q[:, :, 0] = 1.0
    blocks = torch.arange(top, dtype=torch.int32, device="cuda").reshape(1, 1, top).contiguous()
    out, lse = torch.full_like(q, 3.0), torch.zeros(1, 4, device="cuda")
    ibp.ibp_sparse_attention(kp.pages, vp.pages, q, t, t, torch.tensor([6400], dtype=torch.int32, device="cuda"),
                             blocks, out, lse, scale=0.1)
    assert torch.equal(out, torch.zeros_like(out)) and bool((lse == -math.inf).all())
