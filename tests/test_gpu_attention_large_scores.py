"""Attention with scores so large that neighbouring numbers of 32 bits lie many
octaves apart: the softmax is the mean of the values whose score is the
highest."""
from __future__ import annotations

import math

import pytest
import torch

from lossless_tensor_compression_ibp_amd import ibp
from tests.kv_util import DT, Pool, assert_close, half_step

pytestmark = pytest.mark.gpu

T, D = 16, 64


def setting(n, dtype, seed):
    """Keys 1 .. 256 in their first number, exact in both types, the highest and
    the lowest a few times each; values of any kind."""
    g = torch.Generator("cuda").manual_seed(seed)
    k = torch.zeros(n, D, device="cuda")
    k[:, 0] = torch.randint(2, 256, (n,), device="cuda", generator=g)
    at = torch.randperm(n, device="cuda", generator=g)
    k[at[:3], 0], k[at[3:5], 0] = 256, 1
    v = torch.randn(n, D, device="cuda", generator=g)
    return k.to(DT[dtype]), v.to(DT[dtype])


@pytest.mark.parametrize("dtype,q0", [(t, x) for t in ("bf16", "fp16") for x in (1e4, 6e4)]
                         + [("bf16", x) for x in (1e6, 1e7, 1e9, 1e12, 1e20, 1e34)])
@pytest.mark.parametrize("scale", [1.0, 0.1, 7.3])
@pytest.mark.parametrize("n", [64, 6000])
@pytest.mark.parametrize("rows", [1, 40])
def test_highest_scores(rows, n, scale, dtype, q0):
    """Products are exact and neighbouring scores a 256th apart, thousands of
    octaves; scores stay within 32 bits."""
    if q0 * 256 * scale * 1.5 > 3e38:
        pytest.skip("the scores pass 32 bits")
    k, v = setting(n, dtype, rows + n)
    kp, vp = Pool(k.reshape(-1, T, D), None), Pool(v.reshape(-1, T, D), None)
    t = torch.arange(n // T, device="cuda").reshape(1, 1, -1).contiguous()
    q = torch.zeros(rows, 2, D, device="cuda")
    q[:, 0, 0], q[:, 1, 0] = q0, -q0
    q = q.to(DT[dtype])
    new = torch.zeros(rows, 1, D, dtype=DT[dtype], device="cuda")
    mask = torch.zeros(rows, 1, dtype=torch.int64, device="cuda")
    ends = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(rows, 2, device="cuda")
    ibp.ibp_tree_attention(kp.pages, vp.pages, q, t, t, lens, ends, new, new, mask, out, lse, scale=scale, max_len=n,
                           max_new=rows)
    assert kp.check() == ibp.IBP_OK
    f32 = torch.tensor(scale, dtype=torch.float32).double().item()
    h = half_step(DT[dtype])
    for i in range(2):
        best = k[:, 0] == (256 if i == 0 else 1)
        x = v[best].double()
        # equal weights, rounded alike; a product, a sum and a quotient of a few numbers in 32 bits, the output's rounding
        o, tol = x.mean(0), (h + 16 * 2.0 ** -24) * x.abs().mean(0) + h * x.mean(0).abs()
        top = q[0, i, 0].double() * k[best][0, 0].double() * f32
        l = top + math.log(x.shape[0])
        ltol = 2.0 ** -21 * top.abs() + 2.0 ** -20
        assert_close(out[:, i], o.expand(rows, D), tol.expand(rows, D), f"head {i} out")
        assert_close(lse[:, i], l.expand(rows), ltol.expand(rows), f"head {i} lse")
    if rows == 1:
        blocks = torch.arange(n // T, dtype=torch.int32, device="cuda").reshape(1, 1, -1).contiguous()
        sparse = torch.empty_like(out)
        ibp.ibp_sparse_attention(kp.pages, vp.pages, q, t, t, lens, blocks, sparse, scale=scale)
        assert_close(sparse, out.double(), 2 * h * out.double().abs() + 2.0 ** -20, "sparse out")
