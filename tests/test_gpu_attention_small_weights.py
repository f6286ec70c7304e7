"""Attention in fp16 over long contexts whose weights are far below the largest:
they are rounded to fp16 for the product with the values, and must not vanish
there while the softmax's sum counts them."""
from __future__ import annotations

import math

import pytest
import torch

from lossless_tensor_compression_ibp_amd import ibp
from tests.kv_util import Pool, assert_close, attend64

pytestmark = pytest.mark.gpu

T, D = 16, 64


def tolerance(q, k, v):
    """As attend64's, with two bounds that it takes more widely.  Half a step of
    2^-24 of every weight: the largest weight is kept at 2^7 or more, so it
    weighs at most 2^-32 of the largest.  And the sums: the products with the
    values add 32 tokens at a time and the softmax's sum 16 (four lanes, four
    additions a step of 64), so of up to 65,536 tokens no weight passes through
    more than 4,160 additions."""
    o, lse, _, ltol = attend64(q, k, v, torch.ones(k.shape[0], dtype=torch.bool, device="cuda"), 1.0)
    t = k.double() @ q.double()
    p = torch.exp(t - t.max())
    mean, total = (p @ v.double().abs()) / p.sum(), p.sum()
    h, n = 2.0 ** -11, min(k.shape[0], 4160)
    dts = (D + 4) * 2.0 ** -24 * (k.double().abs() @ q.double().abs()).max() + 2.0 ** -21 * (1 + t.abs().max())
    tol = mean * (h + 2 * (dts + n * 2.0 ** -24)) * (1 + h) + h * o.abs()
    return o, lse, tol + 2.0 ** -32 * v.double().abs().sum(0) / total + 2.0 ** -25, ltol


def context(n, octaves):
    """One key whose score is the highest, first, in the middle or last, and
    n - 1 whose scores are `octaves` octaves below; values near 1."""
    g = torch.Generator("cuda").manual_seed(n)
    k = torch.zeros(n, D, device="cuda")
    k[:, 0] = -octaves * math.log(2.0)  # with q = e_0 and scale 1
    v = 1.0 + 0.1 * torch.rand(n, D, device="cuda", generator=g)
    return k.half(), v.half()


@pytest.mark.parametrize("at", ["first", "middle", "last"])
@pytest.mark.parametrize("octaves", [18.0, 25.1, 27.0])
@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("seqs", [1, 64])
def test_many_small_weights(seqs, rows, octaves, at):
    """One sequence, whose context is split over many workgroups (each with a
    maximum of its own), and so many that every context is one workgroup's."""
    n, HK = 65536, 1 if seqs == 1 else 8
    k, v = context(n, octaves)
    big = {"first": 0, "middle": n // 2 + 5, "last": n - 1}[at]
    k[big, 0] = 0
    v[big] = 0
    kp, vp = Pool(k.reshape(-1, T, D), None), Pool(v.reshape(-1, T, D), None)
    t = torch.arange(n // T, device="cuda").expand(seqs, HK, n // T).contiguous()
    R = seqs * rows
    q = torch.zeros(R, HK, D, dtype=torch.float16, device="cuda")
    q[:, :, 0] = 1.0
    new = torch.zeros(R, HK, D, dtype=torch.float16, device="cuda")
    mask = torch.zeros(R, 1, dtype=torch.int64, device="cuda")
    ends = rows * torch.arange(seqs + 1, dtype=torch.int32, device="cuda")
    lens = torch.full((seqs,), n, dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(R, HK, device="cuda")
    o, l, tol, ltol = tolerance(q[0, 0], k, v)
    ltol = torch.full((R, HK), ltol, device="cuda")
    ibp.ibp_tree_attention(kp.pages, vp.pages, q, t, t, lens, ends, new, new, mask, out, lse, scale=1.0, max_len=n,
                           max_new=rows)
    assert kp.check() == ibp.IBP_OK
    assert_close(out, o.expand(out.shape), tol.expand(out.shape), "tree out")
    assert_close(lse, l.expand(R, HK), ltol, "tree lse")
    if rows == 1:
        blocks = torch.arange(n // T, dtype=torch.int32, device="cuda").expand(R, HK, n // T).contiguous()
        ibp.ibp_sparse_attention(kp.pages, vp.pages, q, t, t, lens, blocks, out, lse, scale=1.0)
        assert_close(out, o.expand(out.shape), tol.expand(out.shape), "sparse out")
        assert_close(lse, l.expand(R, HK), ltol, "sparse lse")


def test_rising_scores():
    """The maximum rises step by step: every key that passes the highest so far
    by an octave or two; the weights stay inside fp16's range."""
    n = 4096
    for step in (0.02, 0.4, 9.0):
        k, v = context(n, 0.0)
        k[:, 0] = torch.arange(n, device="cuda") * step - n * step / 2
        v = torch.where(torch.arange(n, device="cuda")[:, None] % 2 == 0, v, v * 3e4).half()
        kp, vp = Pool(k.reshape(-1, T, D), None), Pool(v.reshape(-1, T, D), None)
        t = torch.arange(n // T, device="cuda").reshape(1, 1, -1).contiguous()
        q = torch.zeros(1, 1, D, dtype=torch.float16, device="cuda")
        q[:, :, 0] = 1.0
        o, l, tol, ltol = tolerance(q[0, 0], k, v)
        out, lse = torch.empty_like(q), torch.empty(1, 1, device="cuda")
        blocks = torch.arange(n // T, dtype=torch.int32, device="cuda").reshape(1, 1, -1).contiguous()
        ibp.ibp_sparse_attention(kp.pages, vp.pages, q, t, t, torch.tensor([n], dtype=torch.int32, device="cuda"),
                                 blocks, out, lse, scale=1.0)
        assert_close(out[0], o[None], tol[None], f"step {step} out")
        assert_close(lse[0], l[None], torch.full((1,), ltol, device="cuda"), f"step {step} lse")
