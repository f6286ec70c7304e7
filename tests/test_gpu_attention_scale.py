"""Attention with scales of zero and far below one, beside scores that are
large before they are scaled."""
from __future__ import annotations

import pytest
import torch

from lossless_tensor_compression_ibp_amd import ibp
from tests.kv_util import Pool, assert_close, attend64, values

pytestmark = pytest.mark.gpu

T, D = 16, 128


@pytest.mark.parametrize("scale,large", [(0.0, 1.0), (0.0, 1e15), (1e-35, 2e16), (-1e-35, 2e16), (3e-38, 4e18),
                                         (1e-40, 4e18)])
@pytest.mark.parametrize("rows", [1, 40])
def test_scale(rows, scale, large):
    """Numbers of q and of the keys around `large`, scores up to 1e37 before
    the scale."""
    k, v = values(9, T, D, torch.bfloat16, 1) * large, values(9, T, D, torch.bfloat16, 2)
    kp, vp = Pool(k, None), Pool(v, None)
    t = torch.arange(9, device="cuda").reshape(1, 1, 9).contiguous()
    n = 9 * T - 5
    q = (torch.randn(rows, 2, D, device="cuda") * min(large, 1e17)).bfloat16()
    new = torch.zeros(rows, 1, D, dtype=torch.bfloat16, device="cuda")
    mask = torch.zeros(rows, 1, dtype=torch.int64, device="cuda")
    ends = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(rows, 2, device="cuda")
    ibp.ibp_tree_attention(kp.pages, vp.pages, q, t, t, lens, ends, new, new, mask, out, lse, scale=scale, max_new=rows)
    assert kp.check() == ibp.IBP_OK
    seen = torch.ones(n, dtype=torch.bool, device="cuda")
    kc, vc = k.reshape(-1, D)[:n], v.reshape(-1, D)[:n]
    f32 = torch.tensor(scale, dtype=torch.float32).item()  # what the call takes
    for r in range(rows):
        for h in range(2):
            o, l, tol, ltol = attend64(q[r, h], kc, vc, seen, f32)
            assert_close(out[r, h], o, tol, f"row {r} out")
            assert_close(lse[r, h], l, torch.tensor(ltol, device="cuda"), f"row {r} lse")
