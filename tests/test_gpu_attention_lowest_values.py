"""Attention over keys of the type's lowest value: scores near the lowest
number of 32 bits, and beyond it."""
from __future__ import annotations

import math

import pytest
import torch

from lossless_tensor_compression_ibp_amd import ibp
from tests.kv_util import DT, Pool, assert_close, attend64, values

pytestmark = pytest.mark.gpu

T, D = 16, 128


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("tokens", [0, 64, 5000])
@pytest.mark.parametrize("rows", [2, 40])
def test_lowest_keys(rows, tokens, dtype):
    """The first drafted key is the type's lowest value, and so is one key in
    the context.  Their weights are 0 in 64 bits, so the reference leaves them
    out; a row that sees nothing else has, where its score passes 32 bits
    (bf16), a score of -infinity, else that key's value."""
    dt = DT[dtype]
    low = torch.finfo(dt).min
    n = max(1, -(-tokens // T))
    k, v = values(n, T, D, dt, 1), values(n, T, D, dt, 2)
    k.view(-1, D)[n * T // 3] = low
    kp, vp = Pool(k, None), Pool(v, None)
    t = torch.arange(n, device="cuda").reshape(1, 1, n).contiguous()
    g = torch.Generator("cuda").manual_seed(rows)
    q = torch.randn(rows, 2, D, device="cuda", generator=g).to(dt).abs()
    k_new, v_new = (torch.randn(rows, 1, D, device="cuda", generator=g).to(dt) for _ in range(2))
    k_new[0] = low
    sees = [(1 << r) | 1 for r in range(rows)]
    mask = torch.tensor(sees, dtype=torch.int64, device="cuda")[:, None].contiguous()
    ends = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(rows, 2, device="cuda")
    scale = D ** -0.5
    ibp.ibp_tree_attention(kp.pages, vp.pages, q, t, t, torch.tensor([tokens], dtype=torch.int32, device="cuda"), ends,
                           k_new, v_new, mask, out, lse, scale=scale, max_len=tokens, max_new=rows)
    assert kp.check() == ibp.IBP_OK
    ctx = torch.ones(tokens, dtype=torch.bool, device="cuda")
    if tokens > n * T // 3:
        ctx[n * T // 3] = False
    kc, vc = k.view(-1, D)[:tokens][ctx], v.view(-1, D)[:tokens][ctx]
    for r in range(rows):
        for h in range(2):
            if tokens == 0 and r == 0:  # only the lowest key
                t32 = (q[0, h].double() @ k_new[0, 0].double())
                if t32 < -torch.finfo(torch.float32).max:
                    assert not out[0, h].any() and lse[0, h] == -math.inf
                    continue
            mine = slice(r, r + 1 if r or tokens == 0 else 0)
            kr, vr = torch.cat([kc, k_new[mine, 0]]), torch.cat([vc, v_new[mine, 0]])
            seen = torch.ones(kr.shape[0], dtype=torch.bool, device="cuda")
            o, l, tol, ltol = attend64(q[r, h], kr, vr, seen, scale)
            assert_close(out[r, h], o, tol, f"row {r} out")
            assert_close(lse[r, h], l, torch.tensor(ltol, device="cuda"), f"row {r} lse")
