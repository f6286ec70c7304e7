"""ibp_pages_compact on a pool of no slots: refused, like every call on one."""
from __future__ import annotations

import pytest
import torch

from lossless_tensor_compression_ibp_amd import ibp
from tests.kv_util import Pool, values

pytestmark = pytest.mark.gpu


def test_empty_pool():
    p = Pool(values(64, 16, 64, torch.bfloat16, 1))
    e32, e64 = torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    live = torch.full((1,), 9, dtype=torch.int64, device="cuda")
    with pytest.raises(ibp.IBPError) as e:
        ibp.ibp_pages_compact(p.meta, p.slots, 0, p.bitmask, e32, e64, live)
    assert e.value.status == ibp.IBP_ERR_INVALID_ARG
    assert int(live) == 9
