"""ibp_pages_alloc_raw's refusals that need no GPU."""
import pytest
import torch

from lossless_tensor_compression_ibp_amd import ibp


def test_refusals():
    assert ibp.lib().ibp_pages_alloc_raw(None, None, 1, None, None, 1, None, 0, None) == ibp.IBP_ERR_INVALID_ARG
    meta = ibp.Meta(None, 4096, 32)
    refs, bm, ids = torch.zeros(40, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(4, dtype=torch.int64)
    for what, args in (("refs", (refs[:8], 40, bm, ids)), ("bitmask", (refs, 40, bm[:1], ids)),
                       ("ids", (refs, 40, bm, ids.int())), ("refs", (refs.long(), 40, bm, ids))):
        with pytest.raises(ValueError, match=what):
            ibp.ibp_pages_alloc_raw(meta, *args)
