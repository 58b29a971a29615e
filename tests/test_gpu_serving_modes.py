"""GPU: what the cache's calls do with tensors that are being differentiated."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

import block_sparse_masked_tile_b200 as bsmt
from tests.serving_helpers import ints

pytestmark = pytest.mark.gpu


def test_nothing_is_differentiated_through_the_cache():
    c = bsmt.create_paged_cache(4, 2, 64, 2, 2, 16)
    x = torch.randn((1, 2, 64), device="cuda").bfloat16()
    seqs = ints([1])
    starts = bsmt.cache_extend(c, seqs)
    before = [t.clone() for t in (c.k.view(torch.int8), c.v.view(torch.int8), c.k_scale, c.v_scale)]
    y = x.clone().requires_grad_()
    with fwd.dual_level():
        dual = fwd.make_dual(x, torch.ones_like(x))
        for bad in (y, dual):
            for k, v in ((bad, x), (x, bad)):
                with pytest.raises(ValueError, match="no backward"):
                    bsmt.cache_write(c, seqs, starts, k, v)
            with pytest.raises(ValueError, match="no backward"):
                bsmt.paged_attention(bad, c, seqs)
    assert all(torch.equal(a, b) for a, b in zip(before, (c.k.view(torch.int8), c.v.view(torch.int8), c.k_scale, c.v_scale)))
    with torch.no_grad():  # no gradient is asked for
        bsmt.cache_write(c, seqs, starts, y, y)
        got = bsmt.paged_attention(y, c, seqs)[0]
    k, _ = bsmt.cache_gather(c, seqs, starts, 1)
    bsmt.check_device_status()
    assert torch.equal(got, k) and k.any()  # one key: its value
