"""GPU: rotary in forward mode."""
import numpy as np
import pytest
import torch
import torch.autograd.forward_ad as fwd

import block_sparse_masked_tile_b200 as bsmt
from tests.test_gpu_rotary import close, oracle, tensor

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_tangents_turn_as_their_tensors(dtype):
    spec = bsmt.rotary_spec(64, [12, 10, 6])
    q, k, dq = tensor((29, 3, 64), dtype), tensor((29, 1, 64), dtype, 1), tensor((29, 3, 64), dtype, 2)
    pos = np.random.default_rng(0).integers(0, 500, (3, 29))
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    with fwd.dual_level():
        y, _ = bsmt.rotary(fwd.make_dual(q.cuda(), dq.cuda()), k.cuda(), p, spec)
        y, tangent = fwd.unpack_dual(y)
    close(y, oracle(q, pos, spec), q)
    close(tangent, oracle(dq, pos, spec), dq)
