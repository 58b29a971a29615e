"""GPU: rotary in forward mode, and where a token's heads go side by side."""
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


@pytest.mark.parametrize("inter", [False, True])
def test_many_tokens_of_many_heads(inter):
    # enough of both that four heads of a token go side by side (19 heads: the last are fewer), forward and gradient
    spec = bsmt.rotary_spec(128, [24, 20, 20], interleaved=inter)
    T = 20001
    q, k, dq, dk = (tensor((T, h, 128), seed=s) for s, h in enumerate((17, 2, 17, 2)))
    pos = np.random.default_rng(0).integers(0, 30000, (3, T))
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    a, b = q.cuda().requires_grad_(), k.cuda().requires_grad_()
    y, z = bsmt.rotary(a, b, p, spec)
    ga, gb = torch.autograd.grad((y, z), (a, b), (dq.cuda(), dk.cuda()))
    for got, x, inverse in ((y.detach(), q, False), (z.detach(), k, False), (ga, dq, True), (gb, dk, True)):
        close(got, oracle(x, pos, spec, inverse), x)
