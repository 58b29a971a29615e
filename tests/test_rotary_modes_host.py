"""Host: rotary's differentiation in reverse and forward mode, with a plain 64-bit
turn in the kernel's place."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

import block_sparse_masked_tile_b200 as bsmt
from block_sparse_masked_tile_b200 import serving as sv

SPEC = bsmt.rotary_spec(10, [2, 2])  # the last two elements pass through
POS = torch.tensor([[3, 1, 4], [1, 5, -9]], dtype=torch.int32)


def plain(tensors, positions, spec, inverse):
    n = len(spec.inv_freq)
    t = (positions.double()[list(spec.axis)].t() * torch.tensor(spec.inv_freq, dtype=torch.float64))[:, None]
    c, s = t.cos(), t.sin() * (-1 if inverse else 1)
    out = []
    for x in tensors:
        assert x.stride(-1) == 1
        x = x.detach()
        a, b = x[..., :n], x[..., n:2 * n]
        out.append(torch.cat((a * c - b * s, a * s + b * c, x[..., 2 * n:]), -1))
    return out


@pytest.fixture(autouse=True)
def no_kernel(monkeypatch):
    monkeypatch.setattr(sv, "_rotary", plain)
    monkeypatch.setattr(sv, "_rotary_args", lambda q, k, positions, spec: [q] if k is None else [q, k])


def heads(n, seed=0, grad=False):
    return torch.randn((3, n, 10), dtype=torch.float64, generator=torch.Generator().manual_seed(seed)).requires_grad_(grad)


def test_every_mode_against_differences():
    f = lambda q, k: bsmt.rotary(q, k, POS, SPEC)  # noqa: E731
    args = heads(2, 0, True), heads(1, 1, True)
    assert torch.autograd.gradcheck(f, args, check_forward_ad=True)
    assert torch.autograd.gradgradcheck(f, args, check_fwd_over_rev=True)


def test_tangents_are_kept():
    q, k, tangent = heads(2), heads(1, 1), heads(2, 2)
    with fwd.dual_level():
        for grad in (True, False):
            with torch.set_grad_enabled(grad):
                y, z = bsmt.rotary(fwd.make_dual(q, tangent), k, POS, SPEC)
                assert torch.equal(fwd.unpack_dual(y).tangent, plain([tangent], POS, SPEC, False)[0])
                assert torch.equal(y, plain([q], POS, SPEC, False)[0])
                other = fwd.unpack_dual(z).tangent
                assert other is None or not other.any()
                # rows of stride 0
                (y, _) = bsmt.rotary(fwd.make_dual(q, torch.ones(3, 2, 1, dtype=torch.float64).expand(3, 2, 10)), None, POS, SPEC)
                assert torch.equal(fwd.unpack_dual(y).tangent, plain([torch.ones_like(q)], POS, SPEC, False)[0])
    assert bsmt.rotary(q, None, POS, SPEC)[0].grad_fn is None


def test_rotary_backward_keeps_the_graph():
    f = lambda dq, dk: bsmt.rotary_backward(dq, dk, POS, SPEC)  # noqa: E731
    assert torch.autograd.gradcheck(f, (heads(2, 0, True), heads(1, 1, True)), check_forward_ad=True)
    assert bsmt.rotary_backward(heads(2), None, POS, SPEC)[0].grad_fn is None


def test_an_output_needs_a_gradient_where_its_tensor_does():
    for q, k in ((heads(2, 0, True), heads(1, 1)), (heads(2), heads(1, 1, True)), (heads(2, 0, True), heads(1, 1, True))):
        y, z = bsmt.rotary(q, k, POS, SPEC)
        assert y.requires_grad == q.requires_grad and z.requires_grad == k.requires_grad
        (y.sum() + z.sum()).backward()
        assert (q.grad is not None) == q.requires_grad and (k.grad is not None) == k.requires_grad
