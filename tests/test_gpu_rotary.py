"""GPU: rotary positions against the fp64 oracle, and their gradients."""
import numpy as np
import pytest
import torch

import block_sparse_masked_tile_b200 as bsmt
from oracle import serving as osv

pytestmark = pytest.mark.gpu


def tensor(shape, dtype=torch.bfloat16, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def oracle(x, pos, spec, inverse=False):
    """x [T, H, D], or [B, H, T, D] with pos [axes, B, T]."""
    y = x.double().numpy()
    y = y.transpose(0, 2, 1, 3) if x.dim() == 4 else y
    y = osv.rotary(y, np.asarray(pos, np.int64), spec.inv_freq, spec.axis, spec.interleaved, inverse)
    return y.transpose(0, 2, 1, 3) if x.dim() == 4 else y


def close(got, want, x):
    # the result's rounding (half a step: 2^-8 or 2^-24 of it), and 2^-20 of the pair for the angle (2^-22 of a turn's
    # half, sincospi) and the fp32 products
    eps = torch.finfo(got.dtype).eps / 2
    top = float(x.double().abs().max())
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= eps * np.abs(want) + 2.0 ** -20 * 2 * top).all(), err.max()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D, sections, inter, per_axis", [
    (128, [64], False, False), (128, [24, 20, 20], False, False), (128, [16, 24, 24], True, True), (64, [16, 16], False, True),
    (64, [8], False, False),       # the last 48 elements pass through
    (64, [5, 6], True, False),     # an odd number of pairs: element by element
    (80, [20, 20], False, False), (256, [128], True, False), (6, [1, 1], False, False), (2, [1], False, False)])
@pytest.mark.parametrize("T", [1, 37])
def test_packed(dtype, D, sections, inter, per_axis, T):
    spec = bsmt.rotary_spec(D, sections, interleaved=inter, per_axis=per_axis)
    q, k = tensor((T, 5, D), dtype), tensor((T, 1, D), dtype, 1)
    pos = np.random.default_rng(T).integers(0, 4000, (len(sections), T))
    got = bsmt.rotary(q.cuda(), k.cuda(), torch.tensor(pos, dtype=torch.int32, device="cuda"), spec)
    for g, x in zip(got, (q, k)):
        close(g, oracle(x, pos, spec), x)


def test_batched_layout_and_broadcast_positions():
    spec = bsmt.rotary_spec(64, [20, 12])
    q, k = tensor((3, 4, 50, 64)), tensor((3, 2, 50, 64), seed=1)
    pos = np.random.default_rng(0).integers(0, 900, (2, 3, 50))
    got = bsmt.rotary(q.cuda(), k.cuda(), torch.tensor(pos, dtype=torch.int32, device="cuda"), spec)
    for g, x in zip(got, (q, k)):
        close(g, oracle(x, pos, spec), x)
    one = torch.tensor(pos[:, 0], dtype=torch.int32, device="cuda")
    got = bsmt.rotary(q.cuda(), None, one, spec)
    assert got[1] is None
    close(got[0], oracle(q, np.broadcast_to(pos[:, :1], pos.shape), spec), q)


def test_far_and_negative_positions_keep_accuracy():
    spec = bsmt.rotary_spec(64)
    pos = np.array([[0, 1, -1, 2 ** 20, 2 ** 31 - 1, -2 ** 31, 123456789]])
    x = tensor((7, 2, 64), torch.float32)
    got, _ = bsmt.rotary(x.cuda(), None, torch.tensor(pos, dtype=torch.int32, device="cuda"), spec)
    # the oracle's own angle: 2^31 in fp64 is off by 2^-22
    err = np.abs(got.double().cpu().numpy() - oracle(x, pos, spec))
    assert err.max() <= 2.0 ** -19 * float(x.abs().max())


def test_strided_views_of_a_fused_projection():
    spec = bsmt.rotary_spec(128, [30, 34])
    T, Hq, Hkv = 33, 4, 2
    fused = tensor((T, Hq + 2 * Hkv, 128))
    pos = np.random.default_rng(0).integers(0, 100, (2, T))
    dev = fused.cuda()
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    for off in (0, 1):  # off 1: rows that are not 16-byte aligned
        wide = torch.zeros((T, Hq + 2 * Hkv, 136), dtype=torch.bfloat16, device="cuda")
        wide[..., off:128 + off] = dev
        q, k = wide[:, :Hq, off:128 + off], wide[:, Hq:Hq + Hkv, off:128 + off]
        got = bsmt.rotary(q, k, p, spec)
        for g, x in zip(got, (fused[:, :Hq], fused[:, Hq:Hq + Hkv])):
            assert g.is_contiguous()
            close(g, oracle(x, pos, spec), x)
    # positions with strides of their own, and [B, H, T, D] as a view of [B, T, H, D]
    q = tensor((2, T, Hq, 128)).cuda().transpose(1, 2)
    p2 = torch.tensor(np.stack([pos, pos + 3], -1), dtype=torch.int32, device="cuda").movedim(-1, 1)
    got, _ = bsmt.rotary(q, None, p2, spec)
    close(got, oracle(q.cpu(), p2.cpu().numpy(), spec), q)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
def test_gradients(dtype, inter):
    spec = bsmt.rotary_spec(64, [12, 10, 6], interleaved=inter)
    T = 29
    q, k = tensor((2, 3, T, 64), dtype), tensor((2, 1, T, 64), dtype, 1)
    dq, dk = tensor((2, 3, T, 64), dtype, 2), tensor((2, 1, T, 64), dtype, 3)
    pos = np.random.default_rng(0).integers(0, 500, (3, 2, T))
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    a, b = q.cuda().requires_grad_(), k.cuda().requires_grad_()
    yq, yk = bsmt.rotary(a, b, p, spec)
    gq, gk = torch.autograd.grad((yq, yk), (a, b), (dq.cuda(), dk.cuda()))
    close(gq, oracle(dq, pos, spec, True), dq)
    close(gk, oracle(dk, pos, spec, True), dk)
    for g, w in zip(bsmt.rotary_backward(dq.cuda(), dk.cuda(), p, spec), (gq, gk)):
        assert torch.equal(g, w)
    # one of the two alone, a broadcast gradient, and leaves that need none
    yq, yk = bsmt.rotary(a, b.detach(), p, spec)
    (gq,) = torch.autograd.grad(yq.float().sum(), a)
    close(gq, oracle(torch.ones_like(q), pos, spec, True), torch.ones_like(q))
    yq, yk = bsmt.rotary(a, b, p, spec)
    yk.float().sum().backward()
    assert a.grad is None or not a.grad.any()
    assert b.grad is not None


def test_gradient_equals_differences_and_differentiates_again():
    spec = bsmt.rotary_spec(6, [2, 1])
    p = torch.tensor([[3, 1, 4], [1, 5, 9]], dtype=torch.int32, device="cuda")
    x = tensor((3, 2, 6), torch.float32).cuda().requires_grad_()
    w = tensor((3, 2, 6), torch.float32, 1).cuda()
    f = lambda t: (bsmt.rotary(t, None, p, spec)[0] * w).sin().sum()  # noqa: E731
    (g,) = torch.autograd.grad(f(x), x, create_graph=True)
    with torch.no_grad():
        for at in ((0, 0, 0), (1, 1, 2), (2, 0, 5)):
            h = torch.zeros_like(x)
            h[at] = 0.01
            # central differences: h^2 / 6 of the third derivative (w^3 at most 30 here), and fp32 sums
            assert abs(((f(x + h) - f(x - h)) / 0.02 - g[at]).item()) < 2e-3
    (gg,) = torch.autograd.grad(g.square().sum(), x)
    assert torch.isfinite(gg).all() and gg.abs().max() > 0


def test_captured_backward_beside_nothing_eager():
    spec = bsmt.rotary_spec(64)
    p = torch.arange(16, dtype=torch.int32, device="cuda")
    x, w = tensor((16, 2, 64)).cuda().requires_grad_(), tensor((16, 2, 64), seed=1).cuda()
    want = torch.autograd.grad(bsmt.rotary(x, None, p, spec)[0], x, w)[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(bsmt.rotary(x, None, p, spec)[0], x, w)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = torch.autograd.grad(bsmt.rotary(x, None, p, spec)[0], x, w)[0]
    g.replay()
    assert torch.equal(got, want)
    p.add_(5)
    g.replay()
    assert torch.equal(got, torch.autograd.grad(bsmt.rotary(x, None, p, spec)[0], x, w)[0])


def test_empty_and_argument_errors():
    spec, pos = bsmt.rotary_spec(64), torch.zeros(4, dtype=torch.int32, device="cuda")
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    q, k = bsmt.rotary(x[:0], x[:0], pos[:0], spec)
    assert q.shape == (0, 2, 64) and k.shape == (0, 2, 64)
    for bad in (pos.long(), pos[:3], pos.cpu(), pos.view(2, 2)):
        with pytest.raises(ValueError, match="positions"):
            bsmt.rotary(x, None, bad, spec)
    for k in (x[:3], x.float(), x[None]):
        with pytest.raises(ValueError, match="share"):
            bsmt.rotary(x, k, pos, spec)


def test_more_than_two_billion_elements():
    # strides pass 32 bits: two heads of a wide buffer (allocated in bf16, 4.4 GB)
    spec = bsmt.rotary_spec(64)
    big = torch.zeros((2, 1100000000), dtype=torch.bfloat16, device="cuda")
    x = big[:, -64 * 3:].view(2, 3, 64)
    x.copy_(tensor((2, 3, 64)))
    p = torch.tensor([7, 11], dtype=torch.int32, device="cuda")
    got, _ = bsmt.rotary(x, None, p, spec)
    close(got, oracle(tensor((2, 3, 64)), np.array([[7, 11]]), spec), x)
