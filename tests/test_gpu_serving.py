"""GPU: the serving operators as they are used together: a prompt through rotary
positions and flex_attention_varlen into the cache, forked continuations
decoded token by token, a prompt that goes on from its cached part, and a
compacted pool."""
import numpy as np
import pytest
import torch

import block_sparse_masked_tile_b200 as bsmt
from oracle import serving as osv
from tests.serving_helpers import Both, ints, running

pytestmark = pytest.mark.gpu

HQ, HKV, D = 8, 2, 64


def projected(T, gen):
    """q, k, v as views of one projection."""
    x = torch.randn((T, HQ + 2 * HKV, D), generator=gen).bfloat16()
    return x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:]


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_prefill_fork_decode_compact(code):
    gen = torch.Generator().manual_seed(0)
    spec = bsmt.rotary_spec(D, [12, 10, 10])
    b = Both(60, HKV, D, 8, 12, 16, 1, code)
    lens = [37, 64, 1]
    cu = running(lens)
    # prompts
    q, k, v = projected(cu[-1], gen)
    pos = np.concatenate([np.stack([np.arange(n), np.arange(n) // 4, np.arange(n) % 4]) for n in lens], 1)
    qr, kr = bsmt.rotary(q.cuda(), k.cuda(), torch.tensor(pos, dtype=torch.int32, device="cuda"), spec)
    turned = [osv.rotary(x.double().numpy(), pos, spec.inv_freq, spec.axis) for x in (q, k)]
    # half a bf16 step of the value, and fp32's share of the pair
    assert np.abs(kr.double().cpu().numpy() - turned[1]).max() <= 2.0 ** -8 * np.abs(turned[1]).max() + 1e-5
    out, _ = bsmt.flex_attention_varlen(qr, kr, v.cuda().contiguous(), ints(cu), ints(cu), causal=True, enable_gqa=True)
    seqs = [4, 0, 2]
    starts = b.extend(seqs, lens)
    bsmt.cache_write(b.dev, ints(seqs), ints(starts), kr, v.cuda(), ints(cu))
    b.ref.write(0, seqs, starts, kr.double().cpu().numpy(), v.double().numpy(), cu)
    b.equal()
    # the prompt's last tokens over the cache: what the prompt's attention gave, up to the codes' rounding
    last = [c - 1 for c in cu[1:]]
    got, _ = b.attend(qr[last].cpu(), seqs, [1] * 3, ("causal",))
    step = 2.0 ** -4 if code == "e4m3" else 2.0 ** -6
    assert (got - out[last]).abs().max() <= 8 * step
    # three continuations
    b.fork([4, 4, 0], [1, 3, 5])
    b.equal()
    live = [4, 1, 3, 0, 5, 2]
    for stepno in range(20):
        q, k, v = projected(len(live), gen)
        at = b.ref.seq_lens[live].astype(np.int64)
        qr, kr = bsmt.rotary(q.cuda(), k.cuda(), torch.tensor(np.stack([at] * 3), dtype=torch.int32, device="cuda"), spec)
        starts = b.extend(live, [1] * len(live))
        b.write(0, live, starts, kr.cpu(), v, [1] * len(live))
        b.attend(qr.cpu(), live, [1] * len(live), ("and", ("causal",), ("or", ("sink", 2), ("window", 40))))
        if stepno == 9:
            b.free([4, 0])
            live = [1, 3, 5, 2]
            before = bsmt.paged_attention(qr[:4], b.dev, ints(live), enable_gqa=True)[0]
            b.compact()
            b.equal()
            assert torch.equal(bsmt.paged_attention(qr[:4], b.dev, ints(live), enable_gqa=True)[0], before)
    b.equal()


def test_prompt_goes_on_from_its_cached_part():
    gen = torch.Generator().manual_seed(1)
    b = Both(40, HKV, D, 3, 12, 32, 1, "int8")
    b.add([0, 2], [50, 90])
    new = [13, 40]
    starts = b.extend([0, 2], new)
    q, k, v = projected(sum(new), gen)
    b.write(0, [0, 2], starts, k, v, new)
    # the new queries over the cache
    out, lse = b.attend(q, [0, 2], new, ("causal",))
    # and through flex_attention_varlen on the whole dequantised sequences: q padded in front
    lens = [63, 130]
    cu = running(lens)
    ck, cv = bsmt.cache_gather(b.dev, ints([0, 2]), None, cu[-1], ints(cu))
    full = torch.zeros((cu[-1], HQ, D), dtype=torch.bfloat16, device="cuda")
    rows = [r for i in range(2) for r in range(cu[i + 1] - new[i], cu[i + 1])]
    full[rows] = q.cuda()
    want, want_lse = bsmt.flex_attention_varlen(full, ck, cv, ints(cu), ints(cu), causal=True, enable_gqa=True)
    bsmt.check_device_status()
    # both are within the library's tolerance of the exact result (2e-2 and 1e-2 for flex_attention)
    assert (out.float() - want[rows].float()).abs().max() <= 2e-2 + 2e-2
    assert (lse - want_lse[:, rows]).abs().max() <= 1e-2 + 1e-3


def test_training_step_through_rotary_and_attention():
    gen = torch.Generator().manual_seed(2)
    spec = bsmt.rotary_spec(D, [16, 16])
    T = 70
    x = torch.randn((1, HQ + 2 * HKV, T, D), generator=gen).bfloat16()
    pos = np.stack([np.arange(T) // 7, np.arange(T) % 7])
    dout = torch.randn((1, HQ, T, D), generator=gen).bfloat16()
    q, k, v = (t.cuda().contiguous().requires_grad_() for t in (x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:]))
    qr, kr = bsmt.rotary(q, k, torch.tensor(pos, dtype=torch.int32, device="cuda"), spec)
    bm = bsmt.create_block_mask(bsmt.causal(), 1, 1, T, T, device="cuda")
    out, _ = bsmt.flex_attention(qr, kr, v, block_mask=bm, enable_gqa=True)
    out.backward(dout.cuda())
    # the formula in 64 bits: a softmax attention of turned q and k
    q6, k6, v6 = (t.detach().cpu().double().requires_grad_() for t in (q, k, v))
    ang = torch.tensor(pos).double()[list(spec.axis)].T * torch.tensor(spec.inv_freq).double()

    def turn(t):
        a, c = t.chunk(2, -1)
        return torch.cat((a * ang.cos() - c * ang.sin(), a * ang.sin() + c * ang.cos()), -1)

    z = turn(q6) @ turn(k6).repeat_interleave(HQ // HKV, 1).transpose(-1, -2) / D ** 0.5
    z = z.masked_fill(torch.ones(T, T, dtype=torch.bool).triu(1), -torch.inf)
    (z.softmax(-1) @ v6.repeat_interleave(HQ // HKV, 1)).backward(dout.double())
    for name, a, w in (("dq", q, q6), ("dk", k, k6), ("dv", v, v6)):
        # the library's backward tolerance: 2e-2 of the tensor's largest gradient
        err, top = (a.grad.cpu().double() - w.grad).abs().max().item(), max(1.0, w.grad.abs().max().item())
        assert err <= 2e-2 * top, (name, err)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_captured_decode_step(code):
    # extend, rotary, write and attention of a padded batch in one CUDA graph, replayed as the sequences grow
    gen = torch.Generator().manual_seed(3)
    spec = bsmt.rotary_spec(D, [16, 16])
    b = Both(60, HKV, D, 6, 12, 16, 1, code)
    b.add([0, 1, 2, 3], [15, 1, 40, 100])
    n = 5
    seqs = ints([2, 0, -1, 3, 1])
    fused = torch.empty((n, HQ + 2 * HKV, D), dtype=torch.bfloat16, device="cuda")
    source = torch.empty_like(fused)
    pos = torch.zeros((2, n), dtype=torch.int32, device="cuda")
    starts = torch.empty(n, dtype=torch.int32, device="cuda")
    mask = bsmt.and_masks(bsmt.causal(), bsmt.or_masks(bsmt.sink(3), bsmt.sliding_window(50)))

    def step():
        fused.copy_(source)
        bsmt.cache_extend(b.dev, seqs, None, starts)
        q, k = bsmt.rotary(fused[:, :HQ], fused[:, HQ:HQ + HKV], pos, spec)
        bsmt.cache_write(b.dev, seqs, starts, k, fused[:, HQ + HKV:])
        return k, q, bsmt.paged_attention(q, b.dev, seqs, mask_mod=mask, enable_gqa=True)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        k, q, (out, lse) = step()
    for i in range(12):
        if i == 6:
            seqs.copy_(ints([3, -1, 1, 4, 0]))
        now = seqs.tolist()
        x = torch.randn((n, HQ + 2 * HKV, D), generator=gen).bfloat16()
        source.copy_(x)
        at = torch.tensor([max(0, int(b.ref.seq_lens[s])) if s >= 0 else 0 for s in now], dtype=torch.int32)
        pos.copy_(torch.stack([at, at // 3]))
        g.replay()
        want = b.ref.extend(now, [1] * n)
        assert starts.tolist() == want
        b.ref.write(0, now, want, k.double().cpu().numpy(), x[:, HQ + HKV:].double().numpy(), range(n + 1))
        b.equal()
        tree = ("and", ("causal",), ("or", ("sink", 3), ("window", 50)))
        o, ls = osv.paged_attention(q.double().cpu().numpy(), b.ref, now, range(n + 1), tree, ())
        b.close(out, lse, o, ls, q.cpu())
