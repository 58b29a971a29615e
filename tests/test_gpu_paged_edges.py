"""GPU: attention over the paged cache where its work list, its modifiers or its
arguments are at an edge, against the fp64 oracle."""
import numpy as np
import pytest
import torch

import block_sparse_masked_tile_b200 as bsmt
from oracle import serving as osv
from tests.serving_helpers import Both, ints, queries, running

pytestmark = pytest.mark.gpu


def filled(lens, heads, dim, page, code, seed=0):
    b = Both(sum(-(-n // page) for n in lens) + 3, heads, dim, len(lens), max(-(-n // page) for n in lens) + 1, page, 1, code, seed)
    order = [int(s) for s in np.random.default_rng(seed).permutation(len(lens))]
    b.add(order, [lens[s] for s in order])
    return b


# Sequences without a query stand, in runs, between others that fall into the same block's share of the work. Many
# sequences of a few tiles each (the plan has several for each thread), or at most 128 (one for each thread) behind one
# whose many queries make the shares large.
@pytest.mark.parametrize("dim, group", [(128, 4), (128, 12), (64, 4), (64, 12), (64, 32)])  # row tiles of 8, 16 and 32
@pytest.mark.parametrize("n, first", [(1500, 0), (129, 600), (128, 600), (121, 600)])
def test_runs_of_sequences_without_queries(dim, group, n, first):
    rng = np.random.default_rng(n + group)
    lens = [int(x) for x in rng.integers(1, 70, n)]
    counts = [int(x) for x in rng.choice([0, 0, 0, 1, 2, 3], n)]
    for at in rng.integers(0, n - 9, 5):
        counts[at:at + 8] = [0] * 8
    if first:
        lens[0], counts[0] = 3000, first
        group = max(1, group // 4) if dim == 64 else group
    b = filled(lens, 1, dim, 32, "e4m3")
    q = queries(sum(counts), group, dim)
    out, lse = b.attend(q, range(n), counts, ("causal",))
    qd, cu, seqs = q.cuda(), ints(running(counts)), ints(range(n))
    for _ in range(30):
        again = bsmt.paged_attention(qd, b.dev, seqs, cu, bsmt.causal(), enable_gqa=True)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    bsmt.check_device_status()


@pytest.mark.parametrize("also", [(), (("alibi", None),)])
@pytest.mark.parametrize("cap", [1e-44, 1e-39, 1e-30, 1e36, 1e38, 2.4e38, 3.4e38])
def test_soft_caps_at_the_ends_of_fp32(cap, also):
    lens = [150, 33]
    b = filled(lens, 2, 64, 32, "e4m3")
    q = queries(4, 4, 64)
    out, lse = b.attend(q, [0, 1], [2, 2], ("causal",), (("softcap", cap),) + also)
    if cap < 1 and not also:  # every score is (nearly) 0
        want = torch.tensor([float(n - 1 + i) for n in lens for i in range(2)]).log()
        assert ((lse.cpu() - want).abs() <= 2e-6 * want).all()


def test_soft_cap_far_below_large_scores():
    # scores beyond any float over the cap, and products q . k of 0 among them (a token of zeros in the query's elements)
    b = filled([60], 1, 64, 32, "int8")
    k = b.values(3)
    k[1, :, 32:] = 0
    starts = b.extend([0], [3])
    b.write(0, [0], starts, k, b.values(3), [3])
    q = queries(2, 4, 64)
    q[:, :, :32] = 0
    q[0] *= 2.0 ** 110
    cap = 2.0 ** -100
    out, lse = bsmt.paged_attention(q.cuda(), b.dev, ints([0]), ints([0, 2]), bsmt.causal(), bsmt.softcap(cap), enable_gqa=True)
    bsmt.check_device_status()
    # scores of magnitude 2^-100: the mean of the values, to P's 11 bits and bf16's half step
    n = torch.tensor([62.0, 63.0])
    assert ((lse.cpu() - n.log()).abs() <= 2e-6 * n.log()).all()
    v = b.ref.tokens(0, 0, 0, 63)[1][:, 0]
    for t in range(2):
        want = v[:62 + t].mean(0)
        top = np.abs(v).max()
        assert (np.abs(out[t].double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -14) * top).all()


@pytest.mark.parametrize("dim, group, count", [(128, 4, 1), (64, 4, 6), (128, 4, 6)])
def test_outputs_as_the_next_calls_queries(dim, group, count):
    # Each call may be set up while the one before it runs, and reads what that one's last kernel writes: the outputs of
    # units that blocks share, in two buffers in turn.
    lens = [9000, 700, 20000, 31]
    b = filled(lens, 2, dim, 64, "e4m3")
    seqs, cu = ints([2, 0, 3, 1]), ints(running([count] * 4))
    start = queries(4 * count, 2 * group, dim).cuda()
    lse = torch.empty((2 * group, 4 * count), device="cuda")
    ws = torch.empty(bsmt.paged_attention_workspace_bytes(dim), dtype=torch.uint8, device="cuda")

    def chain(wait):
        a, c = start.clone(), torch.empty_like(start)
        got = []
        for _ in range(12):
            bsmt.paged_attention(a, b.dev, seqs, cu, bsmt.causal(), None, 4.0, True, out=c, lse=lse, workspace=ws)
            if wait:
                torch.cuda.synchronize()
                got.append(c.clone())
                torch.cuda.synchronize()
            a, c = c, a
        return a, got

    want, steps = chain(True)
    assert all(not torch.equal(x, y) for x, y in zip(steps, steps[1:]))
    for _ in range(20):
        assert torch.equal(chain(False)[0], want)
    bsmt.check_device_status()


@pytest.mark.parametrize("dim, group", [(128, 1), (64, 12), (64, 30)])
@pytest.mark.parametrize("far", [14.0, 20.0, 26.0])  # log2 by which the first token's weight is above each other's
def test_many_small_weights_beside_a_large_one(dim, group, far):
    # A first token that takes most of the weight and whose value is 0, as sinks do: the rest is the output. The sequence
    # is listed so often that a block has all of its keys.
    n, times = 16384, 500
    b = Both(n // 128, 1, dim, 1, n // 128, 128, 1, "e4m3")
    starts = b.extend([0], [n])
    k, v = torch.zeros((n, 1, dim)), 0.75 + 0.5 * torch.rand((n, 1, dim), generator=b.gen)
    k[0, 0, 0], v[0] = 4.0, 0.0
    k[1:, 0, 1] = (torch.arange(1, n) % 4) * 0.25  # small differences among the others
    b.write(0, [0], starts, k.bfloat16(), v.bfloat16(), [n])
    q = torch.zeros((1, group, dim))
    q[..., 0], q[..., 1] = far * float(np.log(2.0)) / 4.0, 0.5
    q = q.bfloat16()
    out, lse = bsmt.paged_attention(q.cuda().repeat(times, 1, 1), b.dev, ints([0] * times), None, None, None, 1.0, True)
    bsmt.check_device_status()
    want, want_lse = osv.paged_attention(q.double().numpy(), b.ref, [0], [0, 1], None, (), 1.0)
    total = np.exp(want_lse[0, 0] - 4.0 * float(q[0, 0, 0]))  # of the weights, the first token's as 1
    # bf16's half step (counted as 2^-8 of the output); P in halves: 2^-11 of each term, and for small ones half of the
    # step 2^-24 where the largest term is 2^7 at least; 2^-14 for exp2, the scores' rounding and fp32 sums
    top = float(np.abs(b.ref.tokens(0, 0, 0, n)[1]).max())
    tol = (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -14) * np.abs(want) + n * 2.0 ** -32 * top / total
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all(), (out[0, 0, :4], want[0, 0, :4])
    assert (np.abs(lse.double().cpu().numpy() - want_lse) <= 1e-5 * np.abs(want_lse)).all()


def test_offsets_that_do_not_begin_at_0():
    b = filled([40, 17], 2, 64, 32, "e4m3")
    q, seqs, cu = queries(8, 4, 64).cuda(), ints([0, 1]), ints([3, 5, 6])

    def reported():
        with pytest.raises(RuntimeError, match="PRECONDITION"):
            bsmt.check_device_status()

    out, lse = torch.full_like(q, 7.0), torch.full((4, 8), 7.0, device="cuda")
    bsmt.paged_attention(q, b.dev, seqs, cu, bsmt.causal(), enable_gqa=True, out=out, lse=lse)
    reported()
    want, want_lse = bsmt.paged_attention(q[3:6], b.dev, seqs, ints([0, 2, 3]), bsmt.causal(), enable_gqa=True)
    assert not out[:3].any() and not out[6:].any() and torch.equal(out[3:6], want)
    assert torch.isneginf(lse[:, :3]).all() and torch.isneginf(lse[:, 6:]).all() and torch.equal(lse[:, 3:6], want_lse)
    bsmt.paged_attention(q, b.dev, ints([]), ints([5]), enable_gqa=True, out=out.fill_(7.0), lse=lse.fill_(7.0))  # no sequence at all
    reported()
    assert not out.any() and torch.isneginf(lse).all()
    k, v = bsmt.cache_gather(b.dev, seqs, ints([0, 0]), 8, cu)
    reported()
    assert not k[:3].any() and k[3:6].any() and not v[6:].any()
    # the tokens inside the offsets are written as they say
    for T, offsets in ((8, [3, 5, 6]), (60, [50, 52, 53])):  # few tokens a sequence, and many
        x = torch.randn((T, 2, 64), generator=torch.Generator().manual_seed(T)).bfloat16().cuda()
        bsmt.cache_write(b.dev, seqs, ints([38, 16]), x, x, ints(offsets))
        reported()
        y = x.double().cpu().numpy()
        b.ref.write(0, [0, 1], [38, 16], y, y, offsets)
        b.equal()
