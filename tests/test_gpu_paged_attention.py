"""GPU: attention over the paged cache against the fp64 oracle."""
import numpy as np
import pytest
import torch

import block_sparse_masked_tile_b200 as bsmt
import workloads
from oracle import serving as osv
from tests.serving_helpers import Both, ints, queries

pytestmark = pytest.mark.gpu

STREAM = ("and", ("causal",), ("or", ("sink", 4), ("window", 70)))


def filled(lens, heads=2, dim=128, page=64, code="e4m3", layers=1, spare=3, spread=1.0, seed=0):
    b = Both(sum(-(-n // page) for n in lens) + spare, heads, dim, len(lens) + 1, max(1, max(-(-n // page) for n in lens)) + 1,
             page, layers, code, seed)
    order = [int(s) for s in np.random.default_rng(seed).permutation(len(lens))]  # pages of the sequences interleave
    for part in range(2):
        b.add(order, [(lens[s] + part) // 2 for s in order], spread)
    return b


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_one_query_each(code, dim, page):
    lens = [1, 2, 15, 16, 17, 31, 33, 64, 65, 127, 129, 500, 0]
    b = filled(lens, 2, dim, page, code)
    b.attend(queries(len(lens), 8, dim), range(len(lens)), [1] * len(lens), ("causal",))
    b.attend(queries(len(lens), 8, dim), list(range(len(lens)))[::-1], [1] * len(lens), None)


@pytest.mark.parametrize("heads, group", [(1, 1), (3, 2), (1, 7), (2, 16), (1, 17), (1, 40)])
@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_groups(heads, group, code):
    lens = [200, 77, 1]
    b = filled(lens, heads, 64, 32, code)
    b.attend(queries(3, heads * group, 64), range(3), [1] * 3, ("causal",))
    b.attend(queries(9, heads * group, 64), [1, 0, 2], [4, 4, 1], ("causal",))


@pytest.mark.parametrize("tree", [None, ("causal",), STREAM, ("and", ("causal",), ("window", 33)), ("sink", 0), ("window", -1000),
                                  ("and", ("causal",), ("sink", 3)), ("prefix_lm", 90), ("window", 1),
                                  ("or", ("and", ("sink", 40), ("window", 5)), ("and", ("causal",), ("window", 2)))])
@pytest.mark.parametrize("dim, page, code", [(128, 16, "int8"), (64, 64, "e4m3")])
def test_masks(tree, dim, page, code):
    lens = [300, 129, 5, 70]
    b = filled(lens, 2, dim, page, code)
    for counts in ([1] * 4, [7, 3, 5, 0], [40, 1, 2, 33]):
        b.attend(queries(sum(counts), 8, dim), range(4), counts, tree)


def test_random_masks():
    rng = np.random.default_rng(7)
    b = filled([250, 91, 33], 1, 64, 16, "e4m3")
    for _ in range(25):
        tree = workloads.random_mask_tree(rng, 1, 250, 250, depth=3, allow_document=False)
        try:
            counts = [int(x) for x in rng.integers(0, 9, 3)]
            if sum(counts):
                b.attend(queries(sum(counts), 4, 64), range(3), counts, tree)
        except RuntimeError as e:
            assert "UNSUPPORTED" in str(e)  # more than 16 alternatives


@pytest.mark.parametrize("mods", [(("softcap", 2.0),), (("alibi", None),), (("softcap", 5.0), ("alibi", None)),
                                  (("alibi", [0.5, -0.1, 0.0, 2.0, 0.3, 0.01, 1.0, 0.2]), ("softcap", 3.0))])
@pytest.mark.parametrize("dim, code, count", [(128, "e4m3", 1), (64, "int8", 5)])
def test_score_mods(mods, dim, code, count):
    b = filled([150, 64, 9], 2, dim, 32, code)
    b.attend(queries(3 * count, 8, dim), [2, 1, 0], [count] * 3, ("causal",), mods)
    b.attend(queries(3 * count, 8, dim), [2, 1, 0], [count] * 3, STREAM, mods, scale=0.3)


@pytest.mark.parametrize("cap", [0.25, 64.0, 65.0, 1e4, 1e30])
@pytest.mark.parametrize("also", [(), (("alibi", None),)])
def test_soft_caps_of_any_size(cap, also):
    # far above the scores a cap changes nothing; far below, every score is its sign times the cap
    b = filled([150, 33], 2, 64, 32, "e4m3")
    q = queries(4, 4, 64)
    out, lse = b.attend(q, [0, 1], [2, 2], ("causal",), (("softcap", cap),) + also)
    if cap == 1e30:
        b.close(out, lse, *osv.paged_attention(q.double().numpy(), b.ref, [0, 1], [0, 2, 4], ("causal",), also), q)


def test_padded_batches_and_empty_sequences():
    b = filled([40, 0, 17], 2, 128, 16, "e4m3")
    q = queries(10, 4, 128)
    out, lse = b.attend(q, [0, -1, 1, 2, -1], [2, 3, 1, 2, 0], ("causal",))  # 2 rows behind the pack
    assert not out[2:6].any() and torch.isinf(lse[:, 2:6]).all() and not out[8:].any() and torch.isinf(lse[:, 8:]).all()
    assert out[:2].any() and out[6:8].any()
    # more queries than tokens: those at negative positions see nothing under causal, everything under no mask
    b.attend(queries(20, 4, 128), [2], [20], ("causal",))
    b.attend(queries(20, 4, 128), [2], [20], None)
    # nothing but padding
    out, lse = bsmt.paged_attention(q.cuda(), b.dev, ints([]), ints([0]), enable_gqa=True)
    bsmt.check_device_status()
    assert not out.any() and torch.isinf(lse).all()
    assert bsmt.paged_attention(q[:0].cuda(), b.dev, ints([]), enable_gqa=True)[0].shape == (0, 4, 128)


@pytest.mark.parametrize("dim, group, count", [(128, 8, 1), (64, 1, 1), (128, 4, 9)])
def test_long_sequences_split_over_blocks(dim, group, count):
    lens = [9000, 3, 4096, 1]
    b = filled(lens, 1, dim, 128, "e4m3")
    q = queries(sum(min(count, n) for n in lens), group, dim)
    first = b.attend(q, range(4), [min(count, n) for n in lens], ("causal",))
    again = b.attend(q, range(4), [min(count, n) for n in lens], ("causal",))
    assert all(torch.equal(x, y) for x, y in zip(first, again))
    b.attend(q, range(4), [min(count, n) for n in lens], STREAM)


def test_many_short_sequences():
    n = 700  # more than one sequence for each thread of the plan, more units than blocks
    lens = [int(x) for x in np.random.default_rng(0).integers(0, 40, n)]
    b = filled(lens, 2, 64, 16, "int8")
    b.attend(queries(n, 4, 64), [int(x) for x in np.random.default_rng(1).permutation(n)], [1] * n, ("causal",))


def test_scales_far_apart():
    # V values of one sequence over 2^40, K's over 2^12: P times the scale stays a half
    b = Both(20, 1, 64, 1, 20, 16, 1, "e4m3")
    for i, e in enumerate((0, 20, -20, 3, -6, 12, 0)):
        starts = b.extend([0], [16])
        b.write(0, [0], starts, b.values(16) * 2.0 ** (e % 7 - 3), b.values(16) * 2.0 ** e, [16])
    b.equal()
    q = queries(1, 4, 64)
    for tree in (None, ("window", 17), ("and", ("sink", 16), ("causal",))):
        mask = None if tree is None else bsmt.mask_from_tree(tree)
        out, lse = bsmt.paged_attention(q.cuda(), b.dev, ints([0]), None, mask, enable_gqa=True)
        want, want_lse = osv.paged_attention(q.double().numpy(), b.ref, [0], [0, 1], tree, ())
        b.close(out, lse, want, want_lse, q)
    # a window that sees the small values alone is as exact as they are
    b = Both(4, 1, 64, 1, 4, 16, 1, "e4m3")
    for e in (20, -20):
        starts = b.extend([0], [16])
        b.write(0, [0], starts, b.values(16), b.values(16) * 2.0 ** e, [16])
    out, _ = bsmt.paged_attention(q.cuda(), b.dev, ints([0]), None, bsmt.sliding_window(16), enable_gqa=True)
    want, _ = osv.paged_attention(q.double().numpy(), b.ref, [0], [0, 1], ("window", 16), ())
    assert np.abs(out.double().cpu().numpy() - want).max() <= (2.0 ** -8 + 2.0 ** -10) * 448 * 2.0 ** -28


def test_large_small_and_non_finite_queries():
    b = filled([100], 1, 64, 16, "int8")
    q = queries(6, 2, 64)
    q[0] *= 2.0 ** 60
    q[1] *= 2.0 ** -100
    q[2, 0, 3] = float("nan")
    q[3, 1, 0] = float("inf")
    q[4] = 0
    q[5, 0, :32] *= 2.0 ** -30
    seqs, cu = ints([0]), ints([0, 6])
    out, lse = bsmt.paged_attention(q.cuda(), b.dev, seqs, cu, bsmt.causal(), None, 2.0 ** -60, True)
    bsmt.check_device_status()
    assert torch.isnan(out[2, 0]).all() and torch.isnan(lse[0, 2]) and torch.isnan(out[3, 1]).all()
    with np.errstate(invalid="ignore"):
        want, want_lse = osv.paged_attention(q.double().numpy(), b.ref, [0], [0, 6], ("causal",), (), 2.0 ** -60)
    fine = [0, 1, 4, 5]
    top = 127 * b.ref.v_scale.max()
    assert np.abs(out[fine].double().cpu().numpy() - want[fine]).max() <= (2.0 ** -8 + 2.0 ** -10) * top
    assert torch.isfinite(out[2, 1]).all() and torch.isfinite(out[3, 0]).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("count, group", [(6, 4), (3, 4), (1, 4)])  # row tiles of 16 or 32, 16, 8
def test_masked_nan_does_not_reach_the_result(count, group, dim):
    b = filled([90], 2, dim, 32, "e4m3")
    q = queries(count, 2 * group, dim)
    clean, _ = b.attend(q, [0], [count], STREAM)
    # NaN where no query looks: behind the end, between the sinks and the window
    d = b.dev
    k, v = d.k.view(torch.int8), d.v.view(torch.int8)
    for x in (k, v):
        for tok in (90, 95, 10, 4, 13):
            x[0, d.page_table[0, tok // 32], :, tok % 32] = 0x7F
    got, lse = bsmt.paged_attention(q.cuda(), d, ints([0]), ints([0, count]), bsmt.mask_from_tree(STREAM), enable_gqa=True)
    bsmt.check_device_status()
    assert torch.equal(got, clean)
    # NaN in the V of the newest token reaches the query that sees it, in that column, and no other
    v[0, d.page_table[0, 2], 1, 89 - 64, 5] = 0x7F
    got, lse = bsmt.paged_attention(q.cuda(), d, ints([0]), ints([0, count]), bsmt.mask_from_tree(STREAM), enable_gqa=True)
    want = clean.clone()
    want[-1, group:, 5] = float("nan")
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))
    assert torch.isfinite(lse).all()


def test_bad_pages_and_lists_are_reported():
    b = filled([90, 40], 2, 64, 32, "e4m3")
    q = queries(2, 4, 64).cuda()

    def raises(status):
        with pytest.raises(RuntimeError, match=status):
            bsmt.check_device_status()

    for seqs in ([0, 5], [-2, 1]):
        bsmt.paged_attention(q, b.dev, ints(seqs), enable_gqa=True)
        raises("BOUNDS")
    for cu in ([0, 2, 1], [0, 1, 3], [-1, 1, 2]):
        bsmt.paged_attention(q, b.dev, ints([0, 1]), ints(cu), enable_gqa=True)
        raises("PRECONDITION")
    for page in (-1, 100, -2 ** 31, 2 ** 31 - 1):
        b.dev.page_table[0, 1] = page
        bsmt.paged_attention(q, b.dev, ints([0, 1]), enable_gqa=True)
        raises("BOUNDS")
    b.dev.seq_lens[1] = 33 * 32
    bsmt.paged_attention(q, b.dev, ints([0, 1]), enable_gqa=True)
    raises("BOUNDS")


def test_layers_workspace_and_out():
    b = filled([90, 40], 2, 64, 32, "int8", layers=3)
    q = queries(2, 4, 64)
    ws = torch.full((bsmt.paged_attention_workspace_bytes(64),), 255, dtype=torch.uint8, device="cuda")
    for layer in (2, 0):
        out, lse = torch.empty_like(q, device="cuda"), torch.empty((4, 2), device="cuda")
        got = b.attend(q, [0, 1], [1, 1], ("causal",), layer=layer, workspace=ws, out=out, lse=lse)
        assert got[0] is out and got[1] is lse
    with pytest.raises(ValueError, match="workspace"):
        bsmt.paged_attention(q.cuda(), b.dev, ints([0, 1]), enable_gqa=True, workspace=ws[:100])
    with pytest.raises(ValueError, match="no backward"):
        bsmt.paged_attention(q.cuda().requires_grad_(), b.dev, ints([0, 1]), enable_gqa=True)
    with pytest.raises(RuntimeError, match="UNSUPPORTED"):
        bsmt.paged_attention(q.cuda(), b.dev, ints([0, 1]), None, bsmt.document(ints([0, 0])), enable_gqa=True)
    with pytest.raises(ValueError, match="enable_gqa"):
        bsmt.paged_attention(q.cuda(), b.dev, ints([0, 1]))


def test_two_streams_at_once():
    b = filled([5000, 777], 2, 128, 64, "e4m3")
    qs = [queries(2, 16, 128, seed=s).cuda() for s in range(2)]
    want = [bsmt.paged_attention(q, b.dev, ints([0, 1]), enable_gqa=True)[0] for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    seqs = ints([0, 1])
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(bsmt.paged_attention(qs[i], b.dev, seqs, enable_gqa=True)[0])
    torch.cuda.synchronize()
    for w, outs in zip(want, got):
        assert all(torch.equal(w, o) for o in outs)
