"""GPU: the paged cache against its model, bit for bit: quantised writes, reads
back, page bookkeeping and refusals that only the device can see."""
import numpy as np
import pytest
import torch

import block_sparse_masked_tile_b200 as bsmt
from oracle import serving as osv
from tests.serving_helpers import Both, ints, running

pytestmark = pytest.mark.gpu


def raises(status):
    with pytest.raises(RuntimeError, match=status):
        bsmt.check_device_status()
    bsmt.check_device_status()  # it was cleared


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("page, dim, heads", [(16, 128, 1), (32, 64, 3), (64, 128, 2), (128, 64, 2), (128, 128, 1)])
def test_writes(code, page, dim, heads):
    b = Both(40, heads, dim, 6, 20, page, 2, code, seed=page)
    b.add([0], [1])
    b.equal()
    b.add([3, 0, 5], [page - 1, page, 2 * page + 3])        # to a page's edge, past it, over whole pages
    b.equal()
    b.add([5, 3, 0, 1], [1, 1, 1, 1], spread=6.0)           # one token each: scales rise, held codes are rounded anew
    b.equal()
    b.add([1, 2, 5, 0], [0, 5, 1, 0], spread=6.0)           # none for some
    b.equal()
    b.add([-1, 2], [0, page + 1])                           # an entry passed over
    b.equal()
    for _ in range(6):
        b.add([5, 1, 2], [1, 1, 1], spread=10.0)
    b.equal()


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_writes_of_special_values(code):
    b = Both(8, 2, 64, 2, 4, 16, 1, code)
    k = torch.zeros((6, 2, 64)).bfloat16()
    v = k.clone()
    k[1, 0, :4] = torch.tensor([448.0, -448.0, 449.0, 2.0 ** -9])
    k[2, 1, 0] = 3.0e38
    k[3, 0, 5], k[4, 0, 6] = float("inf"), float("-inf")
    v[5, 1, :2] = torch.tensor([1e-38, 1e-40])                 # the smallest scale, and a subnormal
    v[0, 0] = torch.linspace(-2, 2, 64).bfloat16()
    for counts in ([6], [1] * 6):
        b = Both(8, 2, 64, 2, 4, 16, 1, code)
        at = 0
        for c in counts:
            starts = b.extend([1], [c])
            b.write(0, [1], starts, k[at:at + c], v[at:at + c], [c])
            at += c
        b.equal()
    # NaN: kept by e4m3, a reported 0 in int8; it takes no part in the scale
    k[0, 0, 0] = float("nan")
    b = Both(8, 2, 64, 2, 4, 16, 1, code)
    starts = b.extend([0], [6])
    b.write(0, [0], starts, k, v, [6])
    if code == "int8":
        raises("PRECONDITION")
    b.equal()


def test_the_same_write_again_gives_the_same_cache():
    b = Both(20, 2, 128, 3, 8, 16, 1, "e4m3")
    b.add([0, 1], [5, 20])
    starts = b.extend([0, 1], [30, 1])
    k, v = b.values(31, 5.0), b.values(31, 5.0)
    for _ in range(3):
        b.write(0, [0, 1], starts, k, v, [30, 1])
        b.equal()


def test_strided_sources_and_rows_behind_the_pack():
    b = Both(20, 2, 64, 3, 8, 16, 1, "int8")
    fused = torch.randn((40, 8, 72), generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    k, v = fused[:, 1:3, 8:], fused[:, 4:8:2, :64]
    starts = b.extend([2, 0], [17, 9])
    cu = running([17, 9])
    bsmt.cache_write(b.dev, ints([2, 0]), ints(starts), k, v, ints(cu))  # 14 rows more than the pack has
    b.ref.write(0, [2, 0], starts, k.double().cpu().numpy(), v.double().cpu().numpy(), cu)
    b.equal()
    for bad in (fused[:, 1:3, 4:68], fused[:, 1:3, ::1].transpose(1, 2)[:, :64].transpose(1, 2)[..., :63]):
        with pytest.raises(ValueError):
            bsmt.cache_write(b.dev, ints([2, 0]), ints(starts), bad, bad, ints(cu))


@pytest.mark.parametrize("code, page, dim", [("e4m3", 16, 64), ("int8", 64, 128)])
def test_gather(code, page, dim):
    b = Both(60, 3, dim, 4, 20, page, 2, code)
    b.add([2, 0, 1], [3 * page + 5, 1, 40], spread=4.0)
    seqs, starts, counts = [1, 2, -1, 0, 2], [7, 0, 0, 0, page], [20, 3 * page + 5, 3, 1, 0]
    cu = running(counts)
    total = cu[-1] + 4  # rows behind the pack
    k, v = bsmt.cache_gather(b.dev, ints(seqs), ints(starts), total, ints(cu), layer=1)
    b.equal()
    for i, (s, st, n) in enumerate(zip(seqs, starts, counts)):
        want = b.ref.tokens(1, s, st, st + n) if s >= 0 else (np.zeros((n, 3, dim)),) * 2
        for got, w in zip((k, v), want):
            assert np.array_equal(got[cu[i]:cu[i + 1]].double().cpu().numpy(), w)
    assert not k[cu[-1]:].any() and not v[cu[-1]:].any()
    k, v = bsmt.cache_gather(b.dev, ints([0, 2]), ints([0, 5]), 2)  # one token each
    assert np.array_equal(v.double().cpu().numpy(), np.concatenate([b.ref.tokens(0, 0, 0, 1)[1], b.ref.tokens(0, 2, 5, 6)[1]]))
    k, v = bsmt.cache_gather(b.dev, ints([2]), None, 3 * page + 5, ints([0, 3 * page + 5]))  # from 0
    assert np.array_equal(k.double().cpu().numpy(), b.ref.tokens(0, 2, 0, 3 * page + 5)[0])
    # positions past the end are 0 and reported
    k, v = bsmt.cache_gather(b.dev, ints([0]), None, 3, ints([0, 3]))
    raises("BOUNDS")
    assert k[0].any() and not k[1:].any()
    assert bsmt.cache_gather(b.dev, ints([0]), None, 0, ints([0, 0]))[0].shape == (0, 3, dim)


def test_pages_by_random_calls():
    rng = np.random.default_rng(4)
    for code, page, layers in (("e4m3", 16, 3), ("int8", 32, 1)):
        b = Both(70, 2, 64, 9, 12, page, layers, code, seed=page)
        for _ in range(60):
            held = [s for s in range(9) if b.ref.seq_lens[s] > 0]
            empty = [s for s in range(9) if b.ref.seq_lens[s] == 0]
            what = rng.integers(5)
            if what <= 1:
                seqs = [int(s) for s in rng.permutation(9)[:rng.integers(1, 5)]]
                counts = [int(rng.integers(0, 2 * page)) for _ in seqs]
                room = all(b.ref.seq_lens[s] + c <= 12 * page for s, c in zip(seqs, counts))
                need = sum(b.ref.pages_of(b.ref.seq_lens[s] + c) - b.ref.pages_of(b.ref.seq_lens[s]) for s, c in zip(seqs, counts))
                if room and need <= (b.ref.ref_counts == 0).sum():
                    b.add(seqs, counts, spread=4.0)
            elif what == 2 and held and empty:
                dst = [int(s) for s in rng.permutation(empty)[:rng.integers(1, 4)]]
                src = [int(rng.choice(held)) for _ in dst]
                if len(dst) <= (b.ref.ref_counts == 0).sum():
                    b.fork([-1] + src, [empty[0]] + dst)
            elif what == 3 and held:
                gone = [int(s) for s in rng.permutation(held)[:2]]
                b.free([-1] + gone)
                bsmt.cache_free(b.dev, ints(gone + gone))  # again: nothing left to free
            else:
                b.compact()
            b.equal()


def test_large_pool_and_many_sequences():
    # more pages than one step of the pool scan (16384), more sequences than threads of the planner (1024)
    pages, seqs = 40000, 2500
    b = Both(pages, 1, 64, seqs, 40, 16, 1, "e4m3")
    rng = np.random.default_rng(0)
    order = [int(s) for s in rng.permutation(seqs)]
    b.extend(order, [int(x) for x in rng.integers(0, 300, seqs)])
    b.equal(codes=False)
    b.free(order[::3])
    b.fork(order[1::3][:200], order[::3][:200])
    b.equal(codes=False)
    b.extend(order, [1] * seqs)
    b.equal(codes=False)
    b.free(order[:900])
    b.compact()
    b.equal(codes=False)
    b.extend(order[:1100], [int(x) for x in rng.integers(0, 200, 1100)])
    b.equal(codes=False)


def state(c):
    return [t.clone() for t in (c.page_table, c.seq_lens, c.ref_counts, c.k.view(torch.int8), c.v.view(torch.int8), c.k_scale)]


def test_refusals_change_nothing():
    b = Both(10, 2, 64, 6, 4, 16, 1, "e4m3")
    b.add([0, 1], [20, 33])
    c = b.dev
    before = state(c)

    def refused(status, call):
        got = call()
        raises(status)
        assert all(torch.equal(x, y) for x, y in zip(before, state(c)))
        return got

    for status, seqs, counts in (("CAPACITY", [2, 3], [64, 17]), ("CAPACITY", [1], [32]), ("PRECONDITION", [2, 2], [1, 1]),
                                 ("PRECONDITION", [2], [-1]), ("BOUNDS", [6], [1]), ("BOUNDS", [-2], [1]),
                                 ("CAPACITY", [2, 3, 4], [2 ** 31 - 1] * 3)):
        starts = refused(status, lambda: bsmt.cache_extend(c, ints(seqs), ints(counts)))
        assert starts.tolist() == [-1] * len(seqs)
        # the write of the same step then writes nothing
        x = torch.ones((len(seqs), 2, 64), dtype=torch.bfloat16, device="cuda")
        bsmt.cache_write(c, ints(seqs), starts, x, x)
        bsmt.check_device_status()
        assert all(torch.equal(x, y) for x, y in zip(before, state(c)))
    for status, src, dst in (("PRECONDITION", [0], [1]), ("PRECONDITION", [0, 1], [2, 2]), ("BOUNDS", [0], [6]),
                             ("BOUNDS", [-3], [2]), ("CAPACITY", [0] * 4 + [1] * 2, [2, 3, 4, 5, 0, 1])):
        if status == "CAPACITY":
            b.extend([2], [60])
            b.free([1])
            b.add([1], [33])
            b.extend([3], [16])
            before = state(c)
            src, dst = [0, 1], [4, 5]
        refused(status, lambda: bsmt.cache_fork(c, ints(src), ints(dst)))
    # freeing out of range is reported, the rest of the list is freed
    bsmt.cache_free(c, ints([9, 3, -7]))
    raises("BOUNDS")
    b.ref.free([3])
    b.equal(codes=False)


def test_writes_that_do_not_fit_are_left_out():
    b = Both(10, 2, 64, 4, 4, 16, 1, "int8")
    b.add([0], [20])
    b.fork([0], [1])
    c = b.dev
    before = state(c)
    x = torch.ones((1, 2, 64), dtype=torch.bfloat16, device="cuda")
    for status, seq, start in (("BOUNDS", 0, 20), ("BOUNDS", 0, -2), ("BOUNDS", 7, 0), ("PRECONDITION", 0, 3)):
        bsmt.cache_write(c, ints([seq]), ints([start]), x, x)  # past the end, no place, no sequence, a shared page
        raises(status)
    bsmt.cache_write(c, ints([-1]), ints([0]), x, x)
    bsmt.cache_write(c, ints([0]), ints([0]), x, x, ints([0, 0]))
    bsmt.check_device_status()
    for cu in ([1, 0], [-1, 1], [0, 2]):
        bsmt.cache_write(c, ints([0]), ints([19]), x, x, ints(cu))
        raises("PRECONDITION")
    assert all(torch.equal(x, y) for x, y in zip(before, state(c)))
    # a page number out of range in the table: reported by every call that reads it, and passed over
    c.page_table[0, 1] = 10
    bsmt.cache_write(c, ints([0]), ints([19]), x, x)
    raises("BOUNDS")
    k, _ = bsmt.cache_gather(c, ints([0]), None, 20, ints([0, 20]))
    raises("BOUNDS")
    assert k[:16].any() and not k[16:].any()
    bsmt.cache_extend(c, ints([0]))
    raises("BOUNDS")
    bsmt.cache_fork(c, ints([0]), ints([2]))
    raises("BOUNDS")
    bsmt.cache_free(c, ints([0]))
    raises("BOUNDS")
    assert c.seq_lens.tolist() == [0, 20, 0, 0]
    assert c.ref_counts.tolist() == [1, 1, 1] + [0] * 7  # the lost page keeps its count


def test_one_captured_step_serves_a_growing_batch():
    b = Both(40, 2, 64, 4, 8, 16, 1, "e4m3")
    b.add([0, 1, 2], [15, 1, 30])
    seqs, starts = ints([0, -1, 2, 1]), torch.empty(4, dtype=torch.int32, device="cuda")
    ws = torch.empty(bsmt.cache_workspace_bytes(b.dev, 4), dtype=torch.uint8, device="cuda")
    k, v = (torch.empty((4, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bsmt.cache_extend(b.dev, seqs, None, starts, ws)
        bsmt.cache_write(b.dev, seqs, starts, k, v)
    for step in range(20):
        nk, nv = b.values(4, 4.0), b.values(4, 4.0)
        k.copy_(nk)
        v.copy_(nv)
        if step == 10:
            seqs.copy_(ints([3, 0, -1, 1]))
        g.replay()
        now = seqs.tolist()
        want = b.ref.extend(now, [1] * 4)
        assert starts.tolist() == want
        b.ref.write(0, now, want, nk.double().numpy(), nv.double().numpy(), range(5))
        b.equal()


def test_work_on_a_side_stream_is_ordered_there():
    b = Both(60, 2, 128, 4, 30, 16, 1, "e4m3")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        for _ in range(5):
            b.add([0, 1], [9, 30], spread=3.0)
        side.synchronize()
        b.equal()


def test_pool_past_four_gigabytes():
    # pages whose bytes lie past 2^32: codes of 5 GB
    P, D, heads = 128, 128, 8
    pages = (5 << 30) // (P * D * heads)
    c = bsmt.PagedCache(*(torch.empty((1, pages, heads, P, D), dtype=torch.int8, device="cuda") for _ in range(2)),
                        *(torch.zeros((1, pages, heads), device="cuda") for _ in range(2)),
                        torch.full((4, 3), -1, dtype=torch.int32, device="cuda"),
                        torch.zeros(4, dtype=torch.int32, device="cuda"), torch.ones(pages, dtype=torch.int32, device="cuda"))
    c.ref_counts[-5:] = 0
    starts = bsmt.cache_extend(c, ints([2]), ints([200]))
    assert c.page_table[2, :2].tolist() == [pages - 5, pages - 4]
    k = torch.randn((200, heads, D), generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    bsmt.cache_write(c, ints([2]), starts, k, -k, ints([0, 200]))
    bsmt.cache_fork(c, ints([2, 2]), ints([0, 1]))
    q = torch.randn((3, 16, D), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    outs = bsmt.paged_attention(q[:1].expand(3, -1, -1).contiguous(), c, ints([2, 0, 1]), enable_gqa=True)[0]
    gk, gv = bsmt.cache_gather(c, ints([1]), None, 200, ints([0, 200]))
    bsmt.check_device_status()
    # Equal sequences, but cut into shares at different places: each row is within 2^-8 of its value (bf16's rounding)
    # and (2^-11 + 200 * 2^-25 + 2^-14) of the largest |v| = 4.5 (P in halves, exp2 and fp32 sums) of the exact one.
    for other in outs[1:]:
        bound = 2 * (2.0 ** -8 * outs[0].float().abs() + (2.0 ** -11 + 200 * 2.0 ** -25 + 2.0 ** -14) * float(k.abs().max()))
        assert ((outs[0].float() - other.float()).abs() <= bound).all()
    assert torch.equal(gk, -gv)
    ref = osv.Cache(1, 3, heads, P, D, 1, 3, "int8")
    ref.write(0, [0], ref.extend([0], [200]), k.double().cpu().numpy(), -k.double().cpu().numpy(), [0, 200])
    assert np.array_equal(gk.double().cpu().numpy(), ref.tokens(0, 0, 0, 200)[0])
    c.ref_counts[:-5] = 0
    assert bsmt.cache_compact(c).item() == 4
    assert sorted(c.page_table[c.page_table >= 0].unique().tolist()) == [0, 1, 2, 3]
    again = bsmt.paged_attention(q[:1].expand(3, -1, -1).contiguous(), c, ints([2, 0, 1]), enable_gqa=True)[0]
    bsmt.check_device_status()
    assert torch.equal(again, outs)
