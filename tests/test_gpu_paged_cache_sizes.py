"""GPU: the paged cache at sizes where a block has many pieces of work: several
heads of a page, several tokens, many copies one after another. Bit for bit."""
import numpy as np
import pytest
import torch

import block_sparse_masked_tile_b200 as bsmt
from tests.serving_helpers import Both, ints, running

pytestmark = pytest.mark.gpu


# vectors a thread holds: 1 (16 x 64, 16 x 128), 2, 4, 8; two to all heads of k and v a block
@pytest.mark.parametrize("page, dim, heads, n, most, code", [
    (16, 64, 3, 700, 72, "e4m3"), (16, 128, 3, 700, 40, "int8"), (32, 128, 3, 700, 72, "e4m3"), (64, 64, 5, 700, 72, "int8"),
    (64, 128, 3, 600, 72, "e4m3"), (64, 128, 3, 600, 72, "int8"), (128, 128, 3, 400, 130, "e4m3"), (128, 128, 3, 400, 130, "int8")])
def test_long_writes_and_reads(page, dim, heads, n, most, code):
    rng = np.random.default_rng(page + dim)
    held, new = [int(x) for x in rng.integers(0, 40, n)], [int(x) for x in rng.integers(0, most, n)]
    wide = -(-(40 + most) // page)
    b = Both(sum(-(-(x + y) // page) for x, y in zip(held, new)) + 9, heads, dim, n, wide, page, 1, code, seed=page)
    order = [int(s) for s in rng.permutation(n)]
    b.add(order, [held[s] for s in order])
    b.equal()
    b.add(order[::-1], [new[s] for s in order[::-1]], spread=6.0)  # from the middle of pages on: scales rise, codes are rounded anew
    b.equal()
    # all of it back: the last block's tokens are fewer
    lens = [int(x) for x in b.ref.seq_lens]
    for some in (order, order[:n // 3]):
        cu = running([lens[s] for s in some])
        got = bsmt.cache_gather(b.dev, ints(some), None, cu[-1] + 3, ints(cu))
        want = [np.concatenate(x) for x in zip(*(b.ref.tokens(0, s, 0, lens[s]) for s in some))]
        for g, w in zip(got, want):
            assert np.array_equal(g[:cu[-1]].double().cpu().numpy(), w) and not g[cu[-1]:].any()
    # one token each, several tokens a block
    some = [s for s in order if lens[s]] * 5
    at = [int(rng.integers(0, lens[s])) for s in some]
    got = bsmt.cache_gather(b.dev, ints(some), ints(at), len(some))
    want = [np.concatenate(x) for x in zip(*(b.ref.tokens(0, s, t, t + 1) for s, t in zip(some, at)))]
    for g, w in zip(got, want):
        assert np.array_equal(g.double().cpu().numpy(), w)
    bsmt.check_device_status()


# a block's copies: two for each page and layer of 3 heads (16 and 8 KB), or one of 1 KB; ten and more a block
@pytest.mark.parametrize("page, dim, heads, layers, pages, code", [(64, 128, 3, 2, 2600, "e4m3"), (16, 64, 1, 2, 9001, "int8"),
                                                                   (128, 128, 8, 1, 1500, "int8")])
def test_long_compactions(page, dim, heads, layers, pages, code):
    rng = np.random.default_rng(pages)
    wide, seqs = 7, pages // 14  # half of the pool
    c = bsmt.create_paged_cache(pages, heads, dim, seqs + 40, wide, page, layers,
                                torch.float8_e4m3fn if code == "e4m3" else torch.int8)
    gen = torch.Generator(device="cuda").manual_seed(pages)
    k, v = c.k.view(torch.int8), c.v.view(torch.int8)
    for x in (k, v):
        x.copy_(torch.randint(-128, 128, x.shape, generator=gen, device="cuda", dtype=torch.int8))
    for x in (c.k_scale, c.v_scale):
        x.copy_(torch.ldexp(torch.ones_like(x), torch.randint(-20, 20, x.shape, generator=gen, device="cuda")))
    table, lens = np.full((seqs + 40, wide), -1, np.int32), np.zeros(seqs + 40, np.int32)
    held = rng.permutation(pages)[:seqs * wide].reshape(seqs, wide)
    slots = rng.permutation(seqs + 40)
    table[slots[:seqs]], lens[slots[:seqs]] = held, wide * page
    table[slots[seqs:seqs + 30], :4], lens[slots[seqs:seqs + 30]] = held[:30, :4], 4 * page  # shared pages
    refs = np.bincount(table[table >= 0], minlength=pages).astype(np.int32)
    for t, x in ((c.page_table, table), (c.seq_lens, lens), (c.ref_counts, refs)):
        t.copy_(torch.from_numpy(x))
    live = int((refs > 0).sum())
    holes, movers = np.flatnonzero(refs[:live] == 0), live + np.flatnonzero(refs[live:] > 0)
    assert len(movers) * layers * 2 * -(-heads * page * dim // 16384) >= 10 * 3 * 148
    source = np.arange(pages)
    source[holes] = movers
    to = np.arange(pages, dtype=np.int32)
    to[movers] = holes
    want = [x[:, torch.from_numpy(source[:live]).cuda()].clone() for x in (k, v, c.k_scale, c.v_scale)]
    assert bsmt.cache_compact(c).item() == live
    bsmt.check_device_status()
    for x, w in zip((k, v, c.k_scale, c.v_scale), want):
        assert torch.equal(x[:, :live], w)
    assert np.array_equal(c.page_table.cpu().numpy(), np.where(table >= 0, to[table], -1))
    moved = refs.copy()
    moved[holes], moved[movers] = refs[movers], 0
    assert np.array_equal(c.ref_counts.cpu().numpy(), moved) and np.array_equal(c.seq_lens.cpu().numpy(), lens)
