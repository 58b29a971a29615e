"""GPU: attention over the paged cache where its work list, its modifiers or its
arguments are at an edge, against the fp64 oracle."""
import numpy as np
import pytest
import torch

import block_sparse_masked_tile_b200 as bsmt
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
