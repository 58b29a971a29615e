"""Shared helpers of the serving tests: a device cache beside its fp64 model."""
import numpy as np
import torch

import block_sparse_masked_tile_b200 as bsmt
from oracle import serving as osv

CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def ints(values):
    return torch.tensor(list(values), dtype=torch.int32, device="cuda")


def running(counts):
    return [0] + [int(x) for x in np.cumsum(counts)]


class Both:
    """The same calls on a device cache and on its model; equal() compares all of both."""

    def __init__(self, pages, heads, dim, seqs, wide, page=16, layers=1, code="e4m3", seed=0):
        self.dev = bsmt.create_paged_cache(pages, heads, dim, seqs, wide, page, layers, CODES[code])
        self.ref = osv.Cache(layers, pages, heads, page, dim, seqs, wide, code)
        self.gen = torch.Generator().manual_seed(seed)
        self.heads, self.dim, self.layers = heads, dim, layers

    def values(self, T, spread=1.0):
        """bf16 [T, Hkv, D] whose rows differ in magnitude by up to 2^spread either way."""
        x = torch.randn((T, self.heads, self.dim), generator=self.gen)
        x = x * 2.0 ** (spread * (2 * torch.rand((T, self.heads, 1), generator=self.gen) - 1))
        return x.bfloat16()

    def extend(self, seqs, counts):
        got = bsmt.cache_extend(self.dev, ints(seqs), ints(counts))
        want = self.ref.extend(seqs, counts)
        assert got.tolist() == want
        return want

    def write(self, layer, seqs, starts, k, v, counts):
        cu = running(counts)
        one = all(c == 1 for c in counts)
        bsmt.cache_write(self.dev, ints(seqs), ints(starts), k.cuda(), v.cuda(), None if one else ints(cu), layer)
        self.ref.write(layer, seqs, starts, k.double().numpy(), v.double().numpy(), cu)

    def add(self, seqs, counts, spread=1.0):
        """Extend, and write random values in every layer."""
        starts = self.extend(seqs, counts)
        for layer in range(self.layers):
            self.write(layer, seqs, starts, self.values(sum(counts), spread), self.values(sum(counts), spread), counts)

    def fork(self, src, dst):
        bsmt.cache_fork(self.dev, ints(src), ints(dst))
        self.ref.fork(src, dst)

    def free(self, seqs):
        bsmt.cache_free(self.dev, ints(seqs))
        self.ref.free(seqs)

    def compact(self):
        assert bsmt.cache_compact(self.dev).tolist() == [self.ref.compact()]

    def equal(self, codes=True):
        bsmt.check_device_status()
        d, r = self.dev, self.ref
        for name in ("page_table", "seq_lens", "ref_counts"):
            assert np.array_equal(getattr(d, name).cpu().numpy(), getattr(r, name)), name
        if not codes:
            return
        rows = np.zeros(r.k.shape[1:2] + r.k.shape[3:4], bool)  # rows that hold tokens
        for s, n in enumerate(r.seq_lens):
            at = np.arange(n)
            rows[r.page_table[s, at // r.page], at % r.page] = True
        used = np.where(rows.any(1))[0]
        for name in ("k", "v"):
            got = getattr(d, name).float().cpu().numpy().transpose(0, 2, 1, 3, 4)[:, :, rows]
            assert np.array_equal(got, getattr(r, name).transpose(0, 2, 1, 3, 4)[:, :, rows], equal_nan=True), name
            got = getattr(d, name + "_scale").cpu().numpy()[:, used]
            assert np.array_equal(got, getattr(r, name + "_scale")[:, used]), name + "_scale"

    def attend(self, q, seqs, counts, tree, mods=(), layer=0, scale=None, **more):
        """paged_attention on the device against the model; q [T, Hq, D] on the host, T at least sum(counts)."""
        cu = running(counts)
        one = all(c == 1 for c in counts) and q.shape[0] == len(counts)
        mask = None if tree is None else bsmt.mask_from_tree(tree)
        out, lse = bsmt.paged_attention(q.cuda(), self.dev, ints(seqs), None if one else ints(cu), mask,
                                        bsmt.score_mods_from_list(mods), scale, True, layer, **more)
        bsmt.check_device_status()
        want, want_lse = osv.paged_attention(q.double().numpy(), self.ref, seqs, cu, tree, mods, scale, layer)
        self.close(out, lse, want, want_lse, q, layer, scale)
        return out, lse

    def close(self, out, lse, want, want_lse, q, layer=0, scale=None):
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        n = max(1, int(self.ref.seq_lens.max()))
        # out: bf16's rounding (2^-8 of the value); P in halves (2^-11 of each normal term, 2^-25 of the largest
        # for the others), exp2 and fp32 sums (2^-14 in all), each against the largest |v| that the scales allow.
        top = osv.TOP[self.ref.code] * self.ref.v_scale[layer].max()
        tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + n * 2.0 ** -25 + 2.0 ** -14) * top
        bad = ~(np.abs(out - want) <= tol) & ~(np.isnan(out) & np.isnan(want))
        assert not bad.any(), (np.argwhere(bad)[:4], out[bad][:4], want[bad][:4])
        # lse: a score is a sum of D products in fp32, each addition off by 2^-23 of the sum of magnitudes at most,
        # and 2^-20 of that sum for the scaling, the modifiers and the sum of exponentials
        fine = np.isfinite(want_lse)
        assert np.array_equal(np.isneginf(lse), np.isneginf(want_lse))
        assert np.array_equal(np.isnan(lse), np.isnan(want_lse))
        k_top = osv.TOP[self.ref.code] * self.ref.k_scale[layer].max()
        mass = np.nanmax(np.abs(q.double().numpy()).sum(-1)) * k_top * (q.shape[-1] ** -0.5 if scale is None else scale)
        assert np.abs(lse[fine] - want_lse[fine]).max(initial=0.0) <= (q.shape[-1] * 2.0 ** -23 + 2.0 ** -20) * mass + 2e-6 * np.abs(want_lse[fine]).max(initial=0.0)


def queries(T, Hq, D, seed=1):
    return torch.randn((T, Hq, D), generator=torch.Generator().manual_seed(seed)).bfloat16()
