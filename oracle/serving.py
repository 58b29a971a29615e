"""Rotary positions, the 8-bit paged cache and attention over it in fp64 (test
infrastructure only), written from the definitions with plain loops.

* ``rotary`` turns each pair of a head by position times frequency.
* ``Cache`` is a model of the paged cache: codes are held as the numbers they
  stand for, and each page operation is the loop that its description says.
* ``paged_attention`` materialises each query row's scores over its sequence's
  dequantised keys, through ``masks`` and ``attention.apply_score_mods``.
"""
from __future__ import annotations

import numpy as np

from . import attention, masks

TOP = {"e4m3": 448.0, "int8": 127.0}
MIN_EXP = -120


def rotary(x, positions, inv_freq, axis, interleaved=False, inverse=False) -> np.ndarray:
    """x [..., T, H, D] (heads behind tokens), positions [axes, ..., T]."""
    y = np.array(x, dtype=np.float64)
    n = len(inv_freq)
    for i in range(n):
        t = np.asarray(positions[axis[i]], dtype=np.float64)[..., None] * inv_freq[i]
        if inverse:
            t = -t
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        a, b = x[..., ia], x[..., ib]
        y[..., ia] = a * np.cos(t) - b * np.sin(t)
        y[..., ib] = a * np.sin(t) + b * np.cos(t)
    return y


def scale_for(largest: float, code: str) -> float:
    """The smallest 2^e, e >= MIN_EXP, with largest <= top * 2^e."""
    e = MIN_EXP
    if largest > 0:
        e = max(e, int(np.floor(np.log2(largest / TOP[code]))) - 1)
        while largest > TOP[code] * 2.0 ** e:
            e += 1
    return 2.0 ** e


def encode(x: np.ndarray, code: str) -> np.ndarray:
    """Values in units of the scale -> the numbers of their codes: nearest, ties
    to even, saturating; NaN stays (e4m3) or is 0 (int8)."""
    with np.errstate(invalid="ignore"):
        if code == "int8":
            return np.nan_to_num(np.clip(np.rint(x), -127, 127), nan=0.0)
        mag = np.where(np.isfinite(x), np.abs(x), 1.0)
        step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(mag, 2.0 ** -40))), -6) - 3)
        return np.clip(np.where(np.isfinite(x), np.rint(x / step) * step, x), -448.0, 448.0)


class Full(Exception):
    """A refused extend or fork."""


class Cache:
    def __init__(self, layers, pages, heads, page, dim, seqs, wide, code):
        self.code, self.page = code, page
        self.k, self.v = (np.zeros((layers, pages, heads, page, dim)) for _ in range(2))
        self.k_scale, self.v_scale = (np.zeros((layers, pages, heads)) for _ in range(2))
        self.page_table = np.full((seqs, wide), -1, np.int32)
        self.seq_lens = np.zeros(seqs, np.int32)
        self.ref_counts = np.zeros(pages, np.int32)

    def pages_of(self, tokens: int) -> int:
        return -(-int(tokens) // self.page)

    def free_pages(self, n: int) -> list:
        found = [int(p) for p in np.flatnonzero(self.ref_counts == 0)[:n]]
        if len(found) < n:
            raise Full
        return found

    def extend(self, seqs, counts) -> list:
        need = sum(self.pages_of(self.seq_lens[s] + c) - self.pages_of(self.seq_lens[s]) for s, c in zip(seqs, counts) if s >= 0)
        got = iter(self.free_pages(need))
        starts = []
        for s, c in zip(seqs, counts):
            if s < 0:
                starts.append(-1)
                continue
            have = int(self.seq_lens[s])
            for at in range(self.pages_of(have), self.pages_of(have + c)):
                page = next(got)
                self.page_table[s, at] = page
                self.ref_counts[page] = 1
            self.seq_lens[s] = have + c
            starts.append(have)
        return starts

    def write(self, layer, seqs, starts, k, v, cu):
        for i, (s, start) in enumerate(zip(seqs, starts)):
            if s < 0 or start < 0:
                continue
            for at in range(start // self.page, self.pages_of(start + cu[i + 1] - cu[i])):
                lo, hi = max(start, at * self.page), min(start + cu[i + 1] - cu[i], (at + 1) * self.page)
                if lo >= hi:
                    continue
                page, row = self.page_table[s, at], lo % self.page
                for codes, scales, x in ((self.k, self.k_scale, k), (self.v, self.v_scale, v)):
                    for h in range(codes.shape[2]):
                        new = np.asarray(x[cu[i] + lo - start:cu[i] + hi - start, h], np.float64)
                        fine = np.abs(new[np.isfinite(new)])
                        scale = scale_for(fine.max(initial=0.0), self.code)
                        if row > 0:
                            held = scales[layer, page, h]
                            scale = max(scale, held)
                            codes[layer, page, h, :row] = encode(codes[layer, page, h, :row] * (held / scale), self.code)
                        codes[layer, page, h, row:row + hi - lo] = encode(new / scale, self.code)
                        scales[layer, page, h] = scale

    def tokens(self, layer, seq, lo, hi):
        """(k, v) [hi - lo, Hkv, D] of positions lo .. hi of a sequence, dequantised."""
        got = []
        for codes, scales in ((self.k, self.k_scale), (self.v, self.v_scale)):
            pages, rows = self.page_table[seq][np.arange(lo, hi) // self.page], np.arange(lo, hi) % self.page
            got.append(codes[layer, pages, :, rows] * scales[layer, pages][..., None])
        return got

    def fork(self, src, dst):
        parts = [s for s, d in zip(src, dst) if s >= 0 and d >= 0 and self.seq_lens[s] % self.page]
        got = iter(self.free_pages(len(parts)))
        lens = self.seq_lens.copy()
        for s, d in zip(src, dst):
            if s < 0 or d < 0:
                continue
            n = int(lens[s])
            self.seq_lens[d] = n
            for at in range(n // self.page):
                self.page_table[d, at] = self.page_table[s, at]
                self.ref_counts[self.page_table[s, at]] += 1
            if n % self.page:
                old, page = self.page_table[s, n // self.page], next(got)
                self.page_table[d, n // self.page] = page
                self.ref_counts[page] = 1
                for x in (self.k, self.v):
                    x[:, page, :, :n % self.page] = x[:, old, :, :n % self.page]
                for x in (self.k_scale, self.v_scale):
                    x[:, page] = x[:, old]

    def free(self, seqs):
        for s in seqs:
            if s < 0:
                continue
            for at in range(self.pages_of(self.seq_lens[s])):
                self.ref_counts[self.page_table[s, at]] -= 1
                self.page_table[s, at] = -1
            self.seq_lens[s] = 0

    def compact(self) -> int:
        live = int((self.ref_counts > 0).sum())
        holes = [p for p in range(live) if self.ref_counts[p] == 0]
        movers = [p for p in range(live, len(self.ref_counts)) if self.ref_counts[p] > 0]
        for to, page in zip(holes, movers):
            for x in (self.k, self.v, self.k_scale, self.v_scale):
                x[:, to] = x[:, page]
            self.page_table[self.page_table == page] = to
            self.ref_counts[to], self.ref_counts[page] = self.ref_counts[page], 0
        return live


def paged_attention(q, cache: Cache, seqs, cu, tree, mods, scale=None, layer=0):
    """q [T, Hq, D] -> (out [T, Hq, D], lse [Hq, T])."""
    q = np.asarray(q, np.float64)
    T, Hq, D = q.shape
    out, lse = np.zeros((T, Hq, D)), np.full((Hq, T), -np.inf)
    scale = D ** -0.5 if scale is None else scale
    for i, s in enumerate(seqs):
        if s < 0:
            continue
        n, m = int(cache.seq_lens[s]), cu[i + 1] - cu[i]
        k, v = cache.tokens(layer, s, 0, n)
        group = Hq // cache.k.shape[2]
        at, keys = np.arange(n - m, n), np.arange(n)
        for h in range(Hq):
            S = scale * (q[cu[i]:cu[i + 1], h] @ k[:, h // group].T)
            S = attention.apply_score_mods(S, mods, h, Hq, at, keys)
            see = masks.evaluate(tree or ("noop",), 0, at[:, None], keys[None])
            for r in range(m):
                row, vv = S[r, see[r]], v[see[r], h // group]
                if not len(row):
                    continue
                top = row.max()
                p = np.exp(row - top)
                lse[h, cu[i] + r] = top + np.log(p.sum())
                out[cu[i] + r, h] = (p / p.sum()) @ vv
    return out, lse
