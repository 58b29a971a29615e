"""Pins of the serving oracle (CPU): closed forms and library routines."""
import numpy as np
import pytest
import torch

from oracle import attention as oa
from oracle import serving as osv


def test_rotary_is_a_complex_turn_and_inverts():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((7, 3, 8))
    pos = rng.integers(-50, 50, (2, 7))
    freq, axis = [1.0, 0.3, 0.1, 0.01], [0, 1, 1, 0]
    for inter in (False, True):
        y = osv.rotary(x, pos, freq, axis, inter)
        for i in range(4):
            a, b = (2 * i, 2 * i + 1) if inter else (i, i + 4)
            z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * pos[axis[i]] * freq[i])[:, None]
            assert np.allclose(y[..., a], z.real) and np.allclose(y[..., b], z.imag)
        assert np.allclose(osv.rotary(y, pos, freq, axis, inter, inverse=True), x)
    # scores depend on the distance of two positions alone
    q, k = rng.standard_normal((1, 1, 8)), rng.standard_normal((1, 1, 8))
    dots = [np.sum(osv.rotary(q, [[p + 5]], [1.0, 0.3, 0.1, 0.01], [0] * 4) * osv.rotary(k, [[p]], [1.0, 0.3, 0.1, 0.01], [0] * 4))
            for p in (0, 9, 100)]
    assert np.allclose(dots, dots[0])


def test_encode_equals_torch_and_scales_are_the_smallest():
    x = np.concatenate([np.linspace(-460, 460, 4001), 2.0 ** np.arange(-14, 9), [0.0, np.inf, -np.inf]])
    want = torch.tensor(x).float().clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(osv.encode(x, "e4m3"), want)
    assert np.isnan(osv.encode(np.array([np.nan]), "e4m3")[0]) and osv.encode(np.array([np.nan]), "int8")[0] == 0
    assert np.array_equal(osv.encode(np.array([0.5, 1.5, 2.5, -200.0]), "int8"), [0, 2, 2, -127])
    for code, top in osv.TOP.items():
        for e in (-20, 0, 13):
            assert osv.scale_for(top * 2.0 ** e, code) == 2.0 ** e
            assert osv.scale_for(top * 2.0 ** e * (1 + 2.0 ** -40), code) == 2.0 ** (e + 1)
    assert osv.scale_for(0.0, "int8") == 2.0 ** osv.MIN_EXP


def make(code="e4m3"):
    return osv.Cache(2, 12, 2, 4, 8, 5, 6, code)


def fill(c, seq, n, seed):
    rng = np.random.default_rng(seed)
    k, v = rng.standard_normal((2, n, 2, 8))
    starts = c.extend([seq], [n])
    for layer in range(2):
        c.write(layer, [seq], starts, k, v, [0, n])
    return k, v


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_cache_holds_what_was_written(code):
    c = make(code)
    k, v = fill(c, 3, 10, 1)
    gk, gv = c.tokens(1, 3, 0, 10)
    # half a step of the code at its largest value: 2^-4 of it (e4m3), half a code (int8)
    bound = np.abs(k).max() * (2.0 ** -4 if code == "e4m3" else 1 / 127)
    assert np.abs(gk - k).max() <= bound and np.abs(gv - v).max() <= np.abs(v).max() * bound / np.abs(k).max()
    assert list(c.page_table[3, :3]) == [0, 1, 2] and c.ref_counts.sum() == 3


def test_fork_free_compact_keep_every_sequence():
    c = make()
    fill(c, 0, 10, 1)
    fill(c, 1, 7, 2)
    before = [c.tokens(1, s, 0, n) for s, n in ((0, 10), (1, 7))]
    c.fork([1, 1, 0], [2, 3, 4])
    assert list(c.ref_counts) == [2, 2, 1, 3, 1, 1, 1, 1, 0, 0, 0, 0]
    c.free([0, 1])
    assert c.compact() == 7 - 1
    assert list(c.ref_counts > 0) == [True] * 6 + [False] * 6
    for s, want in ((4, before[0]), (2, before[1]), (3, before[1])):
        for got, w in zip(c.tokens(1, s, 0, int(c.seq_lens[s])), want):
            assert np.array_equal(got, w)
    with pytest.raises(osv.Full):
        c.extend([0], [25])


def test_paged_attention_equals_flex_attention_on_the_gathered_cache():
    c = make()
    fill(c, 0, 10, 1)
    fill(c, 2, 1, 4)
    q = np.random.default_rng(5).standard_normal((4, 4, 8))
    tree = ("and", ("causal",), ("or", ("sink", 1), ("window", 3)))
    mods = (("softcap", 5.0), ("alibi", None))
    out, lse = osv.paged_attention(q, c, [0, 2], [0, 3, 4], tree, mods, layer=1)
    for s, rows in ((0, slice(0, 3)), (2, slice(3, 4))):
        n = int(c.seq_lens[s])
        k, v = (x.transpose(1, 0, 2)[None] for x in c.tokens(1, s, 0, n))
        m = rows.stop - rows.start
        full = np.zeros((1, 4, n, 8))
        full[0, :, n - m:] = q[rows].transpose(1, 0, 2)
        o, ls = oa.flex_attention(full, k, v, tree, mods, None, True)
        assert np.allclose(out[rows], o[0, :, n - m:].transpose(1, 0, 2), atol=1e-12)
        assert np.allclose(lse[:, rows], ls[0, :, n - m:], atol=1e-12)
