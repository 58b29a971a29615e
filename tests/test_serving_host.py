"""Host-only checks of the serving entry points: argument errors of the C ABI
and of the binding. Nothing here reaches a CUDA call."""
import ctypes
import math

import pytest
import torch

import block_sparse_masked_tile_b200 as bsmt
from block_sparse_masked_tile_b200 import _lib, _MaskSpec, _ScoreSpec
from block_sparse_masked_tile_b200 import serving as sv

OK, INVALID, SHAPE, UNSUPPORTED = 0, 1, 2, 3
FAKE = 0x10000  # 256-byte aligned, never dereferenced by these calls
BIG = 1 << 40


def cache_struct(**changes):
    c = sv._KvCache(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 2, 100, 4, 64, 128, 8, 10, 0)
    for k, v in changes.items():
        setattr(c, k, v)
    return c


def strides(*s):
    return (ctypes.c_int64 * len(s))(*s)


def test_header_declares_what_the_binding_calls():
    import os
    import re
    text = open(os.path.join(os.path.dirname(__file__), "..", "include", "bsmt_serving.h")).read()
    names = sorted(set(re.findall(r"^bsmt_status\s+(bsmt_\w+)\s*\(", text, re.M)))
    assert names == ["bsmt_cache_compact", "bsmt_cache_extend", "bsmt_cache_fork", "bsmt_cache_free", "bsmt_cache_gather",
                     "bsmt_cache_workspace_bytes", "bsmt_cache_write", "bsmt_paged_attention",
                     "bsmt_paged_attention_workspace_bytes", "bsmt_rotary", "bsmt_rotary_sections"]
    for n in names:
        assert hasattr(_lib, n), n


# every call of a cache checks it the same way
@pytest.mark.parametrize("change, status", [
    (dict(head_dim=96), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED), (dict(page_size=256), UNSUPPORTED),
    (dict(dtype=2), UNSUPPORTED), (dict(num_layers=0), INVALID), (dict(num_pages=0), INVALID),
    (dict(num_kv_heads=0), INVALID), (dict(max_seqs=0), INVALID), (dict(max_pages=0), INVALID),
    (dict(max_seqs=(1 << 18) + 1), UNSUPPORTED), (dict(max_pages=1 << 25), UNSUPPORTED), (dict(k=None), INVALID),
    (dict(v=FAKE + 8), INVALID), (dict(ref_counts=FAKE + 4), INVALID), (dict(page_table=FAKE + 2), INVALID),
    (dict(num_kv_heads=70000), UNSUPPORTED), (dict(seq_lens=None), INVALID), (dict(k_scale=FAKE + 1), INVALID),
])
def test_cache_checks(change, status):
    c = ctypes.byref(cache_struct(**change))
    st = strides(512, 128)
    assert _lib.bsmt_cache_write(c, 0, FAKE, FAKE, 1, None, FAKE, FAKE, 1, st, st, None) == status
    assert _lib.bsmt_cache_gather(c, 0, FAKE, FAKE, 1, None, 1, FAKE, FAKE, None) == status
    assert _lib.bsmt_cache_extend(c, FAKE, None, 1, FAKE, FAKE, BIG, None) == status
    assert _lib.bsmt_cache_fork(c, FAKE, FAKE, 1, FAKE, BIG, None) == status
    assert _lib.bsmt_cache_free(c, FAKE, 1, None) == status
    assert _lib.bsmt_cache_compact(c, FAKE, FAKE, BIG, None) == status
    assert _lib.bsmt_paged_attention(FAKE, 1, 8, c, 0, FAKE, 1, None, None, None, 0.0, 1, FAKE, FAKE, FAKE, BIG, None) == status


def test_null_cache_and_lists():
    st = strides(512, 128)
    assert _lib.bsmt_cache_free(None, FAKE, 1, None) == INVALID
    c = ctypes.byref(cache_struct())
    for layer in (-1, 2):
        assert _lib.bsmt_cache_write(c, layer, FAKE, FAKE, 1, None, FAKE, FAKE, 1, st, st, None) == INVALID
        assert _lib.bsmt_cache_gather(c, layer, FAKE, None, 1, None, 1, FAKE, FAKE, None) == INVALID
    for args in ((None, FAKE, 1, None, FAKE, FAKE, 1, st, st), (FAKE, None, 1, None, FAKE, FAKE, 1, st, st),
                 (FAKE + 2, FAKE, 1, None, FAKE, FAKE, 1, st, st), (FAKE, FAKE, -1, None, FAKE, FAKE, -1, st, st),
                 (FAKE, FAKE, 1, None, None, FAKE, 1, st, st), (FAKE, FAKE, 1, None, FAKE, FAKE + 8, 1, st, st),
                 (FAKE, FAKE, 2, None, FAKE, FAKE, 2, strides(516, 128), st),
                 (FAKE, FAKE, 2, None, FAKE, FAKE, 2, st, strides(-512, 128)),
                 (FAKE, FAKE, 1, None, FAKE, FAKE, 1, strides(512, 100), st), (FAKE, FAKE, 1, FAKE + 1, FAKE, FAKE, 9, st, st)):
        assert _lib.bsmt_cache_write(c, 0, *args, None) == INVALID, args
    # without offsets there is one token for each sequence
    assert _lib.bsmt_cache_write(c, 0, FAKE, FAKE, 2, None, FAKE, FAKE, 3, st, st, None) == SHAPE
    assert _lib.bsmt_cache_gather(c, 0, FAKE, FAKE, 2, None, 1, FAKE, FAKE, None) == SHAPE
    assert _lib.bsmt_paged_attention(FAKE, 3, 8, c, 0, FAKE, 2, None, None, None, 0.0, 1, FAKE, FAKE, FAKE, BIG, None) == SHAPE
    assert _lib.bsmt_cache_extend(c, FAKE, FAKE, 1, None, FAKE, BIG, None) == INVALID
    assert _lib.bsmt_cache_compact(c, None, FAKE, BIG, None) == INVALID
    # calls without work do nothing
    assert _lib.bsmt_cache_write(c, 0, None, None, 0, None, None, None, 0, st, st, None) == OK
    assert _lib.bsmt_cache_gather(c, 0, None, None, 0, None, 0, None, None, None) == OK
    assert _lib.bsmt_cache_extend(c, None, None, 0, None, None, 0, None) == OK
    assert _lib.bsmt_cache_fork(c, None, None, 0, None, 0, None) == OK
    assert _lib.bsmt_cache_free(c, None, 0, None) == OK
    assert _lib.bsmt_paged_attention(None, 0, 8, c, 0, None, 0, None, None, None, 0.0, 1, None, None, None, 0, None) == OK


def test_workspaces():
    c, b = ctypes.byref(cache_struct()), ctypes.c_int64(0)
    assert _lib.bsmt_cache_workspace_bytes(c, 7, ctypes.byref(b)) == OK
    need = b.value
    assert need >= 3 * 100 * 4 and need >= 100 * 4 + 7 * 8
    assert _lib.bsmt_cache_workspace_bytes(c, -1, ctypes.byref(b)) == INVALID
    for ws, size in ((None, BIG), (FAKE + 128, BIG), (FAKE, need - 1)):
        assert _lib.bsmt_cache_extend(c, FAKE, None, 7, FAKE, ws, size, None) == INVALID
        assert _lib.bsmt_cache_fork(c, FAKE, FAKE, 7, ws, size, None) == INVALID
    assert _lib.bsmt_cache_compact(c, FAKE, FAKE, 100, None) == INVALID
    assert _lib.bsmt_paged_attention_workspace_bytes(96, ctypes.byref(b)) == UNSUPPORTED
    assert _lib.bsmt_paged_attention_workspace_bytes(128, ctypes.byref(b)) == OK
    assert _lib.bsmt_paged_attention(FAKE, 1, 8, c, 0, FAKE, 1, None, None, None, 0.0, 1, FAKE, FAKE, FAKE, b.value - 1, None) == INVALID


def test_paged_attention_arguments():
    c = ctypes.byref(cache_struct())

    def call(q=FAKE, T=1, Hq=8, mask=None, score=None, scale=0.0, gqa=1, out=FAKE, lse=FAKE, layer=0):
        return _lib.bsmt_paged_attention(q, T, Hq, c, layer, FAKE, T, None, mask, score, scale, gqa, out, lse, FAKE, BIG, None)

    assert call(Hq=6) == SHAPE and call(Hq=0) == SHAPE
    assert call(Hq=8, gqa=0) == SHAPE
    assert call(q=None) == INVALID and call(out=None) == INVALID and call(lse=None) == INVALID
    assert call(q=FAKE + 8) == INVALID and call(out=FAKE + 8) == INVALID and call(lse=FAKE + 2) == INVALID
    assert call(scale=math.nan) == INVALID and call(scale=math.inf) == INVALID and call(layer=2) == INVALID
    doc = _MaskSpec()
    doc.num_nodes = 1
    doc.nodes[0].kind = bsmt.MASK_DOCUMENT
    assert call(mask=ctypes.byref(doc)) == UNSUPPORTED
    assert b"DOCUMENT" in _lib.bsmt_last_error()
    bad = _MaskSpec()
    bad.num_nodes = 2
    assert call(mask=ctypes.byref(bad)) == INVALID
    cap = _ScoreSpec()
    cap.num_ops = 1
    cap.ops[0].kind, cap.ops[0].value = bsmt.SCORE_SOFTCAP, -1.0
    assert call(score=ctypes.byref(cap)) == INVALID


def rotary(spec=None, dtype=0, B=1, T=4, pos=FAKE, heads=(2,), addr=FAKE, n=None):
    t = (sv._RotaryTensor * 2)()
    for i, h in enumerate(heads):
        t[i].inp = t[i].out = addr
        t[i].heads = h
    spec = spec if spec is not None else bsmt.rotary_spec(64)._c
    return _lib.bsmt_rotary(ctypes.byref(spec), dtype, B, T, pos, strides(0, 0, 1), 0, t, len(heads) if n is None else n, None)


def test_rotary_arguments():
    assert rotary(dtype=2) == UNSUPPORTED and rotary(n=0) == INVALID and rotary(n=3) == INVALID
    assert rotary(B=-1) == INVALID and rotary(addr=None) == INVALID and rotary(addr=FAKE + 1) == INVALID
    assert rotary(heads=(-1,)) == INVALID and rotary(heads=(40000, 40000)) == UNSUPPORTED
    assert rotary(pos=None) == INVALID and rotary(pos=FAKE + 2) == INVALID
    assert rotary(T=0, pos=None) == OK and rotary(heads=(0,)) == OK
    for field, value in (("num_pairs", 0), ("num_pairs", 129), ("num_pairs", 33), ("num_axes", 0), ("num_axes", 128)):
        spec = sv._RotarySpecC.from_buffer_copy(bsmt.rotary_spec(64)._c)
        setattr(spec, field, value)
        assert rotary(spec) == INVALID, field
    spec = sv._RotarySpecC.from_buffer_copy(bsmt.rotary_spec(64)._c)
    spec.inv_freq[3] = math.inf
    assert rotary(spec) == INVALID
    spec = sv._RotarySpecC.from_buffer_copy(bsmt.rotary_spec(64)._c)
    spec.axis[3] = 1
    assert rotary(spec) == INVALID


def test_rotary_spec():
    s = bsmt.rotary_spec(128, [24, 20, 20])
    assert s.axis == (0,) * 24 + (1,) * 20 + (2,) * 20 and s.num_axes == 3
    assert s.inv_freq[0] == 1.0 and math.isclose(s.inv_freq[32], 0.01)
    s = bsmt.rotary_spec(64, [8, 8], base=100.0, per_axis=True)
    assert s.inv_freq[:8] == s.inv_freq[8:] and math.isclose(s.inv_freq[4], 0.1)
    assert len(bsmt.rotary_spec(64).inv_freq) == 32
    for args in ((64, [33]), (64, []), (64, [-1, 4]), (64, [0, 0])):
        with pytest.raises(ValueError):
            bsmt.rotary_spec(*args)
    for base in (0.0, -1.0, math.inf, math.nan):
        with pytest.raises(ValueError, match="base"):
            bsmt.rotary_spec(64, base=base)
    # the same spec, pair by pair
    s = bsmt.rotary_spec(80, [10, 0, 7], base=500.0, interleaved=True)
    t = bsmt.RotarySpec(80, tuple(500.0 ** (-i / 17) for i in range(17)), (0,) * 10 + (2,) * 7, 3, True)
    assert s == t and bytes(s._c) == bytes(t._c)
    with pytest.raises(ValueError, match="axes"):
        bsmt.RotarySpec(64, (1.0, 0.5), (0,))
    with pytest.raises(ValueError, match="axis"):
        bsmt.RotarySpec(64, (1.0, 0.5), (0, 1), 1)


def test_rotary_refuses_tensors():
    spec, pos = bsmt.rotary_spec(64), torch.zeros(4, dtype=torch.int32)
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    for q, match in ((x.half(), "bfloat16"), (x[0], "T, H, D"), (x[..., :32], "head dim"),
                     (x.transpose(0, 2).contiguous().transpose(0, 2), "contiguous"), (x, "CUDA")):
        with pytest.raises(ValueError, match=match):
            bsmt.rotary(q, None, pos, spec)


def host_cache(**more):
    return bsmt.create_paged_cache(10, 2, 64, 3, 4, 16, device="cpu", **more)


def test_cache_refuses_tensors():
    with pytest.raises(ValueError, match="dtype"):
        host_cache(dtype=torch.float16)
    c = host_cache(dtype=torch.int8)
    assert c.page_size == 16 and (c.page_table == -1).all() and (c.ref_counts == 0).all()
    fields = {f: getattr(c, f) for f in ("k", "v", "k_scale", "v_scale", "page_table", "seq_lens", "ref_counts")}
    for name, t in (("k", c.k[0]), ("v", c.v.float()), ("v", c.v[:, :9]), ("k_scale", c.k_scale.double()),
                    ("v_scale", c.v_scale[:, :, :1]), ("page_table", c.page_table[0]), ("page_table", c.page_table.long()),
                    ("seq_lens", c.seq_lens[:2]), ("ref_counts", c.ref_counts[:3]),
                    ("page_table", torch.zeros((4, 3), dtype=torch.int32).t())):
        with pytest.raises(ValueError):
            bsmt.PagedCache(**{**fields, name: t})
    s = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: bsmt.cache_extend(c, s), lambda: bsmt.cache_free(c, s), lambda: bsmt.cache_fork(c, s, s),
                 lambda: bsmt.cache_compact(c), lambda: bsmt.cache_gather(c, s, None, 1),
                 lambda: bsmt.cache_write(c, s, s, torch.zeros(1, 2, 64).bfloat16(), torch.zeros(1, 2, 64).bfloat16()),
                 lambda: bsmt.paged_attention(torch.zeros(1, 2, 64).bfloat16(), c, s)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
