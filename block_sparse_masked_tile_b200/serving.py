"""Positions and serving beside flex_attention: rotary positions with several
axes, a paged cache of keys and values in 8 bits, and attention over it.

Like the rest of the package this only marshals arguments; the kernels are in
``libbsmt.so`` (``include/bsmt_serving.h`` states each call's conditions).

* ``rotary(q, k, positions, spec)`` turns q and k before attention
  (differentiable); ``rotary_spec`` describes the axes and frequencies.
* ``create_paged_cache`` / ``PagedCache``: codes (float8_e4m3fn or int8) in
  pages, with a power-of-two scale for each page and head.
* ``cache_extend`` makes room for new tokens, ``cache_write`` quantises them,
  ``cache_gather`` reads tokens back, ``cache_fork``, ``cache_free`` and
  ``cache_compact`` manage the pages.
* ``paged_attention`` attends from each sequence's newest tokens to its cache.

Errors that only the device can see (a full cache, a page out of range) are
raised by ``check_device_status``.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Iterable, Sequence

import torch

from . import MaskMod, ScoreMod, _check, _check_launch, _lib, _MaskSpec, _score_spec, _ScoreSpec, _stream_ptr

__all__ = [
    "RotarySpec", "rotary_spec", "rotary", "rotary_backward", "PagedCache", "create_paged_cache", "cache_extend",
    "cache_write", "cache_gather", "cache_fork", "cache_free", "cache_compact", "cache_workspace_bytes",
    "paged_attention", "paged_attention_workspace_bytes",
]

MAX_ROTARY_PAIRS = 128
_CACHE_DTYPES = {torch.float8_e4m3fn: 0, torch.int8: 1}
_ROTARY_DTYPES = {torch.bfloat16: 0, torch.float32: 1}

_i32, _i64, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p


class _RotarySpecC(ctypes.Structure):
    _fields_ = [("head_dim", _i32), ("num_pairs", _i32), ("num_axes", _i32), ("interleaved", _i32),
                ("inv_freq", ctypes.c_double * MAX_ROTARY_PAIRS), ("axis", ctypes.c_int8 * MAX_ROTARY_PAIRS)]


class _RotaryTensor(ctypes.Structure):
    _fields_ = [("inp", _vp), ("out", _vp), ("in_strides", _i64 * 3), ("out_strides", _i64 * 3), ("heads", _i32)]


class _KvCache(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("k_scale", _vp), ("v_scale", _vp), ("page_table", _vp), ("seq_lens", _vp),
                ("ref_counts", _vp), ("num_layers", _i32), ("num_pages", _i32), ("num_kv_heads", _i32),
                ("page_size", _i32), ("head_dim", _i32), ("max_seqs", _i32), ("max_pages", _i32), ("dtype", _i32)]


def _declare() -> None:
    cache, strides = ctypes.POINTER(_KvCache), ctypes.POINTER(_i64)
    for name, args in {
        "bsmt_rotary": [ctypes.POINTER(_RotarySpecC), _i32, _i64, _i64, _vp, strides, _i32,
                        ctypes.POINTER(_RotaryTensor), _i32, _vp],
        "bsmt_cache_workspace_bytes": [cache, _i64, strides],
        "bsmt_cache_extend": [cache, _vp, _vp, _i64, _vp, _vp, _i64, _vp],
        "bsmt_cache_write": [cache, _i32, _vp, _vp, _i64, _vp, _vp, _vp, _i64, strides, strides, _vp],
        "bsmt_cache_gather": [cache, _i32, _vp, _vp, _i64, _vp, _i64, _vp, _vp, _vp],
        "bsmt_cache_fork": [cache, _vp, _vp, _i64, _vp, _i64, _vp],
        "bsmt_cache_free": [cache, _vp, _i64, _vp],
        "bsmt_cache_compact": [cache, _vp, _vp, _i64, _vp],
        "bsmt_paged_attention_workspace_bytes": [_i64, strides],
        "bsmt_paged_attention": [_vp, _i64, _i64, cache, _i32, _vp, _i64, _vp, ctypes.POINTER(_MaskSpec),
                                 ctypes.POINTER(_ScoreSpec), ctypes.c_float, _i32, _vp, _vp, _vp, _i64, _vp],
    }.items():
        f = getattr(_lib, name)
        f.argtypes = args
        f.restype = _i32


_declare()


# ------------------------------------------------------------------ rotary
@dataclass(frozen=True)
class RotarySpec:
    """Rotary positions of a head: pair i turns by position[axis[i]] * inv_freq[i].

    Pairs are (x[i], x[i + pairs]) or, ``interleaved``, (x[2i], x[2i + 1]) of
    the head's first 2 * pairs elements; the rest passes through. inv_freq and
    axis are given freely (scaled frequencies, any assignment of axes);
    ``rotary_spec`` makes the usual ones."""
    head_dim: int
    inv_freq: tuple
    axis: tuple
    num_axes: int = 1
    interleaved: bool = False

    def __post_init__(self):
        pairs = len(self.inv_freq)
        if not 1 <= pairs <= MAX_ROTARY_PAIRS or 2 * pairs > self.head_dim:
            raise ValueError(f"{pairs} rotary pairs in a head of {self.head_dim} (1 to {MAX_ROTARY_PAIRS} pairs)")
        if len(self.axis) != pairs:
            raise ValueError(f"{len(self.axis)} axes for {pairs} pairs")
        if not 1 <= self.num_axes <= 127 or any(not 0 <= a < self.num_axes for a in self.axis):
            raise ValueError(f"axis values must lie in [0, {self.num_axes}), with 1 to 127 axes")
        c = _RotarySpecC()
        c.head_dim, c.num_pairs, c.num_axes = int(self.head_dim), pairs, int(self.num_axes)
        c.interleaved = int(bool(self.interleaved))
        for i in range(pairs):
            c.inv_freq[i] = float(self.inv_freq[i])
            c.axis[i] = int(self.axis[i])
        object.__setattr__(self, "_c", c)


def rotary_spec(head_dim: int, sections: Sequence[int] | None = None, base: float = 10000.0,
                per_axis: bool = False, interleaved: bool = False) -> RotarySpec:
    """Rotary positions with ``sections[a]`` consecutive pairs for axis a (None:
    one axis, all head_dim / 2 pairs). Fewer pairs than head_dim / 2 leave the
    head's last elements as they are.

    inv_freq is base^(-i / pairs) over all pairs in one ladder, or with
    ``per_axis`` base^(-j / sections[a]) over each axis's own."""
    sections = [int(head_dim) // 2] if sections is None else [int(s) for s in sections]
    if any(s < 0 for s in sections) or sum(sections) < 1:
        raise ValueError(f"sections {sections}: pair counts must not be negative, and some pair must turn")
    pairs = sum(sections)
    axis, freq = [], []
    for a, s in enumerate(sections):
        for j in range(s):
            freq.append(float(base) ** (-j / s) if per_axis else float(base) ** (-len(axis) / pairs))
            axis.append(a)
    return RotarySpec(int(head_dim), tuple(freq), tuple(axis), len(sections), bool(interleaved))


def _heads_tokens(t: torch.Tensor) -> tuple:
    """(B, heads, T, strides of batch, head and token) of [T, H, D] or [B, H, T, D]."""
    if t.dim() == 3:
        return 1, t.shape[1], t.shape[0], (0, t.stride(1), t.stride(0))
    return t.shape[0], t.shape[1], t.shape[2], (t.stride(0), t.stride(1), t.stride(2))


def _rotary(tensors, positions: torch.Tensor, spec: RotarySpec, inverse: bool) -> list:
    first = tensors[0]
    dev = first.device
    B, _, T, _ = _heads_tokens(first)
    c = (_RotaryTensor * len(tensors))()
    outs = []
    for i, x in enumerate(tensors):
        b, h, n, s = _heads_tokens(x)
        y = torch.empty(x.shape, dtype=x.dtype, device=dev)
        c[i].inp, c[i].out, c[i].heads = x.data_ptr(), y.data_ptr(), h
        c[i].in_strides[:] = s
        c[i].out_strides[:] = _heads_tokens(y)[3]
        outs.append(y)
    strides = [positions.stride(0) if positions.dim() > 1 else 0,
               positions.stride(1) if positions.dim() == 3 else 0, positions.stride(-1)]
    with torch.cuda.device(dev):
        _check_launch(_lib.bsmt_rotary(ctypes.byref(spec._c), _ROTARY_DTYPES[first.dtype], B, T, positions.data_ptr(),
                                       (_i64 * 3)(*strides), int(inverse), c, len(tensors), _stream_ptr(dev)))
    return outs


class _RotaryFn(torch.autograd.Function):
    """The turn as a differentiable op; its gradient is the inverse turn."""

    @staticmethod
    def forward(ctx, positions, spec, inverse, *tensors):
        ctx.save_for_backward(positions)
        ctx.args = (spec, inverse)
        return tuple(_rotary(tensors, positions, spec, inverse))

    @staticmethod
    def backward(ctx, *grads):
        (positions,) = ctx.saved_tensors
        spec, inverse = ctx.args
        at = [i for i, g in enumerate(grads) if g is not None and ctx.needs_input_grad[3 + i]]
        out: list = [None] * len(grads)
        if at:
            # (a broadcast gradient, as of a sum, has stride 0 in its rows)
            some = [g if g.stride(-1) == 1 or g.shape[-1] == 1 else g.contiguous() for g in (grads[i] for i in at)]
            for i, g in zip(at, _RotaryFn.apply(positions, spec, not inverse, *some)):
                out[i] = g
        return (None, None, None, *out)


def _rotary_args(q, k, positions, spec) -> list:
    tensors = [q] if k is None else [q, k]
    for name, t in zip(("q", "k"), tensors):
        if t.dtype not in _ROTARY_DTYPES:
            raise ValueError(f"{name} must be bfloat16 or float32 (got {t.dtype})")
        if t.dim() not in (3, 4):
            raise ValueError(f"{name} must be [T, H, D] or [B, H, T, D]")
        if t.shape[-1] != spec.head_dim:
            raise ValueError(f"{name} has head dim {t.shape[-1]}, the spec {spec.head_dim}")
        if t.stride(-1) != 1 and t.shape[-1] > 1:
            raise ValueError(f"{name}'s innermost dimension must be contiguous")
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
    if k is not None and (k.dtype != q.dtype or k.device != q.device or k.dim() != q.dim()
                          or _heads_tokens(k)[0] != _heads_tokens(q)[0] or _heads_tokens(k)[2] != _heads_tokens(q)[2]):
        raise ValueError(f"q and k must share type, device, batch and tokens: q {tuple(q.shape)}, k {tuple(k.shape)}")
    if positions.dtype != torch.int32 or positions.device != q.device:
        raise ValueError(f"positions must be int32 on {q.device} (got {positions.dtype} on {positions.device})")
    B, _, T, _ = _heads_tokens(q)
    shapes = [(spec.num_axes, T)] + [(T,)] * (spec.num_axes == 1) + [(spec.num_axes, B, T)] * (q.dim() == 4)
    if tuple(positions.shape) not in shapes:
        raise ValueError(f"positions {tuple(positions.shape)}: expected one of {shapes}")
    return tensors


def rotary(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor, spec: RotarySpec):
    """Rotary positions on q and k (k may be None): bf16 or fp32, [B, H, T, D] or
    packed [T, H, D], their innermost dimension contiguous and the others of any
    strides (views of one fused projection are fine). ``positions``: int32
    [num_axes, T], [num_axes, B, T] for 4-D tensors, or [T] with one axis; any
    int32 value. Returns the turned (q, k), contiguous. Differentiable in q and
    k."""
    tensors = _rotary_args(q, k, positions, spec)
    if torch.is_grad_enabled() and any(t.requires_grad for t in tensors):
        outs = list(_RotaryFn.apply(positions, spec, False, *tensors))
    else:
        outs = _rotary(tensors, positions, spec, False)
    return (outs[0], outs[1]) if k is not None else (outs[0], None)


def rotary_backward(dq: torch.Tensor, dk: torch.Tensor | None, positions: torch.Tensor, spec: RotarySpec):
    """Gradients of ``rotary`` with respect to its q and k: dq and dk (may be
    None) turned back."""
    outs = _rotary(_rotary_args(dq, dk, positions, spec), positions, spec, True)
    return (outs[0], outs[1]) if dk is not None else (outs[0], None)


# ------------------------------------------------------------------- cache
@dataclass
class PagedCache:
    """Keys and values of many sequences in 8-bit pages (bsmt_kv_cache).

    k, v: float8_e4m3fn or int8 codes [layers, pages, Hkv, page_size, D];
    k_scale, v_scale: fp32 [layers, pages, Hkv]; page_table: int32
    [max_seqs, max_pages]; seq_lens: int32 [max_seqs]; ref_counts: int32
    [pages]. ``create_paged_cache`` makes an empty one."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor
    page_table: torch.Tensor
    seq_lens: torch.Tensor
    ref_counts: torch.Tensor

    def __post_init__(self):
        if self.k.dim() != 5 or self.k.dtype not in _CACHE_DTYPES:
            raise ValueError("cache codes must be float8_e4m3fn or int8 [layers, pages, Hkv, page_size, D]")
        layers, pages, heads, size, dim = self.k.shape
        if self.page_table.dim() != 2:
            raise ValueError("page_table must be [max_seqs, max_pages]")
        seqs = self.page_table.shape[0]
        for name, t, dtype, shape in (("v", self.v, self.k.dtype, self.k.shape),
                                      ("k_scale", self.k_scale, torch.float32, (layers, pages, heads)),
                                      ("v_scale", self.v_scale, torch.float32, (layers, pages, heads)),
                                      ("page_table", self.page_table, torch.int32, self.page_table.shape),
                                      ("seq_lens", self.seq_lens, torch.int32, (seqs,)),
                                      ("ref_counts", self.ref_counts, torch.int32, (pages,))):
            if t.dtype != dtype or t.shape != torch.Size(shape) or t.device != self.k.device:
                raise ValueError(f"cache {name} must be {dtype} {tuple(shape)} on {self.k.device} "
                                 f"(got {t.dtype} {tuple(t.shape)} on {t.device})")
        for name in ("k", "v", "k_scale", "v_scale", "page_table", "seq_lens", "ref_counts"):
            if not getattr(self, name).is_contiguous():
                raise ValueError(f"cache {name} must be contiguous")

    @property
    def device(self) -> torch.device:
        return self.k.device

    @property
    def page_size(self) -> int:
        return self.k.shape[3]

    def _struct(self) -> _KvCache:
        if not self.k.is_cuda:
            raise ValueError("the cache must be on a CUDA device")
        layers, pages, heads, size, dim = self.k.shape
        return _KvCache(self.k.data_ptr(), self.v.data_ptr(), self.k_scale.data_ptr(), self.v_scale.data_ptr(),
                        self.page_table.data_ptr(), self.seq_lens.data_ptr(), self.ref_counts.data_ptr(), layers,
                        pages, heads, size, dim, self.page_table.shape[0], self.page_table.shape[1],
                        _CACHE_DTYPES[self.k.dtype])


def create_paged_cache(num_pages: int, num_kv_heads: int, head_dim: int, max_seqs: int, max_pages: int,
                       page_size: int = 64, num_layers: int = 1, dtype: torch.dtype = torch.float8_e4m3fn,
                       device="cuda") -> PagedCache:
    """An empty cache of ``num_pages`` pages for up to ``max_seqs`` sequences of
    up to ``max_pages`` pages each."""
    if dtype not in _CACHE_DTYPES:
        raise ValueError(f"cache dtype must be float8_e4m3fn or int8 (got {dtype})")
    shape = (num_layers, num_pages, num_kv_heads, page_size, head_dim)
    k, v = (torch.zeros(shape, dtype=torch.int8, device=device).view(dtype) for _ in range(2))
    k_scale, v_scale = (torch.zeros(shape[:3], dtype=torch.float32, device=device) for _ in range(2))
    return PagedCache(k, v, k_scale, v_scale,
                      torch.full((max_seqs, max_pages), -1, dtype=torch.int32, device=device),
                      torch.zeros(max_seqs, dtype=torch.int32, device=device),
                      torch.zeros(num_pages, dtype=torch.int32, device=device))


def _list(cache: PagedCache, name: str, t: torch.Tensor | None, n: int | None = None) -> int | None:
    """Address of a list of int32 on the cache's device."""
    if t is None:
        return None
    if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous() or t.device != cache.device:
        raise ValueError(f"{name} must be a contiguous 1-D int32 tensor on {cache.device}")
    if n is not None and t.numel() != n:
        raise ValueError(f"{name} has {t.numel()} entries, expected {n}")
    return t.data_ptr()


def _workspace(workspace: torch.Tensor | None, need: int, device: torch.device) -> torch.Tensor:
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    if workspace.device != device or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {device}")
    return workspace


def cache_workspace_bytes(cache: PagedCache, n: int = 0) -> int:
    """Bytes of device workspace that cache_extend and cache_fork of n entries,
    and cache_compact (n = 0), need."""
    c, b = _KvCache(), _i64(0)
    c.num_pages = cache.k.shape[1]
    _check(_lib.bsmt_cache_workspace_bytes(ctypes.byref(c), int(n), ctypes.byref(b)))
    return int(b.value)


def cache_extend(cache: PagedCache, seqs: torch.Tensor, counts: torch.Tensor | None = None,
                 starts: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Makes room for counts[i] new tokens (None: one each) in sequence seqs[i].
    Returns ``starts`` (int32, written if given): the lengths before, where the
    new tokens go. All or nothing: where pages run out nothing changes, every
    start is -1 (which cache_write passes over) and check_device_status raises."""
    c = cache._struct()
    n = seqs.numel()
    lists = _list(cache, "seqs", seqs), _list(cache, "counts", counts, n)
    if starts is None:
        starts = torch.empty(n, dtype=torch.int32, device=cache.device)
    at = _list(cache, "starts", starts, n)
    ws = _workspace(workspace, cache_workspace_bytes(cache, n), cache.device)
    with torch.cuda.device(cache.device):
        _check_launch(_lib.bsmt_cache_extend(ctypes.byref(c), *lists, n, at, ws.data_ptr(), ws.numel(),
                                             _stream_ptr(cache.device)))
    return starts


def cache_write(cache: PagedCache, seqs: torch.Tensor, starts: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                cu_seqlens: torch.Tensor | None = None, layer: int = 0) -> None:
    """Quantises k, v (bf16 [T, Hkv, D]; the innermost dimension contiguous, the
    other strides multiples of 8) into the pages of sequences seqs from positions
    ``starts`` on, as cache_extend returned them. ``cu_seqlens`` (int32
    [n + 1]): the sequences' tokens in the pack; None: one token each."""
    c = cache._struct()
    n = seqs.numel()
    layers, _, heads, _, dim = cache.k.shape
    for name, t in (("k", k), ("v", v)):
        if t.dtype != torch.bfloat16 or t.dim() != 3 or t.shape[1:] != (heads, dim) or t.device != cache.device:
            raise ValueError(f"{name} must be bfloat16 [tokens, {heads}, {dim}] on {cache.device}")
        if t.numel() > 0 and t.stride(2) != 1:
            raise ValueError(f"{name}'s innermost dimension must be contiguous")
    if k.shape != v.shape:
        raise ValueError(f"shape mismatch: k {tuple(k.shape)}, v {tuple(v.shape)}")
    lists = (_list(cache, "seqs", seqs), _list(cache, "starts", starts, n), n,
             _list(cache, "cu_seqlens", cu_seqlens, n + 1))
    ks, vs = (_i64 * 2)(k.stride(0), k.stride(1)), (_i64 * 2)(v.stride(0), v.stride(1))
    with torch.cuda.device(cache.device):
        _check_launch(_lib.bsmt_cache_write(ctypes.byref(c), int(layer), *lists, k.data_ptr(), v.data_ptr(),
                                            k.shape[0], ks, vs, _stream_ptr(cache.device)))


def cache_gather(cache: PagedCache, seqs: torch.Tensor, starts: torch.Tensor | None, total: int,
                 cu_seqlens: torch.Tensor | None = None, layer: int = 0, k: torch.Tensor | None = None,
                 v: torch.Tensor | None = None):
    """(k, v) bf16 [total, Hkv, D] of cached tokens, dequantised: token t of the
    pack is position starts[i] + t - cu_seqlens[i] of sequence seqs[i]
    (``starts`` None: from 0; ``cu_seqlens`` None: one token each). For a
    prompt that goes on from a cached part, flex_attention_varlen takes them."""
    c = cache._struct()
    n = seqs.numel()
    _, _, heads, _, dim = cache.k.shape
    lists = (_list(cache, "seqs", seqs), _list(cache, "starts", starts, n), n,
             _list(cache, "cu_seqlens", cu_seqlens, n + 1))
    shape = (int(total), heads, dim)
    k = torch.empty(shape, dtype=torch.bfloat16, device=cache.device) if k is None else k
    v = torch.empty(shape, dtype=torch.bfloat16, device=cache.device) if v is None else v
    for name, t in (("k", k), ("v", v)):
        if t.shape != torch.Size(shape) or t.dtype != torch.bfloat16 or not t.is_contiguous() or t.device != cache.device:
            raise ValueError(f"{name} must be a contiguous bf16 tensor {shape} on {cache.device}")
    with torch.cuda.device(cache.device):
        _check_launch(_lib.bsmt_cache_gather(ctypes.byref(c), int(layer), *lists, int(total), k.data_ptr(),
                                             v.data_ptr(), _stream_ptr(cache.device)))
    return k, v


def cache_fork(cache: PagedCache, src: torch.Tensor, dst: torch.Tensor, workspace: torch.Tensor | None = None) -> None:
    """Slot dst[i], empty before, becomes a copy of sequence src[i]: full pages
    are shared, a partial last page is copied. All or nothing, as cache_extend."""
    c = cache._struct()
    n = src.numel()
    lists = _list(cache, "src", src), _list(cache, "dst", dst, n)
    ws = _workspace(workspace, cache_workspace_bytes(cache, n), cache.device)
    with torch.cuda.device(cache.device):
        _check_launch(_lib.bsmt_cache_fork(ctypes.byref(c), *lists, n, ws.data_ptr(), ws.numel(),
                                           _stream_ptr(cache.device)))


def cache_free(cache: PagedCache, seqs: torch.Tensor) -> None:
    """Empties sequences; pages that no other sequence holds become free."""
    c = cache._struct()
    at = _list(cache, "seqs", seqs)
    with torch.cuda.device(cache.device):
        _check_launch(_lib.bsmt_cache_free(ctypes.byref(c), at, seqs.numel(), _stream_ptr(cache.device)))


def cache_compact(cache: PagedCache, live: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Moves the pages in use to the front of the pool. Returns their number as
    an int32 [1] device tensor (``live``, written if given)."""
    c = cache._struct()
    if live is None:
        live = torch.empty(1, dtype=torch.int32, device=cache.device)
    at = _list(cache, "live", live, 1)
    ws = _workspace(workspace, cache_workspace_bytes(cache), cache.device)
    with torch.cuda.device(cache.device):
        _check_launch(_lib.bsmt_cache_compact(ctypes.byref(c), at, ws.data_ptr(), ws.numel(),
                                              _stream_ptr(cache.device)))
    return live


# --------------------------------------------------------------- attention
def paged_attention_workspace_bytes(head_dim: int) -> int:
    """Bytes of device workspace paged_attention needs."""
    b = _i64(0)
    _check(_lib.bsmt_paged_attention_workspace_bytes(int(head_dim), ctypes.byref(b)))
    return int(b.value)


def paged_attention(q: torch.Tensor, cache: PagedCache, seqs: torch.Tensor, cu_seqlens_q: torch.Tensor | None = None,
                    mask_mod: MaskMod | None = None, score_mod: ScoreMod | Iterable[ScoreMod] | None = None,
                    scale: float | None = None, enable_gqa: bool = False, layer: int = 0,
                    out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None):
    """Attention of the newest tokens of sequences ``seqs`` over their cached keys
    and values: q bf16 [T, Hq, D], the last cu_seqlens_q[i+1] - cu_seqlens_q[i]
    tokens of sequence seqs[i] (None: one each), already extended and written.
    ``mask_mod`` sees positions in the sequence (q_idx, kv_idx) and may be any
    mask without document(); None lets every query see every cached token, so
    several queries a sequence want causal(). Keys no query sees are not read.
    Returns (out bf16 [T, Hq, D], lse fp32 [Hq, T]); rows that see nothing get 0
    and -inf. No gradient flows to the cache."""
    if q.dtype != torch.bfloat16 or q.dim() != 3 or not q.is_contiguous() or q.device != cache.device:
        raise ValueError(f"q must be a contiguous bf16 tensor [tokens, Hq, D] on {cache.device}")
    c = cache._struct()
    T, Hq, D = q.shape
    if D != cache.k.shape[4]:
        raise ValueError(f"q has head dim {D}, the cache {cache.k.shape[4]}")
    if torch.is_grad_enabled() and q.requires_grad:
        raise ValueError("paged_attention has no backward; detach q or use flex_attention_varlen")
    n = seqs.numel()
    lists = _list(cache, "seqs", seqs), n, _list(cache, "cu_seqlens_q", cu_seqlens_q, n + 1)
    device = cache.device
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty((Hq, T), dtype=torch.float32, device=device) if lse is None else lse
    if out.shape != q.shape or out.dtype != torch.bfloat16 or not out.is_contiguous() or out.device != device:
        raise ValueError("out must be a contiguous bf16 tensor of q's shape and device")
    if lse.shape != (Hq, T) or lse.dtype != torch.float32 or not lse.is_contiguous() or lse.device != device:
        raise ValueError("lse must be a contiguous fp32 tensor [Hq, tokens] on q's device")
    ws = _workspace(workspace, paged_attention_workspace_bytes(D), device)
    with torch.cuda.device(device):
        mspec, keep_m = (None, []) if mask_mod is None else mask_mod._spec(device, 1)
        sspec, keep_s = _score_spec(score_mod, device, Hq)
        _check_launch(_lib.bsmt_paged_attention(
            q.data_ptr(), T, Hq, ctypes.byref(c), int(layer), *lists,
            ctypes.byref(mspec) if mspec is not None else None, ctypes.byref(sspec),
            ctypes.c_float(0.0 if scale is None else float(scale)), int(bool(enable_gqa)), out.data_ptr(),
            lse.data_ptr(), ws.data_ptr(), ws.numel(), _stream_ptr(device)))
    del keep_m, keep_s
    return out, lse
