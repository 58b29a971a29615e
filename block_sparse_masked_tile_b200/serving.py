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
import torch.autograd.forward_ad as _forward_ad

from . import MaskMod, ScoreMod, _check, _check_launch, _DEBUG_SYNC, _lib, _MaskSpec, _score_spec, _ScoreSpec

__all__ = [
    "RotarySpec", "rotary_spec", "rotary", "rotary_backward", "PagedCache", "create_paged_cache", "cache_extend",
    "cache_write", "cache_gather", "cache_fork", "cache_free", "cache_compact", "cache_workspace_bytes",
    "paged_attention", "paged_attention_workspace_bytes",
]

MAX_ROTARY_PAIRS = 128
_CACHE_DTYPES = {torch.float8_e4m3fn: 0, torch.int8: 1}
_ROTARY_DTYPES = {torch.bfloat16: 0, torch.float32: 1}

_i32, _i64, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
_I64x2, _I64x3 = _i64 * 2, _i64 * 3


class _RotarySpecC(ctypes.Structure):
    _fields_ = [("head_dim", _i32), ("num_pairs", _i32), ("num_axes", _i32), ("interleaved", _i32),
                ("inv_freq", ctypes.c_double * MAX_ROTARY_PAIRS), ("axis", ctypes.c_int8 * MAX_ROTARY_PAIRS)]


class _RotaryTensor(ctypes.Structure):
    _fields_ = [("inp", _vp), ("out", _vp), ("in_strides", _I64x3), ("out_strides", _I64x3), ("heads", _i32)]


class _KvCache(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("k_scale", _vp), ("v_scale", _vp), ("page_table", _vp), ("seq_lens", _vp),
                ("ref_counts", _vp), ("num_layers", _i32), ("num_pages", _i32), ("num_kv_heads", _i32),
                ("page_size", _i32), ("head_dim", _i32), ("max_seqs", _i32), ("max_pages", _i32), ("dtype", _i32)]


def _declare() -> None:
    cache, strides = ctypes.POINTER(_KvCache), ctypes.POINTER(_i64)
    for name, args in {
        "bsmt_rotary_sections": [_i32, ctypes.POINTER(_i32), _i32, ctypes.c_double, _i32, _i32,
                                 ctypes.POINTER(_RotarySpecC)],
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

# Serving calls are small and many, so their way to the library is short: the
# current device and stream as plain integers, no device switch where none is needed.
_device_now = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_byref = ctypes.byref


def _call(device: torch.device, f, *args) -> None:
    """f(*args, current stream of the device), with the device current."""
    index = device.index
    if index == _device_now():
        status = f(*args, torch._C._cuda_getCurrentRawStream(index))
        if status or _DEBUG_SYNC:
            _check_launch(status)
    else:
        with torch.cuda.device(device):
            _check_launch(f(*args, torch._C._cuda_getCurrentRawStream(index)))


def _differentiated(t: torch.Tensor) -> bool:
    """A gradient is to flow to t, or t is a dual tensor of forward mode."""
    return (t.requires_grad and torch.is_grad_enabled()
            or _forward_ad._current_level >= 0 and _forward_ad.unpack_dual(t).tangent is not None)


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
        if not 1 <= self.num_axes <= 127 or min(self.axis) < 0 or max(self.axis) >= self.num_axes:
            raise ValueError(f"axis values must lie in [0, {self.num_axes}), with 1 to 127 axes")
        object.__setattr__(self, "_c", _RotarySpecC(self.head_dim, pairs, self.num_axes, bool(self.interleaved),
                                                    tuple(self.inv_freq), tuple(self.axis)))


def rotary_spec(head_dim: int, sections: Sequence[int] | None = None, base: float = 10000.0,
                per_axis: bool = False, interleaved: bool = False) -> RotarySpec:
    """Rotary positions with ``sections[a]`` consecutive pairs for axis a (None:
    one axis, all head_dim / 2 pairs). Fewer pairs than head_dim / 2 leave the
    head's last elements as they are.

    inv_freq is base^(-i / pairs) over all pairs in one ladder, or with
    ``per_axis`` base^(-j / sections[a]) over each axis's own."""
    sections = [int(head_dim) // 2] if sections is None else list(sections)
    c = _RotarySpecC()
    _check(_lib.bsmt_rotary_sections(head_dim, (_i32 * len(sections))(*sections), len(sections), base, bool(per_axis),
                                     bool(interleaved), _byref(c)))
    spec = object.__new__(RotarySpec)  # (the library has checked it)
    n = c.num_pairs
    for name, value in (("head_dim", c.head_dim), ("inv_freq", tuple(c.inv_freq[:n])), ("axis", tuple(c.axis[:n])),
                        ("num_axes", c.num_axes), ("interleaved", bool(c.interleaved)), ("_c", c)):
        object.__setattr__(spec, name, value)
    return spec


def _heads_tokens(t: torch.Tensor) -> tuple:
    """(B, heads, T, strides of batch, head and token) of [T, H, D] or [B, H, T, D]."""
    shape, stride = t.shape, t.stride()
    if len(shape) == 3:
        return 1, shape[1], shape[0], (0, stride[1], stride[0])
    return shape[0], shape[1], shape[2], stride[:3]


def _rotary(tensors, positions: torch.Tensor, spec: RotarySpec, inverse: bool) -> list:
    first = tensors[0]
    dev, dtype = first.device, first.dtype
    outs, c = [], (_RotaryTensor * len(tensors))()
    for i, x in enumerate(tensors):
        y = torch.empty(x.shape, dtype=dtype, device=dev)
        B, heads, T, strides = _heads_tokens(x)
        c[i] = x.data_ptr(), y.data_ptr(), strides, _heads_tokens(y)[3], heads
        outs.append(y)
    dims = positions.dim()
    strides = _I64x3(positions.stride(0) if dims > 1 else 0, positions.stride(1) if dims == 3 else 0,
                     positions.stride(dims - 1))
    _call(dev, _lib.bsmt_rotary, _byref(spec._c), _ROTARY_DTYPES[dtype], B, T, positions.data_ptr(), strides,
          int(inverse), c, len(tensors))
    return outs


def _turn(tensors, positions: torch.Tensor, spec: RotarySpec, inverse: bool) -> list:
    """_rotary, as a differentiable op where a gradient or a tangent is to flow."""
    if any(_differentiated(t) for t in tensors):
        outs = _RotaryFn.apply(positions, spec, inverse, *tensors)
        return [y if _differentiated(t) else y.detach() for t, y in zip(tensors, outs)]
    return _rotary(tensors, positions, spec, inverse)


def _rows(g: torch.Tensor) -> torch.Tensor:
    """g with contiguous rows (a broadcast gradient, as of a sum, has stride 0 in them)."""
    return g if g.stride(-1) == 1 or g.shape[-1] == 1 else g.contiguous()


class _RotaryFn(torch.autograd.Function):
    """The turn as a differentiable op. It is linear: its gradient is the inverse
    turn, a tangent turns as its tensor does."""

    @staticmethod
    def forward(ctx, positions, spec, inverse, *tensors):
        ctx.save_for_backward(positions)
        ctx.save_for_forward(positions)
        ctx.args = (spec, inverse)
        return tuple(_rotary(tensors, positions, spec, inverse))

    @staticmethod
    def backward(ctx, *grads):
        (positions,) = ctx.saved_tensors
        spec, inverse = ctx.args
        at = [i for i, g in enumerate(grads) if g is not None and ctx.needs_input_grad[3 + i]]
        out: list = [None] * len(grads)
        if at:  # (a gradient that needs one itself, as under create_graph, is turned differentiably)
            for i, g in zip(at, _turn([_rows(grads[i]) for i in at], positions, spec, not inverse)):
                out[i] = g
        return (None, None, None, *out)

    @staticmethod
    def jvp(ctx, _positions, _spec, _inverse, *tangents):
        (positions,) = ctx.saved_tensors
        return tuple(_turn([_rows(t) for t in tangents], positions, *ctx.args))


def _rotary_args(q, k, positions, spec) -> list:
    tensors = [q] if k is None else [q, k]
    for name, t in zip("qk", tensors):
        shape = t.shape
        if t.dtype not in _ROTARY_DTYPES:
            raise ValueError(f"{name} must be bfloat16 or float32 (got {t.dtype})")
        if len(shape) != 3 and len(shape) != 4:
            raise ValueError(f"{name} must be [T, H, D] or [B, H, T, D]")
        if shape[-1] != spec.head_dim:
            raise ValueError(f"{name} has head dim {shape[-1]}, the spec {spec.head_dim}")
        if t.stride(-1) != 1 and shape[-1] > 1:
            raise ValueError(f"{name}'s innermost dimension must be contiguous")
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
    B, _, T, _ = _heads_tokens(q)
    if k is not None:
        Bk, _, Tk, _ = _heads_tokens(k)
        if k.dtype is not q.dtype or k.get_device() != q.get_device() or k.dim() != q.dim() or Bk != B or Tk != T:
            raise ValueError(f"q and k must share type, device, batch and tokens: q {tuple(q.shape)}, k {tuple(k.shape)}")
    if positions.dtype is not torch.int32 or positions.get_device() != q.get_device():
        raise ValueError(f"positions must be int32 on {q.device} (got {positions.dtype} on {positions.device})")
    shape, axes = tuple(positions.shape), spec.num_axes
    if shape != (axes, T) and not (shape == (T,) and axes == 1) and not (shape == (axes, B, T) and q.dim() == 4):
        raise ValueError(f"positions {shape}: expected [{axes}, {T}]" + (f", [{T}]" if axes == 1 else "")
                         + (f" or [{axes}, {B}, {T}]" if q.dim() == 4 else ""))
    return tensors


def rotary(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor, spec: RotarySpec):
    """Rotary positions on q and k (k may be None): bf16 or fp32, [B, H, T, D] or
    packed [T, H, D], their innermost dimension contiguous and the others of any
    strides (views of one fused projection are fine). ``positions``: int32
    [num_axes, T], [num_axes, B, T] for 4-D tensors, or [T] with one axis; any
    int32 value. Returns the turned (q, k), contiguous. Differentiable in q and
    k, in reverse and in forward mode. (As with any torch operation, a step with
    its backward pass is captured into a CUDA graph while no eager graph of the
    same leaves is alive.)"""
    tensors = _rotary_args(q, k, positions, spec)
    outs = _turn(tensors, positions, spec, False)
    return (outs[0], outs[1]) if k is not None else (outs[0], None)


def rotary_backward(dq: torch.Tensor, dk: torch.Tensor | None, positions: torch.Tensor, spec: RotarySpec):
    """Gradients of ``rotary`` with respect to its q and k: dq and dk (may be
    None) turned back. Differentiable as ``rotary`` is."""
    outs = _turn(_rotary_args(dq, dk, positions, spec), positions, spec, True)
    return (outs[0], outs[1]) if dk is not None else (outs[0], None)


# ------------------------------------------------------------------- cache
@dataclass(frozen=True)
class PagedCache:
    """Keys and values of many sequences in 8-bit pages (bsmt_kv_cache).

    k, v: float8_e4m3fn or int8 codes [layers, pages, Hkv, page_size, D];
    k_scale, v_scale: fp32 [layers, pages, Hkv]; page_table: int32
    [max_seqs, max_pages]; seq_lens: int32 [max_seqs]; ref_counts: int32
    [pages]. ``create_paged_cache`` makes an empty one. The tensors' contents
    change under the calls below, their places must not."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor
    page_table: torch.Tensor
    seq_lens: torch.Tensor
    ref_counts: torch.Tensor

    def __post_init__(self):
        k, v, table, at = self.k, self.v, self.page_table, self.k.get_device()  # (-1: the host)
        if k.dim() != 5 or k.dtype not in _CACHE_DTYPES:
            raise ValueError("cache codes must be float8_e4m3fn or int8 [layers, pages, Hkv, page_size, D]")
        if table.dim() != 2:
            raise ValueError("page_table must be [max_seqs, max_pages]")
        layers, pages, heads, size, dim = shape = k.shape
        seqs, wide = table.shape
        f32, i32 = torch.float32, torch.int32
        for name, t, dtype, want in (("k", k, k.dtype, shape), ("v", v, k.dtype, shape),
                                     ("k_scale", self.k_scale, f32, shape[:3]), ("v_scale", self.v_scale, f32, shape[:3]),
                                     ("page_table", table, i32, table.shape), ("seq_lens", self.seq_lens, i32, (seqs,)),
                                     ("ref_counts", self.ref_counts, i32, (pages,))):
            if t.dtype is not dtype or t.shape != want or t.get_device() != at or not t.is_contiguous():
                raise ValueError(f"cache {name} must be contiguous {dtype} {tuple(want)} on {k.device} "
                                 f"(got {t.dtype} {tuple(t.shape)} on {t.device})")
        object.__setattr__(self, "_c", _KvCache(
            k.data_ptr(), v.data_ptr(), self.k_scale.data_ptr(), self.v_scale.data_ptr(), table.data_ptr(),
            self.seq_lens.data_ptr(), self.ref_counts.data_ptr(), layers, pages, heads, size, dim, seqs, wide,
            _CACHE_DTYPES[k.dtype]))

    @property
    def device(self) -> torch.device:
        return self.k.device

    @property
    def page_size(self) -> int:
        return self.k.shape[3]


def _on_gpu(cache: PagedCache) -> tuple:
    """The cache's C form and its device."""
    if not cache.k.is_cuda:
        raise ValueError("the cache must be on a CUDA device")
    return _byref(cache._c), cache.k.device


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


def _list(device: torch.device, name: str, t: torch.Tensor | None, n: int | None = None) -> int | None:
    """Address of a list of n int32 on the cache's device."""
    if t is None:
        return None
    if t.dtype is not torch.int32 or t.dim() != 1 or t.get_device() != device.index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 1-D int32 tensor on {device}")
    if n is not None and t.shape[0] != n:
        raise ValueError(f"{name} has {t.shape[0]} entries, expected {n}")
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
    b = _i64(0)
    _check(_lib.bsmt_cache_workspace_bytes(_byref(cache._c), int(n), _byref(b)))
    return b.value


def cache_extend(cache: PagedCache, seqs: torch.Tensor, counts: torch.Tensor | None = None,
                 starts: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Makes room for counts[i] new tokens (None: one each) in sequence seqs[i].
    Returns ``starts`` (int32, written if given): the lengths before, where the
    new tokens go. All or nothing: where pages run out nothing changes, every
    start is -1 (which cache_write passes over) and check_device_status raises."""
    c, dev = _on_gpu(cache)
    n = seqs.numel()
    at = _list(dev, "seqs", seqs), _list(dev, "counts", counts, n)
    if starts is None:
        starts = torch.empty(n, dtype=torch.int32, device=dev)
    ws = _workspace(workspace, cache_workspace_bytes(cache, n), dev)
    _call(dev, _lib.bsmt_cache_extend, c, *at, n, _list(dev, "starts", starts, n), ws.data_ptr(), ws.numel())
    return starts


def cache_write(cache: PagedCache, seqs: torch.Tensor, starts: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                cu_seqlens: torch.Tensor | None = None, layer: int = 0) -> None:
    """Quantises k, v (bf16 [T, Hkv, D]; the innermost dimension contiguous, the
    other strides multiples of 8) into the pages of sequences seqs from positions
    ``starts`` on, as cache_extend returned them. ``cu_seqlens`` (int32
    [n + 1]): the sequences' tokens in the pack; None: one token each. A
    sequence may be listed once. No gradient flows through the cache: k and v
    that need one are refused."""
    c, dev = _on_gpu(cache)
    n = seqs.numel()
    _, _, heads, _, dim = cache.k.shape
    for name, t in (("k", k), ("v", v)):
        if _differentiated(t):
            raise ValueError(f"cache_write has no backward; detach {name}")
        if t.dtype is not torch.bfloat16 or t.dim() != 3 or t.shape[1:] != (heads, dim) or t.get_device() != dev.index:
            raise ValueError(f"{name} must be bfloat16 [tokens, {heads}, {dim}] on {dev}")
        if t.stride(2) != 1 and t.numel() > 0:
            raise ValueError(f"{name}'s innermost dimension must be contiguous")
    if k.shape != v.shape:
        raise ValueError(f"shape mismatch: k {tuple(k.shape)}, v {tuple(v.shape)}")
    _call(dev, _lib.bsmt_cache_write, c, int(layer), _list(dev, "seqs", seqs), _list(dev, "starts", starts, n), n,
          _list(dev, "cu_seqlens", cu_seqlens, n + 1), k.data_ptr(), v.data_ptr(), k.shape[0],
          _I64x2(k.stride(0), k.stride(1)), _I64x2(v.stride(0), v.stride(1)))


def cache_gather(cache: PagedCache, seqs: torch.Tensor, starts: torch.Tensor | None, total: int,
                 cu_seqlens: torch.Tensor | None = None, layer: int = 0, k: torch.Tensor | None = None,
                 v: torch.Tensor | None = None):
    """(k, v) bf16 [total, Hkv, D] of cached tokens, dequantised: token t of the
    pack is position starts[i] + t - cu_seqlens[i] of sequence seqs[i]
    (``starts`` None: from 0; ``cu_seqlens`` None: one token each). For a
    prompt that goes on from a cached part, flex_attention_varlen takes them."""
    c, dev = _on_gpu(cache)
    n = seqs.numel()
    _, _, heads, _, dim = cache.k.shape
    shape = (int(total), heads, dim)
    if k is None:
        k = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    if v is None:
        v = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    for name, t in (("k", k), ("v", v)):
        if t.shape != shape or t.dtype is not torch.bfloat16 or t.get_device() != dev.index or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous bf16 tensor {shape} on {dev}")
    _call(dev, _lib.bsmt_cache_gather, c, int(layer), _list(dev, "seqs", seqs), _list(dev, "starts", starts, n), n,
          _list(dev, "cu_seqlens", cu_seqlens, n + 1), shape[0], k.data_ptr(), v.data_ptr())
    return k, v


def cache_fork(cache: PagedCache, src: torch.Tensor, dst: torch.Tensor, workspace: torch.Tensor | None = None) -> None:
    """Slot dst[i], empty before, becomes a copy of sequence src[i]: full pages
    are shared, a partial last page is copied. All or nothing, as cache_extend."""
    c, dev = _on_gpu(cache)
    n = src.numel()
    ws = _workspace(workspace, cache_workspace_bytes(cache, n), dev)
    _call(dev, _lib.bsmt_cache_fork, c, _list(dev, "src", src), _list(dev, "dst", dst, n), n, ws.data_ptr(), ws.numel())


def cache_free(cache: PagedCache, seqs: torch.Tensor) -> None:
    """Empties sequences; pages that no other sequence holds become free."""
    c, dev = _on_gpu(cache)
    _call(dev, _lib.bsmt_cache_free, c, _list(dev, "seqs", seqs), seqs.numel())


def cache_compact(cache: PagedCache, live: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Moves the pages in use to the front of the pool. Returns their number as
    an int32 [1] device tensor (``live``, written if given)."""
    c, dev = _on_gpu(cache)
    if live is None:
        live = torch.empty(1, dtype=torch.int32, device=dev)
    ws = _workspace(workspace, cache_workspace_bytes(cache), dev)
    _call(dev, _lib.bsmt_cache_compact, c, _list(dev, "live", live, 1), ws.data_ptr(), ws.numel())
    return live


# --------------------------------------------------------------- attention
def paged_attention_workspace_bytes(head_dim: int) -> int:
    """Bytes of device workspace paged_attention needs."""
    b = _i64(0)
    _check(_lib.bsmt_paged_attention_workspace_bytes(int(head_dim), _byref(b)))
    return b.value


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
    c, device = _on_gpu(cache)
    if q.dtype is not torch.bfloat16 or q.dim() != 3 or q.get_device() != device.index or not q.is_contiguous():
        raise ValueError(f"q must be a contiguous bf16 tensor [tokens, Hq, D] on {device}")
    T, Hq, D = q.shape
    if D != cache.k.shape[4]:
        raise ValueError(f"q has head dim {D}, the cache {cache.k.shape[4]}")
    if _differentiated(q):
        raise ValueError("paged_attention has no backward; detach q or use flex_attention_varlen")
    n = seqs.numel()
    at = _list(device, "seqs", seqs), n, _list(device, "cu_seqlens_q", cu_seqlens_q, n + 1)
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape or out.dtype != torch.bfloat16 or not out.is_contiguous() or out.device != device:
        raise ValueError("out must be a contiguous bf16 tensor of q's shape and device")
    if lse is None:
        lse = torch.empty((Hq, T), dtype=torch.float32, device=device)
    elif lse.shape != (Hq, T) or lse.dtype != torch.float32 or not lse.is_contiguous() or lse.device != device:
        raise ValueError("lse must be a contiguous fp32 tensor [Hq, tokens] on q's device")
    ws = _workspace(workspace, paged_attention_workspace_bytes(D), device)
    mspec, keep_m = (None, None) if mask_mod is None else mask_mod._spec(device, 1)
    sspec, keep_s = _score_spec(score_mod, device, Hq)
    _call(device, _lib.bsmt_paged_attention, q.data_ptr(), T, Hq, c, int(layer), *at,
          None if mspec is None else _byref(mspec), _byref(sspec), 0.0 if scale is None else float(scale),
          int(bool(enable_gqa)), out.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel())
    del keep_m, keep_s
    return out, lse
