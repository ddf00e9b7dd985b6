"""Binding of what a decoder remembers between tokens (see ``include/q1_memory.h``):
keys and values in pages of 4 or 8 bits with the attention that reads them, the
short causal convolution, the selective state space scan.

Argument marshalling only, like ``decode.py``, whose workspaces it shares: every
operation runs in the library's HIP kernels on the current stream of its tensors'
device, and what the checks of the operands' shapes, strides and types found is
kept by those (never by a tensor or its address).
"""
from __future__ import annotations

import ctypes
import struct
from typing import Optional

import torch

from . import decode as _d
from .decode import _dense, _dense_strides, _given, _new, _ptr, _same_device
from .q1 import _TORCH_TO_Q1, _check, load_library

KV_BLOCK = 32  # elements that share a scale


class _KV(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("pages", ctypes.c_int64), ("page_size", ctypes.c_int64),
                ("Hkv", ctypes.c_int32), ("D", ctypes.c_int32), ("bits", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class _KVQuery(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("page_table", ctypes.c_void_p), ("lens", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("q_ld", ctypes.c_int64), ("B", ctypes.c_int64),
                ("T", ctypes.c_int64), ("max_pages", ctypes.c_int64), ("Hq", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("scale", ctypes.c_float)]


class _Conv(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("state", ctypes.c_void_p),
                ("slot_ids", ctypes.c_void_p), ("out", ctypes.c_void_p), ("x_ld", ctypes.c_int64), ("slots", ctypes.c_int64),
                ("C", ctypes.c_int64), ("W", ctypes.c_int32), ("dtype", ctypes.c_int32), ("silu", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class _Scan(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("dt", ctypes.c_void_p), ("B", ctypes.c_void_p), ("C", ctypes.c_void_p),
                ("z", ctypes.c_void_p), ("A", ctypes.c_void_p), ("D", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p),
                ("state", ctypes.c_void_p), ("slot_ids", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("x_ld", ctypes.c_int64), ("dt_ld", ctypes.c_int64), ("b_ld", ctypes.c_int64), ("c_ld", ctypes.c_int64),
                ("z_ld", ctypes.c_int64), ("slots", ctypes.c_int64), ("Di", ctypes.c_int64), ("N", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("dt_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("softplus", ctypes.c_int32), ("reserved", ctypes.c_int32)]


_KV_PACK = struct.Struct("@4P2q4i").pack        # the fields of _KV
_KVQUERY_PACK = struct.Struct("@5P4q3if").pack  # the fields of _KVQuery
_CONV_PACK = struct.Struct("@6P3q4i").pack      # the fields of _Conv
_SCAN_PACK = struct.Struct("@11P7q6i").pack     # the fields of _Scan


def _layout(t: Optional[torch.Tensor]):
    return None if t is None else (t.shape, t.stride(), t.dtype, t.get_device())


def _addr(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.data_ptr()


def _row_stride(t: torch.Tensor, name: str, lead: int) -> int:
    """As for the other calls; a tensor without elements has dense rows."""
    return _d._row_stride(t, name, lead) if t.numel() else t.shape[lead:].numel()


def _keep(kept: dict, key, found):
    if len(kept) > 4096:
        kept.clear()
    kept[key] = found
    return found


class PackedKV:
    """Pages of keys and values in 4 or 8 bits.

    k, v: uint8 ``[pages, Hkv, page_size, D * bits / 8]`` codes (4 bits: two to a
    byte, the even element in the low half); k_scales, v_scales: uint8 ``[pages,
    Hkv, page_size, D / 32]``, the scales' exponents + 127."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor, bits: int = 4):
        if bits not in (4, 8):
            raise ValueError(f"bits must be 4 or 8, not {bits}")
        if k.dim() != 4:
            raise ValueError("k must be [pages, Hkv, page_size, D * bits / 8]")
        _dense(k, "k", torch.uint8, k.shape)
        _dense(v, "v", torch.uint8, k.shape)
        pages, Hkv, page_size, row = k.shape
        D = row * 8 // bits
        if D not in (64, 128, 256):
            raise ValueError(f"D must be 64, 128 or 256 (rows of {row} bytes are {D})")
        _dense(k_scales, "k_scales", torch.uint8, (pages, Hkv, page_size, D // KV_BLOCK))
        _dense(v_scales, "v_scales", torch.uint8, (pages, Hkv, page_size, D // KV_BLOCK))
        for name, t in (("v", v), ("k_scales", k_scales), ("v_scales", v_scales)):
            if t.device != k.device:
                raise ValueError(f"{name} is on {t.device}, not on {k.device}")
        self._tensors = (k, v, k_scales, v_scales)
        self.bits, self.D, self.Hkv, self.pages, self.page_size = bits, D, Hkv, pages, page_size
        self.device = k.device
        self._index = k.get_device()
        self._geometry = (pages, page_size, Hkv, D, bits, self._index)
        self._desc = _KV_PACK(*(t.data_ptr() if pages else 0 for t in self._tensors), pages, page_size, Hkv, D, bits, 0)

    k = property(lambda self: self._tensors[0])
    v = property(lambda self: self._tensors[1])
    k_scales = property(lambda self: self._tensors[2])
    v_scales = property(lambda self: self._tensors[3])

    @staticmethod
    def empty(pages: int, page_size: int, Hkv: int, D: int, bits: int = 4, device="cuda") -> "PackedKV":
        """Pages whose every value is 0."""
        codes = (pages, Hkv, page_size, D * bits // 8)
        scales = (pages, Hkv, page_size, D // KV_BLOCK)
        new = lambda shape: torch.zeros(shape, dtype=torch.uint8, device=device)  # noqa: E731
        return PackedKV(new(codes), new(codes), new(scales), new(scales), bits)


def _check_rows(cache, slots, operands):
    """(rows, layouts' device) of a write or read of the pages."""
    _same_device(slots, pages=cache.k, **operands)
    if slots.dim() != 1:
        raise ValueError("slots must be [rows]")
    _dense(slots, "slots", torch.int32, slots.shape)
    for name, t in operands.items():
        if t is not None and tuple(t.shape) != (slots.shape[0], cache.Hkv, cache.D):
            raise ValueError(f"{name} must have shape {(slots.shape[0], cache.Hkv, cache.D)}, not {tuple(t.shape)}")
    return slots.shape[0]


_write_layouts = {}


def q1_kv_write(cache: PackedKV, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor) -> None:
    """Quantises rows of keys and values into the pages: k, v ``[tokens, Hkv, D]`` bf16
    or fp16 (rows evenly spaced), row t to token ``slots[t] % page_size`` of page
    ``slots[t] // page_size``; slots int32 ``[tokens]``, distinct.  A slot outside the
    pages (such as -1) leaves its row out."""
    key = (_layout(k), _layout(v), _layout(slots), cache._geometry, _d._device())
    found = _write_layouts.get(key)
    if found is None:
        tokens = _check_rows(cache, slots, dict(k=k, v=v))
        if v.dtype != k.dtype:
            raise ValueError("k and v must have one dtype")
        found = _keep(_write_layouts, key, (_TORCH_TO_Q1.get(k.dtype, -1), _row_stride(k, "k", 1), _row_stride(v, "v", 1), tokens))
    status = load_library().q1_kv_write(cache._desc, k.data_ptr(), v.data_ptr(), *found, slots.data_ptr(),
                                        _d._stream_of(cache._index))
    if status:
        _check(status)


_read_layouts = {}


def q1_kv_read(cache: PackedKV, slots: torch.Tensor, out_dtype: Optional[torch.dtype] = None,
               k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None):
    """The values of rows of the pages: returns (k, v) ``[rows, Hkv, D]`` in out_dtype
    (bf16 by default, or that of ``k`` or ``v`` where given to be written); slots int32
    ``[rows]``, which may repeat; zeros for a slot outside the pages."""
    key = (_layout(slots), _layout(k), _layout(v), out_dtype, cache._geometry, _d._device())
    found = _read_layouts.get(key)
    if found is None:
        rows = _check_rows(cache, slots, dict(k=k, v=v))
        dtype = out_dtype or (k.dtype if k is not None else v.dtype if v is not None else torch.bfloat16)
        shape = (rows, cache.Hkv, cache.D)
        _dense(k, "k", dtype, shape)
        _dense(v, "v", dtype, shape)
        found = _keep(_read_layouts, key, (rows, dtype, _TORCH_TO_Q1.get(dtype, -1), shape, _dense_strides(shape)))
    rows, dtype, code, shape, strides = found
    if k is None:
        k = _new(shape, strides, dtype=dtype, device=cache.device)
    if v is None:
        v = _new(shape, strides, dtype=dtype, device=cache.device)
    status = load_library().q1_kv_read(cache._desc, slots.data_ptr(), rows, k.data_ptr(), v.data_ptr(), code,
                                       _d._stream_of(cache._index))
    if status:
        _check(status)
    return k, v


_kv_layouts = {}


def _check_kv_attn(q, cache, page_table, lens, out, out_dtype, lse):
    """The descriptor's fields that follow from the operands' layouts."""
    if q.dim() != 4:
        raise ValueError("q must be [B, T, Hq, D]")
    _same_device(q, pages=cache.k, page_table=page_table, lens=lens, out=out, lse=lse)
    B, T, Hq, D = q.shape
    if D != cache.D:
        raise ValueError(f"q has D = {D}, the pages {cache.D}")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [B, max_pages]")
    _dense(page_table, "page_table", torch.int32, (B, page_table.shape[1]))
    _dense(lens, "lens", torch.int32, (B,))
    if out is not None:
        _dense(out, "out", out.dtype if out_dtype is None else out_dtype, q.shape)
        out_dtype = out.dtype
    elif out_dtype is None:
        out_dtype = q.dtype
    _dense(lse, "lse", torch.float32, (B, T, Hq))
    return ((_row_stride(q, "q", 2), B, T, page_table.shape[1]),
            (Hq, _TORCH_TO_Q1.get(q.dtype, -1), _TORCH_TO_Q1.get(out_dtype, -1)), out_dtype, D ** -0.5,
            (B, T, Hq, D), _dense_strides((B, T, Hq, D)), None)


def q1_kv_attn(q: torch.Tensor, cache: PackedKV, page_table: torch.Tensor, lens: torch.Tensor,
               scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
               out_dtype: Optional[torch.dtype] = None, lse: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None):
    """Attention over quantised pages; returns (out ``[B, T, Hq, D]``, lse fp32 ``[B, T, Hq]``).

    q ``[B, T, Hq, D]`` bf16 or fp16 (rows evenly spaced): the last T of the
    ``lens[b]`` tokens of sequence b, each seeing itself and what is before it;
    page_table int32 ``[B, max_pages]``, lens int32 ``[B]``.  ``scale`` defaults to
    D^-1/2."""
    key = (_layout(q), _layout(page_table), _layout(lens), _layout(out), _layout(lse), out_dtype, cache._geometry,
           _d._device())
    found = _kv_layouts.get(key)
    if found is None:
        found = _check_kv_attn(q, cache, page_table, lens, out, out_dtype, lse)
    longs, ints, dtype, usual, shape, strides, need = found
    if out is None:
        out = _new(shape, strides, dtype=dtype, device=cache.device)
    if lse is None:
        lse = _new(shape[:3], (shape[1] * shape[2], shape[2], 1), dtype=torch.float32, device=cache.device)
    a = _KVQUERY_PACK(q.data_ptr(), page_table.data_ptr() if longs[3] else 0, lens.data_ptr(), out.data_ptr(),
                      lse.data_ptr(), *longs, *ints, usual if scale is None else scale)
    L = load_library()
    stream = _d._stream_of(cache._index)
    if need is None:  # a layout that is new: its workspace depends on nothing else
        need = L.q1_kv_attn_workspace_bytes(cache._desc, a)
        _keep(_kv_layouts, key, (*found[:-1], need))
    if workspace is None:
        workspace = _d._workspace(need, cache._index, stream) if need else None
    else:
        _given(workspace, cache._index)
    status = L.q1_kv_attn(cache._desc, a, _ptr(workspace), 0 if workspace is None else workspace.numel(), stream)
    if status:
        _check(status)
    return out, lse


def _check_cu(cu_seqlens):
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be [nseq + 1]")
    if cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens must be contiguous int32")


_conv_layouts = {}


def _check_conv(x, weight, state, bias, slots, nseq, out, cu_seqlens):
    _same_device(x, weight=weight, state=state, bias=bias, slots=slots, out=out, cu_seqlens=cu_seqlens)
    if cu_seqlens is not None:
        _check_cu(cu_seqlens)
    C = x.shape[-1]
    if weight.dim() != 2:
        raise ValueError("weight must be [C, W]")
    W = weight.shape[1]
    _dense(weight, "weight", x.dtype, (C, W))
    _dense(bias, "bias", x.dtype, (C,))
    if state.dim() != 3:
        raise ValueError("state must be [slots, W - 1, C]")
    _dense(state, "state", x.dtype, (state.shape[0], W - 1, C))
    if slots is not None:
        _dense(slots, "slots", torch.int32, (nseq,))
    if out is not None:
        _dense(out, "out", x.dtype, x.shape)
    shape = tuple(x.shape)
    return ((_row_stride(x, "x", x.dim() - 1), state.shape[0], C), (W, _TORCH_TO_Q1.get(x.dtype, -1)), shape,
            _dense_strides(shape), x.get_device())


def _conv(x, weight, state, bias, slots, nseq, silu, out, cu_seqlens):
    key = (_layout(x), _layout(weight), _layout(state), _layout(bias), _layout(slots), _layout(out), _layout(cu_seqlens),
           nseq, _d._device())
    found = _conv_layouts.get(key)
    if found is None:
        found = _keep(_conv_layouts, key, _check_conv(x, weight, state, bias, slots, nseq, out, cu_seqlens))
    longs, ints, shape, strides, index = found
    if out is None:
        out = _new(shape, strides, dtype=x.dtype, device=x.device)
    return _CONV_PACK(x.data_ptr(), weight.data_ptr(), _addr(bias), state.data_ptr(), _addr(slots), out.data_ptr(),
                      *longs, *ints, 1 if silu else 0, 0), out, index


def q1_conv_step(x: torch.Tensor, weight: torch.Tensor, state: torch.Tensor, bias: Optional[torch.Tensor] = None,
                 slots: Optional[torch.Tensor] = None, silu: bool = True,
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Short causal convolution for T tokens of each of B sequences; returns out
    ``[B, T, C]`` and advances ``state`` in place.

    x ``[B, T, C]`` bf16 or fp16 (rows evenly spaced), weight ``[C, W]`` (W 2 to 4, the
    last for the token itself), bias ``[C]`` and state ``[slots, W - 1, C]`` (the last
    rows, oldest first) of the same dtype; slots int32 ``[B]``, distinct (default: sequence b
    uses state b; outside the states: zeros, and no state touched)."""
    if x.dim() != 3:
        raise ValueError("x must be [B, T, C]")
    d, out, index = _conv(x, weight, state, bias, slots, x.shape[0], silu, out, None)
    status = load_library().q1_conv_step(d, x.shape[0], x.shape[1], _d._stream_of(index))
    if status:
        _check(status)
    return out


def q1_conv_prefill(x: torch.Tensor, weight: torch.Tensor, state: torch.Tensor, cu_seqlens: torch.Tensor,
                    bias: Optional[torch.Tensor] = None, slots: Optional[torch.Tensor] = None, silu: bool = True,
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Short causal convolution over whole prompts packed along the rows: as
    ``q1_conv_step`` with x ``[tokens, C]`` and cu_seqlens int32 ``[nseq + 1]`` on the
    device."""
    if x.dim() != 2:
        raise ValueError("x must be [tokens, C]")
    nseq = cu_seqlens.numel() - 1
    d, out, index = _conv(x, weight, state, bias, slots, nseq, silu, out, cu_seqlens)
    status = load_library().q1_conv_prefill(d, x.shape[0], nseq, cu_seqlens.data_ptr(), _d._stream_of(index))
    if status:
        _check(status)
    return out


_scan_layouts = {}
_scan_needs = {}


def _check_scan(x, dt, A, B, C, state, D, z, dt_bias, slots, nseq, out, out_dtype, cu_seqlens):
    _same_device(x, dt=dt, A=A, B=B, C=C, state=state, D=D, z=z, dt_bias=dt_bias, slots=slots, out=out,
                 cu_seqlens=cu_seqlens)
    if cu_seqlens is not None:
        _check_cu(cu_seqlens)
    lead, Di = x.dim() - 1, x.shape[-1]
    if A.dim() != 2:
        raise ValueError("A must be [Di, N]")
    N = A.shape[1]
    _dense(A, "A", torch.float32, (Di, N))
    _dense(D, "D", torch.float32, (Di,))
    _dense(dt_bias, "dt_bias", torch.float32, (Di,))
    if state.dim() != 3:
        raise ValueError("state must be [slots, Di, N]")
    _dense(state, "state", torch.float32, (state.shape[0], Di, N))
    if slots is not None:
        _dense(slots, "slots", torch.int32, (nseq,))
    rows = tuple(x.shape[:lead])
    for name, t, width in (("dt", dt, Di), ("B", B, N), ("C", C, N), ("z", z, Di)):
        if t is not None and tuple(t.shape) != (*rows, width):
            raise ValueError(f"{name} must have shape {(*rows, width)}, not {tuple(t.shape)}")
        if t is not None and t.dtype != x.dtype and (name != "dt" or t.dtype != torch.float32):
            raise ValueError(f"{name} is {t.dtype}, x {x.dtype}")
    if out is not None:
        _dense(out, "out", out.dtype if out_dtype is None else out_dtype, x.shape)
        out_dtype = out.dtype
    elif out_dtype is None:
        out_dtype = x.dtype
    shape = tuple(x.shape)
    lds = [_row_stride(t, name, lead) for name, t in (("x", x), ("dt", dt), ("B", B), ("C", C))]
    return ((*lds, 0 if z is None else _row_stride(z, "z", lead), state.shape[0], Di),
            (N, _TORCH_TO_Q1.get(x.dtype, -1), _TORCH_TO_Q1.get(dt.dtype, -1), _TORCH_TO_Q1.get(out_dtype, -1)),
            out_dtype, shape, _dense_strides(shape), x.get_device())


def _scan(x, dt, A, B, C, state, D, z, dt_bias, softplus, slots, nseq, out, out_dtype, cu_seqlens):
    key = (_layout(x), _layout(dt), _layout(A), _layout(B), _layout(C), _layout(state), _layout(D), _layout(z),
           _layout(dt_bias), _layout(slots), _layout(out), _layout(cu_seqlens), nseq, out_dtype, _d._device())
    found = _scan_layouts.get(key)
    if found is None:
        found = _keep(_scan_layouts, key,
                      _check_scan(x, dt, A, B, C, state, D, z, dt_bias, slots, nseq, out, out_dtype, cu_seqlens))
    longs, ints, dtype, shape, strides, index = found
    if out is None:
        out = _new(shape, strides, dtype=dtype, device=x.device)
    d = _SCAN_PACK(x.data_ptr(), dt.data_ptr(), B.data_ptr(), C.data_ptr(), _addr(z), A.data_ptr(), _addr(D),
                   _addr(dt_bias), state.data_ptr(), _addr(slots), out.data_ptr(), *longs, *ints, 1 if softplus else 0, 0)
    return d, out, index, (longs[6], ints)


def q1_scan_step(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                 state: torch.Tensor, D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                 dt_bias: Optional[torch.Tensor] = None, softplus: bool = True, slots: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """Selective state space scan for T tokens of each of B sequences; returns out
    ``[B, T, Di]`` and advances ``state`` in place.

    x, z ``[B, T, Di]`` and B, C ``[B, T, N]`` bf16 or fp16, dt ``[B, T, Di]`` of their
    dtype or fp32 (rows evenly spaced: slices of one projection's rows will do); A
    fp32 ``[Di, N]`` (negative), D and dt_bias fp32 ``[Di]``; state fp32 ``[slots, Di,
    N]``; slots int32 ``[B]``, distinct (default: sequence b uses state b; outside the
    states: zeros, and no state touched)."""
    if x.dim() != 3:
        raise ValueError("x must be [B, T, Di]")
    d, out, index, _ = _scan(x, dt, A, B, C, state, D, z, dt_bias, softplus, slots, x.shape[0], out, out_dtype, None)
    status = load_library().q1_scan_step(d, x.shape[0], x.shape[1], _d._stream_of(index))
    if status:
        _check(status)
    return out


def q1_scan_prefill(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                    state: torch.Tensor, cu_seqlens: torch.Tensor, D: Optional[torch.Tensor] = None,
                    z: Optional[torch.Tensor] = None, dt_bias: Optional[torch.Tensor] = None, softplus: bool = True,
                    slots: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                    out_dtype: Optional[torch.dtype] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Selective state space scan over whole prompts packed along the rows: as
    ``q1_scan_step`` with x, dt, z ``[tokens, Di]``, B, C ``[tokens, N]`` and cu_seqlens
    int32 ``[nseq + 1]`` on the device."""
    if x.dim() != 2:
        raise ValueError("x must be [tokens, Di]")
    nseq, tokens = cu_seqlens.numel() - 1, x.shape[0]
    d, out, index, kind = _scan(x, dt, A, B, C, state, D, z, dt_bias, softplus, slots, nseq, out, out_dtype, cu_seqlens)
    L = load_library()
    stream = _d._stream_of(index)
    if workspace is None:
        need = _scan_needs.get((tokens, nseq, kind, index))
        if need is None:
            need = _keep(_scan_needs, (tokens, nseq, kind, index), L.q1_scan_prefill_workspace_bytes(d, tokens, nseq))
        workspace = _d._workspace(need, index, stream) if need else None
    else:
        _given(workspace, index)
    status = L.q1_scan_prefill(d, tokens, nseq, cu_seqlens.data_ptr(), _ptr(workspace),
                               0 if workspace is None else workspace.numel(), stream)
    if status:
        _check(status)
    return out
