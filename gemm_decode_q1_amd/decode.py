"""Binding of the decode-step operators (see ``include/q1_decode.h``): the gated
delta rule, attention over a shared prefix and the sampler.

Argument marshalling only, like ``q1.py``: every operation runs in the library's
HIP kernels on the current stream of its tensors' device.  The calls are as short
as the kernels of a single token, so what the checks of the operands' shapes,
strides and types found is kept by those (never by a tensor or its address), and
descriptors are packed at once.
"""
from __future__ import annotations

import ctypes
import math
import struct
import threading
from typing import Optional

import torch

from .q1 import _TORCH_TO_Q1, _check, _raw_stream, load_library


class _Delta(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("q_ld", ctypes.c_int64), ("k_ld", ctypes.c_int64), ("v_ld", ctypes.c_int64),
                ("g", ctypes.c_void_p), ("beta", ctypes.c_void_p), ("state", ctypes.c_void_p),
                ("slot_ids", ctypes.c_void_p), ("out", ctypes.c_void_p), ("slots", ctypes.c_int64),
                ("Hk", ctypes.c_int32), ("Hv", ctypes.c_int32), ("Dk", ctypes.c_int32), ("Dv", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("l2norm", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class _Attn(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k_prefix", ctypes.c_void_p), ("v_prefix", ctypes.c_void_p),
                ("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("suffix_lens", ctypes.c_void_p), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("q_ld", ctypes.c_int64), ("prefix_ld", ctypes.c_int64), ("B", ctypes.c_int64), ("P", ctypes.c_int64),
                ("pages", ctypes.c_int64), ("max_pages", ctypes.c_int64), ("page_size", ctypes.c_int64),
                ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("D", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("scale", ctypes.c_float)]


_DELTA_PACK = struct.Struct("@3P3q5Pq7if").pack  # the fields of _Delta
_ATTN_PACK = struct.Struct("@9P7q5if").pack      # the fields of _Attn

_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_empty = torch.empty
_new = torch.empty_strided  # half the host time of torch.empty


def _stream_of(index: int) -> int:
    """The current HIP stream of a device."""
    return _raw_stream(index) if _raw_stream is not None else torch.cuda.current_stream(index).cuda_stream


class _Scratch(threading.local):
    """The workspaces of one thread, by (device, stream)."""

    def __init__(self):
        self.kept = {}


_scratch = _Scratch()
_KEEP = 64 << 20  # bytes that are kept; more is a call's own, whose time hides the allocator's
_capturing = torch.cuda.is_current_stream_capturing


def _workspace(nbytes: int, index: int, stream: int) -> torch.Tensor:
    """Device workspace of these calls (no initial contents needed): one per
    (thread, device, stream), grown on demand.  A call is several launches that hand
    data on through it, and another thread's launches may come between them on the
    same stream.  A large one (of a long prompt: 264 MB for 16384 tokens of 48 heads)
    goes back to torch's allocator after the call.  A call under graph capture gets
    one of its own, from the graph's memory: a shared one would be freed as it grows,
    and be used by replays on other streams."""
    if nbytes > _KEEP or _capturing():
        return _empty(nbytes, dtype=torch.uint8, device=torch.device("cuda", index))
    kept = _scratch.kept
    t = kept.get((index, stream))
    if t is None or t.numel() < nbytes:
        t = _empty(max(nbytes, 1 << 16), dtype=torch.uint8, device=torch.device("cuda", index))
        kept[index, stream] = t
    return t


def _given(workspace: torch.Tensor, index: int) -> torch.Tensor:
    """A workspace of the caller's: bytes, all of them there, on the operands' device."""
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.get_device() != index:
        raise ValueError("workspace must be a contiguous uint8 tensor on the operands' device")
    return workspace


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _same_device(first: torch.Tensor, **others):
    if not first.is_cuda:
        raise ValueError("the operands must be device tensors")
    dev = first.device
    for name, t in others.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, not on {dev}")
    if dev.index != torch.cuda.current_device():
        raise ValueError(f"the operands are on {dev}, the current device is {torch.cuda.current_device()}")


def _row_stride(t: torch.Tensor, name: str, lead: int) -> int:
    """Elements between the rows of ``t`` (its first ``lead`` dims flattened);
    the other dims must be dense."""
    inner = 1
    for i in range(t.dim() - 1, lead - 1, -1):
        if t.shape[i] != 1 and t.stride(i) != inner:
            raise ValueError(f"the last {t.dim() - lead} dimensions of {name} must be contiguous")
        inner *= t.shape[i]
    ld, rows = None, 1
    for i in range(lead - 1, -1, -1):
        if t.shape[i] == 1:
            continue
        if ld is None:
            ld = t.stride(i)
        elif t.stride(i) != ld * rows:
            raise ValueError(f"the rows of {name} must be evenly spaced")
        rows *= t.shape[i]
    return inner if ld is None else ld


def _dense(t: Optional[torch.Tensor], name: str, dtype, shape):
    if t is None:
        return
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _dense_strides(shape):
    """Strides of a contiguous tensor."""
    strides, n = [], 1
    for m in reversed(shape):
        strides.append(n)
        n *= m
    return tuple(reversed(strides))


def _check_delta(q, k, v, g, beta, state, slots, nseq, out, out_dtype):
    """The descriptor's fields that follow from the operands' layouts."""
    _same_device(q, k=k, v=v, g=g, beta=beta, state=state, slots=slots, out=out)
    lead = q.dim() - 2
    rows, Hk, Dk = q.shape[:lead], q.shape[-2], q.shape[-1]
    if k.shape != q.shape:
        raise ValueError(f"k has shape {tuple(k.shape)}, q {tuple(q.shape)}")
    if v.dim() != q.dim() or v.shape[:lead] != rows:
        raise ValueError(f"v has shape {tuple(v.shape)}, q {tuple(q.shape)}")
    Hv, Dv = v.shape[-2], v.shape[-1]
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k and v must have one dtype")
    _dense(g, "g", torch.float32, (*rows, Hv))
    _dense(beta, "beta", torch.float32, (*rows, Hv))
    if state.dim() != 4:
        raise ValueError("state must be [slots, Hv, Dk, Dv]")
    _dense(state, "state", torch.float32, (state.shape[0], Hv, Dk, Dv))
    if slots is not None:
        _dense(slots, "slots", torch.int32, (nseq,))
    if out is not None:
        _dense(out, "out", out.dtype if out_dtype is None else out_dtype, v.shape)
        out_dtype = out.dtype
    elif out_dtype is None:
        out_dtype = v.dtype
    lds = (_row_stride(q, "q", lead), _row_stride(k, "k", lead), _row_stride(v, "v", lead))
    return (lds, (state.shape[0], Hk, Hv, Dk, Dv, _TORCH_TO_Q1.get(q.dtype, -1), _TORCH_TO_Q1.get(out_dtype, -1)),
            out_dtype, Dk ** -0.5, q.get_device(), tuple(v.shape), _dense_strides(v.shape), v.device)


_delta_layouts = {}
_prefill_needs = {}


def _delta(q, k, v, g, beta, state, slots, nseq, scale, l2norm, out, out_dtype):
    key = (q.shape, q.stride(), q.dtype, k.shape, k.stride(), k.dtype, v.shape, v.stride(), v.dtype, g.shape,
           g.stride(), g.dtype, beta.shape, beta.stride(), beta.dtype, state.shape, state.stride(), state.dtype,
           q.get_device(), k.get_device(), v.get_device(), g.get_device(), beta.get_device(), state.get_device(),
           None if slots is None else (slots.shape, slots.stride(), slots.dtype, slots.get_device()), nseq,
           None if out is None else (out.shape, out.stride(), out.dtype, out.get_device()), out_dtype, _device())
    found = _delta_layouts.get(key)
    if found is None:
        found = _check_delta(q, k, v, g, beta, state, slots, nseq, out, out_dtype)
        if len(_delta_layouts) > 4096:
            _delta_layouts.clear()
        _delta_layouts[key] = found
    lds, ints, dtype, usual, index, shape, strides, device = found
    if out is None:
        out = _new(shape, strides, dtype=dtype, device=device)
    return _DELTA_PACK(q.data_ptr(), k.data_ptr(), v.data_ptr(), *lds, g.data_ptr(), beta.data_ptr(), state.data_ptr(),
                       0 if slots is None else slots.data_ptr(), out.data_ptr(), *ints, 1 if l2norm else 0,
                       usual if scale is None else scale), out, index, ints


def q1_delta_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                  state: torch.Tensor, slots: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                  l2norm: bool = False, out: Optional[torch.Tensor] = None,
                  out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """Gated delta rule for T tokens of each of B sequences; returns out
    ``[B, T, Hv, Dv]`` and advances ``state`` in place.

    q, k ``[B, T, Hk, Dk]``, v ``[B, T, Hv, Dv]`` bf16 or fp16 (rows evenly
    spaced: slices of one projection's rows will do); g (log decay) and beta
    fp32 ``[B, T, Hv]``; state fp32 ``[slots, Hv, Dk, Dv]``; slots int32 ``[B]``
    (default: sequence b uses state b).  ``scale`` defaults to Dk^-1/2."""
    if q.dim() != 4:
        raise ValueError("q must be [B, T, Hk, Dk]")
    B, T = q.shape[0], q.shape[1]
    d, out, index, _ = _delta(q, k, v, g, beta, state, slots, B, scale, l2norm, out, out_dtype)
    status = load_library().q1_delta_step(d, B, T, _stream_of(index))
    if status:
        _check(status)
    return out


def q1_delta_prefill(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                     state: torch.Tensor, cu_seqlens: torch.Tensor, slots: Optional[torch.Tensor] = None,
                     scale: Optional[float] = None, l2norm: bool = False, out: Optional[torch.Tensor] = None,
                     out_dtype: Optional[torch.dtype] = None,
                     workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gated delta rule over whole prompts packed along the rows: as
    ``q1_delta_step`` with q, k ``[tokens, Hk, Dk]``, v ``[tokens, Hv, Dv]``,
    g, beta ``[tokens, Hv]`` and cu_seqlens int32 ``[nseq + 1]`` on the device."""
    if q.dim() != 3:
        raise ValueError("q must be [tokens, Hk, Dk]")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be [nseq + 1]")
    nseq, tokens = cu_seqlens.numel() - 1, q.shape[0]
    if cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens must be contiguous int32")
    d, out, index, ints = _delta(q, k, v, g, beta, state, slots, nseq, scale, l2norm, out, out_dtype)
    if cu_seqlens.get_device() != index:
        raise ValueError(f"cu_seqlens is on {cu_seqlens.device}, q on {q.device}")
    L = load_library()
    stream = _stream_of(index)
    if workspace is None:
        need = _prefill_needs.get((tokens, nseq, ints))
        if need is None:
            if len(_prefill_needs) > 4096:
                _prefill_needs.clear()
            need = _prefill_needs[tokens, nseq, ints] = L.q1_delta_prefill_workspace_bytes(d, tokens, nseq)
        workspace = _workspace(need, index, stream) if need else None
    else:
        _given(workspace, index)
    status = L.q1_delta_prefill(d, tokens, nseq, cu_seqlens.data_ptr(), _ptr(workspace),
                                0 if workspace is None else workspace.numel(), stream)
    if status:
        _check(status)
    return out


def q1_delta_prefill_workspace_bytes(tokens: int, nseq: int, Hk: int, Hv: int, Dk: int, Dv: int,
                                     dtype: torch.dtype = torch.bfloat16) -> int:
    d = _Delta(Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv, dtype=_TORCH_TO_Q1.get(dtype, -1), out_dtype=_TORCH_TO_Q1.get(dtype, -1))
    return load_library().q1_delta_prefill_workspace_bytes(ctypes.byref(d), tokens, nseq)


def q1_prefix_attn(q: torch.Tensor, k_prefix: Optional[torch.Tensor], v_prefix: Optional[torch.Tensor],
                   k_pages: Optional[torch.Tensor] = None, v_pages: Optional[torch.Tensor] = None,
                   page_table: Optional[torch.Tensor] = None, suffix_lens: Optional[torch.Tensor] = None,
                   scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                   out_dtype: Optional[torch.dtype] = None, lse: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None):
    """One query per sequence over a prefix shared by the batch and its own paged
    suffix; returns (out ``[B, Hq, D]``, lse fp32 ``[B, Hq]``).

    q ``[B, Hq, D]`` bf16 or fp16; k_prefix, v_prefix ``[P, Hkv, D]`` (evenly
    spaced rows) or None; k_pages, v_pages ``[pages, page_size, Hkv, D]``,
    page_table int32 ``[B, max_pages]`` and suffix_lens int32 ``[B]``, or None.
    ``scale`` defaults to D^-1/2."""
    key = (q.shape, q.stride(), q.dtype, q.get_device(), out_dtype, _device(),
           None if k_prefix is None else (k_prefix.shape, k_prefix.stride(), k_prefix.dtype, k_prefix.get_device()),
           None if v_prefix is None else (v_prefix.shape, v_prefix.stride(), v_prefix.dtype, v_prefix.get_device()),
           None if k_pages is None else (k_pages.shape, k_pages.stride(), k_pages.dtype, k_pages.get_device()),
           None if v_pages is None else (v_pages.shape, v_pages.stride(), v_pages.dtype, v_pages.get_device()),
           None if page_table is None else (page_table.shape, page_table.stride(), page_table.dtype, page_table.get_device()),
           None if suffix_lens is None else (suffix_lens.shape, suffix_lens.stride(), suffix_lens.dtype, suffix_lens.get_device()),
           None if out is None else (out.shape, out.stride(), out.dtype, out.get_device()),
           None if lse is None else (lse.shape, lse.stride(), lse.dtype, lse.get_device()))
    found = _attn_layouts.get(key)
    if found is None:
        found = _check_attn(q, k_prefix, v_prefix, k_pages, v_pages, page_table, suffix_lens, out, out_dtype, lse)
    longs, ints, dtype, usual, index, shape, strides, device, need = found
    P, pages, max_pages = longs[3], longs[4], longs[5]
    if out is None:
        out = _new(shape, strides, dtype=dtype, device=device)
    if lse is None:
        lse = _new(shape[:2], (shape[1], 1), dtype=torch.float32, device=device)
    a = _ATTN_PACK(q.data_ptr(), k_prefix.data_ptr() if P else 0, v_prefix.data_ptr() if P else 0,
                   k_pages.data_ptr() if pages else 0, v_pages.data_ptr() if pages else 0,
                   page_table.data_ptr() if max_pages else 0, suffix_lens.data_ptr() if max_pages else 0,
                   out.data_ptr(), lse.data_ptr(), *longs, *ints, usual if scale is None else scale)
    L = load_library()
    stream = _stream_of(index)
    if need is None:  # a layout that is new: its workspace depends on nothing else
        need = L.q1_prefix_attn_workspace_bytes(a)
        if len(_attn_layouts) > 4096:
            _attn_layouts.clear()
        _attn_layouts[key] = (*found[:-1], need)
    if workspace is None:
        workspace = _workspace(need, index, stream) if need else None
    else:
        _given(workspace, index)
    status = L.q1_prefix_attn(a, _ptr(workspace), 0 if workspace is None else workspace.numel(), stream)
    if status:
        _check(status)
    return out, lse


_attn_layouts = {}


def _check_attn(q, k_prefix, v_prefix, k_pages, v_pages, page_table, suffix_lens, out, out_dtype, lse):
    """The descriptor's fields that follow from the operands' layouts."""
    if q.dim() != 3:
        raise ValueError("q must be [B, Hq, D]")
    _same_device(q, k_prefix=k_prefix, v_prefix=v_prefix, k_pages=k_pages, v_pages=v_pages, page_table=page_table,
                 suffix_lens=suffix_lens, out=out, lse=lse)
    B, Hq, D = q.shape
    if (k_prefix is None) != (v_prefix is None):
        raise ValueError("k_prefix and v_prefix go together")
    suffix = (k_pages, v_pages, page_table, suffix_lens)
    if any(t is None for t in suffix) != all(t is None for t in suffix):
        raise ValueError("k_pages, v_pages, page_table and suffix_lens go together")
    if k_prefix is None and k_pages is None:
        raise ValueError("give a prefix, pages or both")
    Hkv = (k_pages if k_prefix is None else k_prefix).shape[-2]
    P, prefix_ld = 0, Hkv * D
    if k_prefix is not None:
        if k_prefix.dim() != 3 or k_prefix.shape[1:] != (Hkv, D) or v_prefix.shape != k_prefix.shape:
            raise ValueError(f"k_prefix and v_prefix must be [P, {Hkv}, {D}]")
        P, prefix_ld = k_prefix.shape[0], _row_stride(k_prefix, "k_prefix", 1)
        if P > 0 and _row_stride(v_prefix, "v_prefix", 1) != prefix_ld and P > 1:  # (one row's stride is never used)
            raise ValueError("k_prefix and v_prefix must have the same row stride")
    pages = max_pages = page_size = 0
    if k_pages is not None:
        if k_pages.dim() != 4 or page_table.dim() != 2:
            raise ValueError("pages must be [pages, page_size, Hkv, D], page_table [B, max_pages]")
        pages, page_size, max_pages = k_pages.shape[0], k_pages.shape[1], page_table.shape[1]
        _dense(k_pages, "k_pages", q.dtype, (pages, page_size, Hkv, D))
        _dense(v_pages, "v_pages", q.dtype, (pages, page_size, Hkv, D))
        _dense(page_table, "page_table", torch.int32, (B, max_pages))
        _dense(suffix_lens, "suffix_lens", torch.int32, (B,))
    if any(t is not None and t.dtype != q.dtype for t in (k_prefix, v_prefix)):
        raise ValueError("q, keys and values must have one dtype")
    if out is not None:
        _dense(out, "out", out.dtype if out_dtype is None else out_dtype, (B, Hq, D))
        out_dtype = out.dtype
    elif out_dtype is None:
        out_dtype = q.dtype
    _dense(lse, "lse", torch.float32, (B, Hq))
    return ((_row_stride(q, "q", 1), prefix_ld, B, P, pages, max_pages, page_size),
            (Hq, Hkv, D, _TORCH_TO_Q1.get(q.dtype, -1), _TORCH_TO_Q1.get(out_dtype, -1)), out_dtype, 1.0 / math.sqrt(D),
            q.get_device(), (B, Hq, D), (Hq * D, D, 1), q.device, None)


def q1_sample(logits: torch.Tensor, u: torch.Tensor, temperature: Optional[torch.Tensor] = None,
              top_k: Optional[torch.Tensor] = None, top_p: Optional[torch.Tensor] = None,
              min_p: Optional[torch.Tensor] = None, tokens: Optional[torch.Tensor] = None,
              logprob: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """One token per row of ``logits [B, V]`` (fp32, bf16 or fp16; rows may be
    spaced) from random numbers ``u`` fp32 ``[B]`` in [0, 1): returns (tokens
    ``[B]`` int64, or the dtype of ``tokens``; logprob fp32 ``[B]``).  The
    filters are per row: temperature, top_p, min_p fp32 and top_k int32, all
    ``[B]`` on the device, or None for off."""
    key = (logits.shape, logits.stride(), logits.dtype, logits.get_device(), u.shape, u.stride(), u.dtype,
           u.get_device(), _device(),
           None if temperature is None else (temperature.shape, temperature.stride(), temperature.dtype, temperature.get_device()),
           None if top_k is None else (top_k.shape, top_k.stride(), top_k.dtype, top_k.get_device()),
           None if top_p is None else (top_p.shape, top_p.stride(), top_p.dtype, top_p.get_device()),
           None if min_p is None else (min_p.shape, min_p.stride(), min_p.dtype, min_p.get_device()),
           None if tokens is None else (tokens.shape, tokens.stride(), tokens.dtype, tokens.get_device()),
           None if logprob is None else (logprob.shape, logprob.stride(), logprob.dtype, logprob.get_device()))
    L = load_library()
    found = _sample_layouts.get(key)
    if found is None:
        found = _check_sample(L, logits, u, temperature, top_k, top_p, min_p, tokens, logprob)
        if len(_sample_layouts) > 4096:
            _sample_layouts.clear()
        _sample_layouts[key] = found
    B, V, ld, dtype, need, index, device = found
    if tokens is None:
        tokens = _new((B,), (1,), dtype=torch.int64, device=device)
    if logprob is None:
        logprob = _new((B,), (1,), dtype=torch.float32, device=device)
    stream = _stream_of(index)
    if workspace is None:
        workspace = _workspace(need, index, stream) if need else None
    else:
        _given(workspace, index)
    status = L.q1_sample(logits.data_ptr(), dtype, B, V, ld, u.data_ptr(), _ptr(temperature), _ptr(top_k), _ptr(top_p),
                         _ptr(min_p), tokens.data_ptr(), 1 if tokens.dtype == torch.int64 else 0, logprob.data_ptr(),
                         _ptr(workspace), 0 if workspace is None else workspace.numel(), stream)
    if status:
        _check(status)
    return tokens, logprob


_sample_layouts = {}


def _check_sample(L, logits, u, temperature, top_k, top_p, min_p, tokens, logprob):
    """What follows from the operands' layouts: (B, V, row stride, dtype, workspace bytes, device index, device)."""
    if logits.dim() != 2:
        raise ValueError("logits must be [B, V]")
    _same_device(logits, u=u, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p, tokens=tokens,
                 logprob=logprob)
    B, V = logits.shape
    _dense(u, "u", torch.float32, (B,))
    _dense(temperature, "temperature", torch.float32, (B,))
    _dense(top_k, "top_k", torch.int32, (B,))
    _dense(top_p, "top_p", torch.float32, (B,))
    _dense(min_p, "min_p", torch.float32, (B,))
    if tokens is not None:
        if tokens.dtype not in (torch.int32, torch.int64):
            raise ValueError("tokens must be int32 or int64")
        _dense(tokens, "tokens", tokens.dtype, (B,))
    _dense(logprob, "logprob", torch.float32, (B,))
    return (B, V, _row_stride(logits, "logits", 1), _TORCH_TO_Q1.get(logits.dtype, -1),
            L.q1_sample_workspace_bytes(B, V) if V > 0 else 0, logits.get_device(), logits.device)
