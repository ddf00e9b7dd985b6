"""Binding of the decode-step operators (see ``include/q1_decode.h``): the gated
delta rule, attention over a shared prefix and the sampler.

Argument marshalling only, like ``q1.py``: every operation runs in the library's
HIP kernels on the current stream of its tensors' device.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional

import torch

from .q1 import _TORCH_TO_Q1, _check, _stream, load_library


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


class _Scratch:
    """Device workspaces of these calls (no initial contents needed), one per
    (device, stream), grown on demand."""

    def __init__(self):
        self._ws = {}

    def get(self, nbytes: int, device: torch.device) -> torch.Tensor:
        key = (device.index, _stream(device).value)
        t = self._ws.get(key)
        if t is None or t.numel() < nbytes:
            t = torch.empty(max(nbytes, 1 << 16), dtype=torch.uint8, device=device)
            self._ws[key] = t
        return t


_SCRATCH = _Scratch()


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


def _delta(q, k, v, g, beta, state, slots, nseq, scale, l2norm, out, out_dtype):
    _same_device(q, k=k, v=v, g=g, beta=beta, state=state, slots=slots, out=out)
    lead = q.dim() - 2
    rows, Hk, Dk = q.shape[:lead], q.shape[-2], q.shape[-1]
    Hv, Dv = v.shape[-2], v.shape[-1]
    if k.shape != q.shape:
        raise ValueError(f"k has shape {tuple(k.shape)}, q {tuple(q.shape)}")
    if v.dim() != q.dim() or v.shape[:lead] != rows:
        raise ValueError(f"v has shape {tuple(v.shape)}, q {tuple(q.shape)}")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k and v must have one dtype")
    _dense(g, "g", torch.float32, (*rows, Hv))
    _dense(beta, "beta", torch.float32, (*rows, Hv))
    _dense(state, "state", torch.float32, (state.shape[0], Hv, Dk, Dv))
    if slots is not None:
        _dense(slots, "slots", torch.int32, (nseq,))
    if out is None:
        out = torch.empty(v.shape, dtype=v.dtype if out_dtype is None else out_dtype, device=v.device)
    else:
        _dense(out, "out", out.dtype if out_dtype is None else out_dtype, v.shape)
    d = _Delta(q.data_ptr(), k.data_ptr(), v.data_ptr(), _row_stride(q, "q", lead), _row_stride(k, "k", lead),
               _row_stride(v, "v", lead), g.data_ptr(), beta.data_ptr(), state.data_ptr(), _ptr(slots), out.data_ptr(),
               state.shape[0], Hk, Hv, Dk, Dv, _TORCH_TO_Q1.get(q.dtype, -1), _TORCH_TO_Q1.get(out.dtype, -1),
               1 if l2norm else 0, Dk ** -0.5 if scale is None else scale)
    return d, out


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
    d, out = _delta(q, k, v, g, beta, state, slots, B, scale, l2norm, out, out_dtype)
    _check(load_library().q1_delta_step(ctypes.byref(d), B, T, _stream(q.device)))
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
    nseq = cu_seqlens.numel() - 1
    _dense(cu_seqlens, "cu_seqlens", torch.int32, (nseq + 1,))
    _same_device(q, cu_seqlens=cu_seqlens)
    d, out = _delta(q, k, v, g, beta, state, slots, nseq, scale, l2norm, out, out_dtype)
    L = load_library()
    need = L.q1_delta_prefill_workspace_bytes(ctypes.byref(d), q.shape[0], nseq)
    ws = workspace if workspace is not None else (_SCRATCH.get(need, q.device) if need else None)
    _check(L.q1_delta_prefill(ctypes.byref(d), q.shape[0], nseq, cu_seqlens.data_ptr(), _ptr(ws),
                              0 if ws is None else ws.numel(), _stream(q.device)))
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
        if P > 1 and _row_stride(v_prefix, "v_prefix", 1) != prefix_ld:
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
    if out is None:
        out = torch.empty(B, Hq, D, dtype=q.dtype if out_dtype is None else out_dtype, device=q.device)
    else:
        _dense(out, "out", out.dtype if out_dtype is None else out_dtype, (B, Hq, D))
    if lse is None:
        lse = torch.empty(B, Hq, dtype=torch.float32, device=q.device)
    else:
        _dense(lse, "lse", torch.float32, (B, Hq))
    a = _Attn(q.data_ptr(), _ptr(k_prefix) if P else None, _ptr(v_prefix) if P else None,
              _ptr(k_pages) if pages else None, _ptr(v_pages) if pages else None,
              _ptr(page_table) if max_pages else None, _ptr(suffix_lens) if max_pages else None, out.data_ptr(),
              lse.data_ptr(), _row_stride(q, "q", 1), prefix_ld, B, P, pages, max_pages, page_size, Hq, Hkv, D,
              _TORCH_TO_Q1.get(q.dtype, -1), _TORCH_TO_Q1.get(out.dtype, -1),
              1.0 / math.sqrt(D) if scale is None else scale)
    L = load_library()
    need = L.q1_prefix_attn_workspace_bytes(ctypes.byref(a))
    ws = workspace if workspace is not None else (_SCRATCH.get(need, q.device) if need else None)
    _check(L.q1_prefix_attn(ctypes.byref(a), _ptr(ws), 0 if ws is None else ws.numel(), _stream(q.device)))
    return out, lse


def q1_sample(logits: torch.Tensor, u: torch.Tensor, temperature: Optional[torch.Tensor] = None,
              top_k: Optional[torch.Tensor] = None, top_p: Optional[torch.Tensor] = None,
              min_p: Optional[torch.Tensor] = None, tokens: Optional[torch.Tensor] = None,
              logprob: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """One token per row of ``logits [B, V]`` (fp32, bf16 or fp16; rows may be
    spaced) from random numbers ``u`` fp32 ``[B]`` in [0, 1): returns (tokens
    ``[B]`` int64, or the dtype of ``tokens``; logprob fp32 ``[B]``).  The
    filters are per row: temperature, top_p, min_p fp32 and top_k int32, all
    ``[B]`` on the device, or None for off."""
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
    if tokens is None:
        tokens = torch.empty(B, dtype=torch.int64, device=logits.device)
    elif tokens.dtype not in (torch.int32, torch.int64):
        raise ValueError("tokens must be int32 or int64")
    else:
        _dense(tokens, "tokens", tokens.dtype, (B,))
    if logprob is None:
        logprob = torch.empty(B, dtype=torch.float32, device=logits.device)
    else:
        _dense(logprob, "logprob", torch.float32, (B,))
    L = load_library()
    need = L.q1_sample_workspace_bytes(B, V)
    ws = workspace if workspace is not None else (_SCRATCH.get(need, logits.device) if need else None)
    _check(L.q1_sample(logits.data_ptr(), _TORCH_TO_Q1.get(logits.dtype, -1), B, V, _row_stride(logits, "logits", 1),
                       u.data_ptr(), _ptr(temperature), _ptr(top_k), _ptr(top_p), _ptr(min_p), tokens.data_ptr(),
                       1 if tokens.dtype == torch.int64 else 0, logprob.data_ptr(), _ptr(ws),
                       0 if ws is None else ws.numel(), _stream(logits.device)))
    return tokens, logprob
