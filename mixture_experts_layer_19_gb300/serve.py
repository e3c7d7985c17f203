"""Operators behind the MoE layer when it serves: what turns a step's
activations into logits that can be sampled from.

    Y = layer.decode(x)                                   moe.RoutedMoELayer: the layer for up to 64 tokens
    z = serve.linear(f, W, A, B, adapter_ids, scale)      a projection with low-rank adapters (LMHead.logits)
    z = serve.process_logits(z, history, lengths, ...)    penalties, biases and grammar masks
                                                          (LMHead.sampling_logits: both)

Argument marshalling only, as in train.py: the kernels are libmoe.so's, the
formulas and error rules those of include/moe.h.  None of them has a gradient.
Calls run on the current stream of the tensors' GPU, or on `stream=` (with train.py's
rules), and can be captured in a CUDA graph.  ValueError says what is wrong with
an argument before anything is enqueued.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from . import moe
from .train import (_BF16, _F32, _I32, _I64, _check, _device_of, _elsewhere, _ids_align, _ptr, _raw_stream, _status_ptr,
                    _workspace)


def _rows(t: torch.Tensor, name: str, index: int, dtypes, T: int, cols: int):
    """(address, row stride) of a matrix with contiguous rows (any row stride) on GPU `index`."""
    if t.dtype not in dtypes or t.shape != (T, cols):
        raise ValueError(f"{name}: expected {' or '.join(map(str, dtypes))} of shape {(T, cols)}, "
                         f"got {t.dtype} of {tuple(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name}: expected a tensor on cuda:{index}, got {t.device}")
    across, along = t.stride()
    if along != 1 and cols > 1 or across < cols and T > 1:
        raise ValueError(f"{name}: rows must be contiguous and apart from each other")
    return t.data_ptr(), across if T > 1 else cols


def _vector(t: Optional[torch.Tensor], name: str, index: int, dtype, T: int) -> Optional[int]:
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != (T,):
        raise ValueError(f"{name}: expected {dtype} of shape {(T,)}, got {t.dtype} of {tuple(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name}: expected a tensor on cuda:{index}, got {t.device}")
    if T > 1 and t.stride(0) != 1:
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr()


_IDS = (_I32, _I64)


@functools.lru_cache(maxsize=1024)
def _linear_workspace_bytes(T, N, d, n, r, index) -> int:
    cfg = moe.moe_linear_config_t(T, N, d, n, r, 0, 0, 0, 0)
    nbytes = ctypes.c_size_t()
    _check(moe.lib().moe_linear_workspace_bytes(ctypes.byref(cfg), ctypes.byref(nbytes)), "moe_linear_workspace_bytes")
    return nbytes.value


def linear(X, W, A=None, B=None, adapter_ids=None, scale=None, out_dtype=_BF16, out=None, stream=None,
           wait_timeout_ns: int = 0, debug_flags: int = 0) -> torch.Tensor:
    """W x_t + scale_a B_a (A_a x_t) for each row t of X, a = adapter_ids[t] (outside [0, n): no adapter).

    X bf16 [T, d], W bf16 [N, d], d a multiple of 8; A bf16 [n, r, d], B bf16 [n, N, r], r a multiple of 8
    up to 256; adapter_ids int32 or int64 [T]; scale fp32 [n] (1 by default); without A, W alone.
    Returns [T, N] of out_dtype (bf16 or fp32), `out` where given.  A wait that expires on the GPU is
    reported by train.device_status().

    Made for adapters and for fp32 results; for bf16 ones without adapters X @ W.T is often as fast or
    faster (64 x 2048 x 32768: 26 us against 31 here; 4096 x 7168 x 2048: 68 against 78; slower where rows of
    the result start off 16 bytes, 777 x 1000 x 5001: 72 against 21)."""
    for name, t in (("X", X), ("W", W)):
        if t is None or t.dtype is not _BF16 or t.dim() != 2:
            raise ValueError(f"{name}: expected a 2-d torch.bfloat16 tensor")
    (T, d), N = X.shape, W.shape[0]
    if W.shape[1] != d:
        raise ValueError(f"W: width {W.shape[1]}, X has {d}")
    if out_dtype is not _BF16 and out_dtype is not _F32:
        raise ValueError(f"out_dtype: {out_dtype}, expected torch.bfloat16 or torch.float32")
    index = _device_of(X, "X")
    xp, wp = _ptr(X, "X", index), _ptr(W, "W", index)
    n = r = 0
    ap = bp = ip = sp = None
    if A is not None:
        if A.dtype is not _BF16 or A.dim() != 3 or A.shape[2] != d or not A.shape[0]:
            raise ValueError(f"A: expected torch.bfloat16 of shape (n, r, {d})")
        n, r = A.shape[:2]
        if B is None or B.dtype is not _BF16 or B.shape != (n, N, r):
            raise ValueError(f"B: expected torch.bfloat16 of shape {(n, N, r)}")
        if adapter_ids is None or (adapter_ids.dtype is not _I32 and adapter_ids.dtype is not _I64) or \
                adapter_ids.shape != (T,):
            raise ValueError(f"adapter_ids: expected int32 or int64 of shape {(T,)}")
        if scale is not None and (scale.dtype is not _F32 or scale.shape != (n,)):
            raise ValueError(f"scale: expected torch.float32 of shape {(n,)}")
        ap, bp = _ptr(A, "A", index), _ptr(B, "B", index)
        ip = _ptr(adapter_ids, "adapter_ids", index, _ids_align(adapter_ids))
        sp = None if scale is None else _ptr(scale, "scale", index, 4)
    elif B is not None or adapter_ids is not None or scale is not None:
        raise ValueError("B, adapter_ids and scale need A")
    if out is not None:
        if out.dtype is not out_dtype or out.shape != (T, N):
            raise ValueError(f"out: expected {out_dtype} of shape {(T, N)}")
        _ptr(out, "out", index, out.element_size())
    there = _elsewhere(index, stream, X, W, A, B, adapter_ids, scale, out)
    if there is not None:
        with there:
            return linear(X, W, A, B, adapter_ids, scale, out_dtype, out, None, wait_timeout_ns, debug_flags)
    if out is None:
        out = torch.empty((T, N), dtype=out_dtype, device=X.device)
    cfg = moe.moe_linear_config_t(T, N, d, n, r, out_dtype is _F32, n > 0 and adapter_ids.dtype is _I64,
                                  wait_timeout_ns, debug_flags)
    nbytes = _linear_workspace_bytes(T, N, d, n, r, index)
    ws = _workspace(nbytes, X.device)
    _check(moe.lib().moe_linear(ctypes.byref(cfg), xp, wp, ap, bp, ip, sp, out.data_ptr(), ws.data_ptr(), nbytes,
                                _status_ptr(index), _raw_stream(index)), "moe_linear")
    return out


def process_logits(logits, history=None, lengths=None, prompt_lengths=None, repetition=None, frequency=None,
                   presence=None, bias_ids=None, bias=None, mask=None, mask_rows=None, out=None, stream=None
                   ) -> torch.Tensor:
    """Penalties for tokens the history holds, biases of single tokens, and masks, on logits [T, V] fp32 or
    bf16; returns `out` (new by default; `logits` itself works in place).

    history int32 or int64 [T, L] with lengths and prompt_lengths int32 [T]; repetition, frequency,
    presence fp32 [T]; bias_ids int32 or int64 [T, K] with bias fp32 [T, K], K at most 1024; mask int32
    [G, ceil(V / 32)], bit v % 32 of word v // 32 allows column v, with mask_rows int32 [T] (row t for
    t by default, -1: no mask)."""
    if logits is None or logits.dim() != 2 or (logits.dtype is not _F32 and logits.dtype is not _BF16):
        raise ValueError("logits: expected a 2-d torch.float32 or torch.bfloat16 tensor")
    T, V = logits.shape
    dtype = logits.dtype
    index = _device_of(logits, "logits")
    if not V:
        raise ValueError("logits: no columns")
    zp, zs = _rows(logits, "logits", index, (dtype,), T, V)
    hp, hs, L, wide = None, 0, 0, False
    if history is not None:
        if history.dim() != 2:
            raise ValueError("history: expected a 2-d tensor")
        L, wide = history.shape[1], history.dtype is _I64
        hp, hs = _rows(history, "history", index, _IDS, T, L)
    elif not (lengths is None and prompt_lengths is None and repetition is None and frequency is None and
              presence is None):
        raise ValueError("lengths and penalties need a history")
    if (bias_ids is None) != (bias is None):
        raise ValueError("bias_ids and bias come together")
    bp, bs, ip, its, K, bias_wide = None, 0, None, 0, 0, False
    if bias is not None:
        if bias.dim() != 2:
            raise ValueError("bias: expected a 2-d tensor")
        K, bias_wide = bias.shape[1], bias_ids.dtype is _I64
        bp, bs = _rows(bias, "bias", index, (_F32,), T, K)
        ip, its = _rows(bias_ids, "bias_ids", index, _IDS, T, K)
    mp, ms, G = None, 0, 0
    if mask is not None:
        if mask.dim() != 2:
            raise ValueError("mask: expected a 2-d tensor")
        G = mask.shape[0]
        mp, ms = _rows(mask, "mask", index, (_I32,), G, -(-V // 32))
        if mask_rows is None and G != T:
            raise ValueError(f"mask: {G} rows for {T} rows of logits, and no mask_rows")
    elif mask_rows is not None:
        raise ValueError("mask_rows needs a mask")
    vectors = [_vector(lengths, "lengths", index, _I32, T), _vector(prompt_lengths, "prompt_lengths", index, _I32, T),
               _vector(repetition, "repetition", index, _F32, T), _vector(frequency, "frequency", index, _F32, T),
               _vector(presence, "presence", index, _F32, T)]
    rows = _vector(mask_rows, "mask_rows", index, _I32, T)
    op, os_ = (None, V) if out is None else _rows(out, "out", index, (dtype,), T, V)
    if stream is not None or index != torch.cuda.current_device():
        there = _elsewhere(index, stream, logits, history, lengths, prompt_lengths, repetition, frequency, presence,
                           bias_ids, bias, mask, mask_rows, out)
        with there:
            return process_logits(logits, history, lengths, prompt_lengths, repetition, frequency, presence, bias_ids,
                                  bias, mask, mask_rows, out)
    if out is None:
        out = torch.empty_like(logits) if logits.is_contiguous() else torch.empty((T, V), dtype=dtype, device=logits.device)
        op = out.data_ptr()
    a = moe.moe_logits_t(T, V, zp, op, zs, os_, dtype is _BF16, wide, bias_wide, hp, L, hs, *vectors, ip, bp, K, its, bs,
                         mp, G, ms, rows)
    _check(moe.lib().moe_process_logits(ctypes.byref(a), _raw_stream(index)), "moe_process_logits")
    return out
