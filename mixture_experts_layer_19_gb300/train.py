"""Training operators around the MoE layer: layer norm, and the loss head
(cross entropy over a large vocabulary, distillation from a teacher's top
logits) whose logits are never stored.

Each operator comes as a pair of plain functions (``*_forward``,
``*_backward``), as an autograd function, and as a module:

    h = train.layer_norm(x, w, b)                      train.LayerNorm(d)
    loss = train.linear_cross_entropy(X, W, labels)    train.LMHead(d, V)
    loss = train.linear_distillation(X, W, teacher_logits, teacher_ids, temperature)

Losses are per token (fp32 [T]); reduce them as the training loop wants.
Argument marshalling only: the kernels are libmoe.so's, and the formulas and
error rules are those of include/moe.h.  Workspace comes from torch's caching
allocator for each call, on the stream the call runs on; a step can be
captured in a CUDA graph after one call outside the capture.  Tensors are
contiguous CUDA tensors, 16-byte aligned; ValueError says what is wrong with
an argument before anything is enqueued.  The differentiable functions and the
modules first copy activations, targets, gradients and norm weights laid out
otherwise.

With `stream=` a call runs there and its outputs belong to that stream.  The
caller makes it wait for what produces the inputs, and waits for it before
using the outputs (which are dropped as torch has it: after record_stream where
another stream reads them).  Inputs may be dropped right after the call.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import moe
from .moe import MOE_DEBUG_STALL_TEST, moe_head_config_t  # noqa: F401  (MOE_DEBUG_STALL_TEST: tests)

_BF16, _F32 = torch.bfloat16, torch.float32
_I32, _I64 = torch.int32, torch.int64
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _check(status: int, where: str) -> None:
    if status != moe.MOE_OK:
        raise moe.MoEError(status, where)


def _device_of(t: torch.Tensor, name: str) -> int:
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name}: expected a CUDA tensor, got one on {t.device}")
    return index


def _ptr(t: torch.Tensor, name: str, index: int, align: int = 16) -> int:
    """The address of a contiguous tensor on GPU `index`, aligned to `align` bytes."""
    p = t.data_ptr()
    if p % align or t.get_device() != index or not t.is_contiguous():
        if t.get_device() != index:
            raise ValueError(f"{name}: expected a tensor on cuda:{index}, got {t.device}")
        if not t.is_contiguous():
            raise ValueError(f"{name}: must be contiguous")
        raise ValueError(f"{name}: must be {align}-byte aligned")
    return p


def _dense(t: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    """t as the library takes it: contiguous, 16-byte aligned, copied where it is not.  The gradient of a
    part of a tensor, as cat and split hand it back, is a contiguous view that starts anywhere."""
    if t is None:
        return None
    t = t.contiguous()
    return t.clone() if t.data_ptr() % 16 else t


def _strided(t: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    """t as the library takes what it reads element by element: contiguous."""
    return None if t is None else t.contiguous()


def _elsewhere(index: int, stream: Optional[torch.cuda.Stream], *inputs: Optional[torch.Tensor]):
    """The context a call has to run in when that is not the current one: the given stream, or the
    tensors' GPU.  Outputs and workspace are then allocated there too, and the memory of the inputs is not
    handed out again, should the caller drop them, before the given stream is done with them."""
    if stream is not None:
        if stream.device_index != index:
            raise ValueError(f"stream: on cuda:{stream.device_index}, the tensors are on cuda:{index}")
        for t in inputs:
            if t is not None:
                t.record_stream(stream)
        return torch.cuda.stream(stream)
    if index != torch.cuda.current_device():
        return torch.cuda.device(index)
    return None


def _workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


_status = {}


def _status_word(index: int) -> Optional[torch.Tensor]:
    """One device word per GPU that receives a kernel's timeout code.  (It cannot be made while the
    stream is being captured: a graph captured before any other call reports no timeouts.)"""
    s = _status.get(index)
    if s is None:
        if torch.cuda.is_current_stream_capturing():
            return None
        s = torch.zeros((1,), dtype=_I32, device=torch.device("cuda", index))
        torch.cuda.current_stream(index).synchronize()   # zeroed before any stream's kernels use it
        _status[index] = s
    return s


def _status_ptr(index: int) -> Optional[int]:
    s = _status_word(index)
    return None if s is None else s.data_ptr()


def device_status(device=0) -> int:
    """Waits for the GPU, returns the status the loss head's kernels left there (0, or
    moe.MOE_ERR_TIMEOUT after a device-side wait expired) and clears it."""
    index = device if isinstance(device, int) else torch.device(device).index
    s = _status_word(torch.cuda.current_device() if index is None else index)
    torch.cuda.synchronize(s.device)
    code = int(s.item())
    if code:
        s.zero_()
        torch.cuda.synchronize(s.device)
    return code


# ------------------------------------------------------------------ layer norm
def _ln_args(x, weight):
    if x is None or weight is None:
        raise ValueError("x and weight are required")
    if x.dtype is not _BF16 and x.dtype is not _F32:
        raise ValueError(f"x: dtype {x.dtype}, expected torch.bfloat16 or torch.float32")
    if weight.dtype is not _BF16 and weight.dtype is not _F32:
        raise ValueError(f"weight: dtype {weight.dtype}, expected torch.bfloat16 or torch.float32")
    shape = x.shape
    if not shape or not shape[-1]:
        raise ValueError(f"x: shape {tuple(shape)}, expected a last dimension that is not empty")
    d = shape[-1]
    if weight.shape != (d,):
        raise ValueError(f"weight: shape {tuple(weight.shape)}, expected {(d,)}")
    return shape, x.numel() // d, d


def layer_norm_forward(x, weight, bias=None, eps: float = 1e-5, stream=None
                       ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """y = (x - mean) rstd weight + bias over the last dimension; returns (y, mean, rstd).

    x: bf16 or fp32, y likewise; weight and bias: both bf16 or both fp32; mean
    and rstd: fp32 of x's leading shape."""
    shape, rows, d = _ln_args(x, weight)
    index = _device_of(x, "x")
    xp, wp, bp = _ptr(x, "x", index), _ptr(weight, "weight", index), None
    if bias is not None:
        if bias.dtype is not weight.dtype or bias.shape != (d,):
            raise ValueError(f"bias: expected {weight.dtype} of shape {(d,)}, got {bias.dtype} of {tuple(bias.shape)}")
        bp = _ptr(bias, "bias", index)
    there = _elsewhere(index, stream, x, weight, bias)
    if there is not None:
        with there:
            return layer_norm_forward(x, weight, bias, eps)
    y = torch.empty_like(x)
    mean = torch.empty(shape[:-1], dtype=_F32, device=x.device)
    rstd = torch.empty_like(mean)
    _check(moe.lib().moe_layer_norm_forward(xp, wp, bp, rows, d, x.dtype is _F32, weight.dtype is _F32, eps,
                                            y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), _raw_stream(index)),
           "moe_layer_norm_forward")
    return y, mean, rstd


@functools.lru_cache(maxsize=1024)
def _ln_workspace_bytes(rows: int, d: int, index: int) -> int:
    n = ctypes.c_size_t()
    _check(moe.lib().moe_layer_norm_workspace_bytes(rows, d, ctypes.byref(n)), "moe_layer_norm_workspace_bytes")
    return n.value


def layer_norm_backward(dy, x, weight, mean, rstd, need_dx: bool = True, need_dweight: bool = True,
                        need_dbias: bool = True, stream=None):
    """(dx, dweight, dbias) of layer_norm_forward from its saved statistics; None for what is not needed."""
    shape, rows, d = _ln_args(x, weight)
    if dy is None or dy.dtype is not x.dtype or dy.shape != shape:
        raise ValueError(f"dy: expected {x.dtype} of shape {tuple(shape)}")
    for name, s in (("mean", mean), ("rstd", rstd)):
        if s is None or s.dtype is not _F32 or s.shape != shape[:-1]:
            raise ValueError(f"{name}: expected torch.float32 of shape {tuple(shape[:-1])}")
    index = _device_of(x, "x")
    args = (_ptr(dy, "dy", index), _ptr(x, "x", index), _ptr(weight, "weight", index), _ptr(mean, "mean", index, 4),
            _ptr(rstd, "rstd", index, 4))
    there = _elsewhere(index, stream, dy, x, weight, mean, rstd)
    if there is not None:
        with there:
            return layer_norm_backward(dy, x, weight, mean, rstd, need_dx, need_dweight, need_dbias)
    dx = torch.empty_like(x) if need_dx else None
    dw = torch.empty_like(weight) if need_dweight else None
    db = torch.empty_like(weight) if need_dbias else None
    n = _ln_workspace_bytes(rows, d, index)
    ws = _workspace(n, x.device)
    _check(moe.lib().moe_layer_norm_backward(
        *args, rows, d, x.dtype is _F32, weight.dtype is _F32, dx.data_ptr() if need_dx else None,
        dw.data_ptr() if need_dweight else None, db.data_ptr() if need_dbias else None, ws.data_ptr(), n,
        _raw_stream(index)), "moe_layer_norm_backward")
    return dx, dw, db


class _LayerNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        x, weight, bias = _dense(x), _dense(weight), _dense(bias)
        y, mean, rstd = layer_norm_forward(x, weight, bias, eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw, db = layer_norm_backward(_dense(dy), x, weight, mean, rstd, need_dx=need[0],
                                         need_dweight=need[1], need_dbias=need[2])
        return dx, dw, db, None


def layer_norm(x, weight, bias=None, eps: float = 1e-5) -> torch.Tensor:
    """Differentiable layer norm over the last dimension."""
    return _LayerNormFunction.apply(x, weight, bias, eps)


class LayerNorm(torch.nn.Module):
    """Layer norm over the last dimension d, weight 1 and bias 0 at the start (bias=False: none)."""

    def __init__(self, d: int, eps: float = 1e-5, bias: bool = True, dtype=_F32, device=0):
        super().__init__()
        dev = torch.device("cuda", device) if isinstance(device, int) else torch.device(device)
        self.eps = eps
        self.weight = torch.nn.Parameter(torch.ones((d,), dtype=dtype, device=dev))
        self.bias = torch.nn.Parameter(torch.zeros((d,), dtype=dtype, device=dev)) if bias else None

    def forward(self, x):
        return layer_norm(x, self.weight, self.bias, self.eps)


# ------------------------------------------------------------------ the loss head
def _head_args(X, W):
    for name, t in (("X", X), ("W", W)):
        if t is None or t.dtype is not _BF16 or t.dim() != 2:
            raise ValueError(f"{name}: expected a 2-d torch.bfloat16 tensor")
    (T, d), (V, dw) = X.shape, W.shape
    if d != dw:
        raise ValueError(f"W: width {dw}, X has {d}")
    return T, d, V


def _label_args(labels, T):
    if labels is None or (labels.dtype is not _I64 and labels.dtype is not _I32) or labels.shape != (T,):
        raise ValueError(f"labels: expected int32 or int64 of shape {(T,)}")


def _teacher_args(teacher, ids, T):
    if teacher is None or (teacher.dtype is not _F32 and teacher.dtype is not _BF16) or teacher.dim() != 2 or \
            teacher.shape[0] != T:
        raise ValueError(f"teacher_logits: expected a torch.float32 or torch.bfloat16 tensor of {T} rows")
    if ids is None or (ids.dtype is not _I64 and ids.dtype is not _I32) or ids.shape != teacher.shape:
        raise ValueError(f"teacher_ids: expected int32 or int64 of shape {tuple(teacher.shape)}")


def _row_vectors(T, dloss, lse):
    for name, t in (("dloss", dloss), ("lse", lse)):
        if t is None or t.dtype is not _F32 or t.shape != (T,):
            raise ValueError(f"{name}: expected torch.float32 of shape {(T,)}")


@functools.lru_cache(maxsize=1024)
def _head_workspace_bytes(T, V, d, K, piece, backward, index) -> int:
    """K = 0: cross entropy."""
    cfg = moe_head_config_t(T, V, d, K, 1.0, 0, 0, piece, 0, 0)
    n = ctypes.c_size_t()
    _check(moe.lib().moe_head_workspace_bytes(ctypes.byref(cfg), K > 0, backward, ctypes.byref(n)),
           "moe_head_workspace_bytes")
    return n.value


def head_info(T: int, V: int, d: int, K: int = 0, backward: bool = False, piece: int = 0) -> dict:
    """How a call of these sizes is laid out on the current GPU (K = 0: cross entropy), as moe_head_info states it."""
    cfg = moe_head_config_t(T, V, d, K, 1.0, 0, 0, piece, 0, 0)
    plan = (ctypes.c_int32 * 6)()
    _check(moe.lib().moe_head_info(ctypes.byref(cfg), K > 0, backward, plan), "moe_head_info")
    return dict(zip(("logits_ctas", "dX_ctas", "dW_ctas", "logits_columns", "dX_splits", "pieces"), plan))


def _ids_align(t) -> int:
    return 8 if t.dtype is _I64 else 4


def cross_entropy_forward(X, W, labels, stream=None, wait_timeout_ns: int = 0, debug_flags: int = 0):
    """(loss, lse), both fp32 [T]: loss_t = lse_t - z_t[labels_t] with z = X W^T.

    X bf16 [T, d], W bf16 [V, d], d a multiple of 8; labels int32 or int64
    [T].  A label outside [0, V) marks a token without a loss (0, and lse 0)."""
    T, d, V = _head_args(X, W)
    _label_args(labels, T)
    index = _device_of(X, "X")
    args = (_ptr(X, "X", index), _ptr(W, "W", index), _ptr(labels, "labels", index, _ids_align(labels)))
    there = _elsewhere(index, stream, X, W, labels)
    if there is not None:
        with there:
            return cross_entropy_forward(X, W, labels, None, wait_timeout_ns, debug_flags)
    cfg = moe_head_config_t(T, V, d, 0, 1.0, labels.dtype is _I64, 0, 0, wait_timeout_ns, debug_flags)
    return _head_forward(moe.lib().moe_cross_entropy_forward, "moe_cross_entropy_forward", cfg, X, args, index)


def _head_forward(call, name, cfg, X, args, index):
    loss = torch.empty(cfg.T, dtype=_F32, device=X.device)
    lse = torch.empty_like(loss)
    n = _head_workspace_bytes(cfg.T, cfg.V, cfg.d, cfg.K, 0, False, index)
    ws = _workspace(n, X.device)
    _check(call(ctypes.byref(cfg), *args, loss.data_ptr(), lse.data_ptr(), ws.data_ptr(), n,
                _status_ptr(index), _raw_stream(index)), name)
    return loss, lse


def cross_entropy_backward(dloss, X, W, labels, lse, need_dX: bool = True, need_dW: bool = True, piece: int = 0,
                           stream=None, wait_timeout_ns: int = 0, debug_flags: int = 0):
    """(dX, dW) bf16 for the upstream gradient dloss fp32 [T] and the forward's lse; None for what is not needed.

    `piece`: vocabulary columns handled at a time (0: as many as take 256 MB of
    workspace, but no fewer than 8192, which take 16 KB per token)."""
    T, d, V = _head_args(X, W)
    _label_args(labels, T)
    _row_vectors(T, dloss, lse)
    index = _device_of(X, "X")
    args = (_ptr(dloss, "dloss", index, 4), _ptr(X, "X", index), _ptr(W, "W", index),
            _ptr(labels, "labels", index, _ids_align(labels)), _ptr(lse, "lse", index, 4))
    there = _elsewhere(index, stream, dloss, X, W, labels, lse)
    if there is not None:
        with there:
            return cross_entropy_backward(dloss, X, W, labels, lse, need_dX, need_dW, piece, None, wait_timeout_ns,
                                          debug_flags)
    cfg = moe_head_config_t(T, V, d, 0, 1.0, labels.dtype is _I64, 0, piece, wait_timeout_ns, debug_flags)
    return _head_backward(moe.lib().moe_cross_entropy_backward, "moe_cross_entropy_backward", cfg, X, W, args, need_dX,
                          need_dW, index)


def _head_backward(call, name, cfg, X, W, args, need_dX, need_dW, index):
    dX = torch.empty_like(X) if need_dX else None
    dW = torch.empty_like(W) if need_dW else None
    n = _head_workspace_bytes(cfg.T, cfg.V, cfg.d, cfg.K, cfg.piece, True, index)
    ws = _workspace(n, X.device)
    _check(call(ctypes.byref(cfg), *args, dX.data_ptr() if need_dX else None, dW.data_ptr() if need_dW else None,
                ws.data_ptr(), n, _status_ptr(index), _raw_stream(index)), name)
    return dX, dW


def distill_forward(X, W, teacher_logits, teacher_ids, temperature: float = 1.0, stream=None,
                    wait_timeout_ns: int = 0, debug_flags: int = 0):
    """(loss, lse), both fp32 [T]: temperature^2 times the divergence of the student's softmax over the
    vocabulary from the teacher's softmax over its K entries, both at the temperature.

    teacher_logits fp32 or bf16 [T, K], teacher_ids int32 or int64 [T, K].  An
    entry whose id is outside [0, V) or whose logit is -inf is not in use."""
    T, d, V = _head_args(X, W)
    _teacher_args(teacher_logits, teacher_ids, T)
    index = _device_of(X, "X")
    args = (_ptr(X, "X", index), _ptr(W, "W", index),
            _ptr(teacher_logits, "teacher_logits", index, teacher_logits.element_size()),
            _ptr(teacher_ids, "teacher_ids", index, _ids_align(teacher_ids)))
    there = _elsewhere(index, stream, X, W, teacher_logits, teacher_ids)
    if there is not None:
        with there:
            return distill_forward(X, W, teacher_logits, teacher_ids, temperature, None, wait_timeout_ns, debug_flags)
    cfg = moe_head_config_t(T, V, d, teacher_ids.shape[1], temperature, teacher_ids.dtype is _I64,
                            teacher_logits.dtype is _BF16, 0, wait_timeout_ns, debug_flags)
    return _head_forward(moe.lib().moe_distill_forward, "moe_distill_forward", cfg, X, args, index)


def distill_backward(dloss, X, W, teacher_logits, teacher_ids, lse, temperature: float = 1.0, need_dX: bool = True,
                     need_dW: bool = True, piece: int = 0, stream=None, wait_timeout_ns: int = 0,
                     debug_flags: int = 0):
    """(dX, dW) bf16 of distill_forward for the upstream gradient dloss fp32 [T]; None for what is not needed."""
    T, d, V = _head_args(X, W)
    _teacher_args(teacher_logits, teacher_ids, T)
    _row_vectors(T, dloss, lse)
    index = _device_of(X, "X")
    args = (_ptr(dloss, "dloss", index, 4), _ptr(X, "X", index), _ptr(W, "W", index),
            _ptr(teacher_logits, "teacher_logits", index, teacher_logits.element_size()),
            _ptr(teacher_ids, "teacher_ids", index, _ids_align(teacher_ids)), _ptr(lse, "lse", index, 4))
    there = _elsewhere(index, stream, dloss, X, W, teacher_logits, teacher_ids, lse)
    if there is not None:
        with there:
            return distill_backward(dloss, X, W, teacher_logits, teacher_ids, lse, temperature, need_dX, need_dW, piece,
                                    None, wait_timeout_ns, debug_flags)
    cfg = moe_head_config_t(T, V, d, teacher_ids.shape[1], temperature, teacher_ids.dtype is _I64,
                            teacher_logits.dtype is _BF16, piece, wait_timeout_ns, debug_flags)
    return _head_backward(moe.lib().moe_distill_backward, "moe_distill_backward", cfg, X, W, args, need_dX, need_dW,
                          index)


class _CrossEntropyFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, W, labels):
        X, labels = _dense(X), _strided(labels)
        loss, lse = cross_entropy_forward(X, W, labels)
        ctx.save_for_backward(X, W, labels, lse)
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss):
        X, W, labels, lse = ctx.saved_tensors
        dX, dW = cross_entropy_backward(dloss.contiguous(), X, W, labels, lse, need_dX=ctx.needs_input_grad[0],
                                        need_dW=ctx.needs_input_grad[1])
        return dX, dW, None


class _DistillFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, W, teacher_logits, teacher_ids, temperature):
        X, teacher_logits, teacher_ids = _dense(X), _strided(teacher_logits), _strided(teacher_ids)
        loss, lse = distill_forward(X, W, teacher_logits, teacher_ids, temperature)
        ctx.temperature = temperature
        ctx.save_for_backward(X, W, teacher_logits, teacher_ids, lse)
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss):
        X, W, teacher, ids, lse = ctx.saved_tensors
        dX, dW = distill_backward(dloss.contiguous(), X, W, teacher, ids, lse, ctx.temperature,
                                  need_dX=ctx.needs_input_grad[0], need_dW=ctx.needs_input_grad[1])
        return dX, dW, None, None, None


def _rows(X, **targets):
    """X [..., d] and what each of its rows is trained on, as matrices of that many rows."""
    if X is None or X.dim() == 2:                    # as they are
        return [X, *targets.values()]
    lead = X.shape[:-1]
    for name, t in targets.items():
        if t is None or t.shape[:len(lead)] != lead:
            raise ValueError(f"{name}: expected a shape that starts with {tuple(lead)}")
    n = lead.numel()
    return [t.reshape(n, *t.shape[len(lead):]) for t in (X, *targets.values())]


def linear_cross_entropy(X, W, labels) -> torch.Tensor:
    """Differentiable per-token loss fp32 [...] of the head W [V, d] on X [..., d] with labels [...]."""
    rows, labels = _rows(X, labels=labels)
    loss = _CrossEntropyFunction.apply(rows, W, labels)
    return loss if rows is X else loss.view(X.shape[:-1])


def linear_distillation(X, W, teacher_logits, teacher_ids, temperature: float = 1.0) -> torch.Tensor:
    """Differentiable per-token distillation loss fp32 [...] of X [..., d] from teacher logits and ids
    [..., K] (the teacher gets no gradient)."""
    rows, teacher_logits, teacher_ids = _rows(X, teacher_logits=teacher_logits, teacher_ids=teacher_ids)
    teacher_logits = None if teacher_logits is None else teacher_logits.detach()
    loss = _DistillFunction.apply(rows, W, teacher_logits, teacher_ids, temperature)
    return loss if rows is X else loss.view(X.shape[:-1])


class LMHead(torch.nn.Module):
    """The head's weight [V, d] (bf16, N(0, 1/d)) with its two losses.  Nothing here waits for the GPU: a
    training loop asks device_status() where it reads its loss."""

    def __init__(self, d: int, V: int, device=0):
        super().__init__()
        dev = torch.device("cuda", device) if isinstance(device, int) else torch.device(device)
        self.weight = torch.nn.Parameter(torch.empty((V, d), dtype=_BF16, device=dev))
        with torch.no_grad():
            self.weight.normal_(0.0, d ** -0.5)

    def forward(self, X, labels):
        return linear_cross_entropy(X, self.weight, labels)

    def distill(self, X, teacher_logits, teacher_ids, temperature: float = 1.0):
        return linear_distillation(X, self.weight, teacher_logits, teacher_ids, temperature)

    @torch.no_grad()
    def logits(self, X, A=None, B=None, adapter_ids=None, scale=None, dtype=_F32):
        """The logits [..., V] of X [..., d], with the tokens' low-rank adapters where given (serve.linear's
        arguments); adapter_ids [...].  No gradient: training uses the losses.  bf16 logits without adapters
        are a plain product, which torch's may do faster: serve.linear has figures."""
        from . import serve
        rows, ids = _rows(X, adapter_ids=adapter_ids) if A is not None else (_rows(X)[0], adapter_ids)
        z = serve.linear(_dense(rows), self.weight, A, B, _strided(ids), scale, out_dtype=dtype)
        return z if rows is X else z.view(*X.shape[:-1], z.shape[1])

    def sampling_logits(self, X, A=None, B=None, adapter_ids=None, scale=None, dtype=_F32, **processing):
        """logits() of X [T, d], processed in place: `processing` is serve.process_logits's history, penalties,
        biases and masks.  Both run on the current stream; there is no `stream=`."""
        from . import serve
        if "stream" in processing:
            raise ValueError("stream: both calls run on the current stream (torch.cuda.stream)")
        z = self.logits(X, A, B, adapter_ids, scale, dtype)
        return serve.process_logits(z, **processing, out=z)
