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
allocator for each call, on the stream the call runs on.  Tensors are
contiguous CUDA tensors, 16-byte aligned; ValueError says what is wrong with
an argument before anything is enqueued.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional, Tuple

import torch

from . import moe
from .moe import MOE_DEBUG_STALL_TEST, moe_head_config_t  # noqa: F401  (MOE_DEBUG_STALL_TEST: tests)

_BF16, _F32 = torch.bfloat16, torch.float32


def _check(status: int, where: str) -> None:
    if status != moe.MOE_OK:
        raise moe.MoEError(status, where)


def _need(ok: bool, message: str) -> None:
    if not ok:
        raise ValueError(message)


def _cuda(device: torch.device, **tensors) -> None:
    """Every given tensor is a contiguous, 16-byte aligned tensor on `device`."""
    for name, t in tensors.items():
        if t is None:
            continue
        _need(t.is_cuda and t.device == device, f"{name}: expected a tensor on {device}, got {t.device}")
        _need(t.is_contiguous(), f"{name}: must be contiguous")
        _need(t.data_ptr() % 16 == 0, f"{name}: must be 16-byte aligned")


def _scope(device: torch.device, stream: Optional[torch.cuda.Stream]):
    """The device and stream a call runs on: outputs and workspace are allocated there too."""
    if stream is not None:
        return torch.cuda.stream(stream)
    if device.index is not None and device.index != torch.cuda.current_device():
        return torch.cuda.device(device)
    return contextlib.nullcontext()


def _stream(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _workspace(nbytes: int, device: torch.device) -> torch.Tensor:
    return torch.empty((nbytes,), dtype=torch.uint8, device=device)


_status = {}


def _status_word(device: torch.device) -> torch.Tensor:
    """One device word per GPU that receives a kernel's timeout code."""
    s = _status.get(device)
    if s is None:
        s = _status[device] = torch.zeros((1,), dtype=torch.int32, device=device)
        torch.cuda.current_stream(device).synchronize()   # zeroed before any stream's kernels use it
    return s


def device_status(device=0) -> int:
    """Waits for the GPU, returns the status the loss head's kernels left there (0, or
    moe.MOE_ERR_TIMEOUT after a device-side wait expired) and clears it."""
    dev = torch.device("cuda", device) if isinstance(device, int) else torch.device(device)
    s = _status_word(torch.device("cuda", dev.index if dev.index is not None else torch.cuda.current_device()))
    torch.cuda.synchronize(s.device)
    code = int(s.item())
    if code:
        s.zero_()
        torch.cuda.synchronize(s.device)
    return code


# ------------------------------------------------------------------ layer norm
def _ln_args(x, weight, other=()):
    _need(x is not None and x.dim() >= 1, "x: expected at least one dimension")
    _need(x.dtype in (_BF16, _F32), f"x: dtype {x.dtype}, expected torch.bfloat16 or torch.float32")
    d = x.shape[-1]
    _need(d >= 1, "x: the last dimension must not be empty")
    _need(weight is not None, "weight is required")
    _need(weight.dtype in (_BF16, _F32), f"weight: dtype {weight.dtype}, expected torch.bfloat16 or torch.float32")
    _need(tuple(weight.shape) == (d,), f"weight: shape {tuple(weight.shape)}, expected {(d,)}")
    return x.numel() // d, d


def layer_norm_forward(x, weight, bias=None, eps: float = 1e-5, stream=None
                       ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """y = (x - mean) rstd weight + bias over the last dimension; returns (y, mean, rstd).

    x: bf16 or fp32, y likewise; weight and bias: both bf16 or both fp32; mean
    and rstd: fp32 of x's leading shape."""
    rows, d = _ln_args(x, weight)
    if bias is not None:
        _need(bias.dtype == weight.dtype and tuple(bias.shape) == (d,),
              f"bias: expected {weight.dtype} of shape {(d,)}, got {bias.dtype} of {tuple(bias.shape)}")
    dev = x.device
    _cuda(dev, x=x, weight=weight, bias=bias)
    with _scope(dev, stream):
        y = torch.empty_like(x)
        mean = torch.empty(x.shape[:-1], dtype=_F32, device=dev)
        rstd = torch.empty(x.shape[:-1], dtype=_F32, device=dev)
        _check(moe.lib().moe_layer_norm_forward(
            x.data_ptr(), weight.data_ptr(), bias.data_ptr() if bias is not None else None, rows, d,
            x.dtype == _F32, weight.dtype == _F32, eps, y.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
            _stream(dev)), "moe_layer_norm_forward")
    return y, mean, rstd


def layer_norm_backward(dy, x, weight, mean, rstd, need_dx: bool = True, need_dweight: bool = True,
                        need_dbias: bool = True, stream=None):
    """(dx, dweight, dbias) of layer_norm_forward from its saved statistics; None for what is not needed."""
    rows, d = _ln_args(x, weight)
    _need(dy is not None and dy.dtype == x.dtype and dy.shape == x.shape,
          f"dy: expected {x.dtype} of shape {tuple(x.shape)}")
    for name, s in (("mean", mean), ("rstd", rstd)):
        _need(s is not None and s.dtype == _F32 and s.shape == x.shape[:-1],
              f"{name}: expected torch.float32 of shape {tuple(x.shape[:-1])}")
    dev = x.device
    _cuda(dev, dy=dy, x=x, weight=weight, mean=mean, rstd=rstd)
    with _scope(dev, stream):
        dx = torch.empty_like(x) if need_dx else None
        dw = torch.empty_like(weight) if need_dweight else None
        db = torch.empty_like(weight) if need_dbias else None
        n = ctypes.c_size_t()
        lib = moe.lib()
        _check(lib.moe_layer_norm_workspace_bytes(rows, d, ctypes.byref(n)), "moe_layer_norm_workspace_bytes")
        ws = _workspace(n.value, dev)
        _check(lib.moe_layer_norm_backward(
            dy.data_ptr(), x.data_ptr(), weight.data_ptr(), mean.data_ptr(), rstd.data_ptr(), rows, d,
            x.dtype == _F32, weight.dtype == _F32, dx.data_ptr() if need_dx else None,
            dw.data_ptr() if need_dweight else None, db.data_ptr() if need_dbias else None, ws.data_ptr(), n.value,
            _stream(dev)), "moe_layer_norm_backward")
    return dx, dw, db


class _LayerNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        x = x.contiguous()
        y, mean, rstd = layer_norm_forward(x, weight, bias, eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw, db = layer_norm_backward(dy.contiguous(), x, weight, mean, rstd, need_dx=need[0],
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
        _need(t is not None and t.dtype == _BF16 and t.dim() == 2, f"{name}: expected a 2-d torch.bfloat16 tensor")
    _need(X.shape[1] == W.shape[1], f"W: width {W.shape[1]}, X has {X.shape[1]}")
    return X.shape[0], X.shape[1], W.shape[0]


def _row_vector(name, t, T):
    _need(t is not None and t.dtype == _F32 and tuple(t.shape) == (T,),
          f"{name}: expected torch.float32 of shape {(T,)}")


def _ids_arg(name, t, shape):
    _need(t is not None and t.dtype in (torch.int32, torch.int64) and tuple(t.shape) == shape,
          f"{name}: expected int32 or int64 of shape {shape}")


def _teacher_args(teacher, ids, T):
    _need(teacher is not None and teacher.dtype in (_F32, _BF16) and teacher.dim() == 2 and teacher.shape[0] == T,
          f"teacher_logits: expected a torch.float32 or torch.bfloat16 tensor of {T} rows")
    _ids_arg("teacher_ids", ids, tuple(teacher.shape))


def _head_config(T, d, V, ids, teacher=None, temperature=1.0, piece=0, wait_timeout_ns=0, debug_flags=0):
    return moe_head_config_t(T, V, d, teacher.shape[1] if teacher is not None else 0, temperature,
                             ids.dtype == torch.int64, teacher is not None and teacher.dtype == _BF16, piece,
                             wait_timeout_ns, debug_flags)


def _head_workspace(cfg, distill: bool, backward: bool, device):
    n = ctypes.c_size_t()
    _check(moe.lib().moe_head_workspace_bytes(ctypes.byref(cfg), distill, backward, ctypes.byref(n)),
           "moe_head_workspace_bytes")
    return _workspace(n.value, device), n.value


def _head_forward(name, X, W, targets, cfg, distill, stream):
    dev = X.device
    with _scope(dev, stream):
        out = torch.empty((2, X.shape[0]), dtype=_F32, device=dev)
        loss, lse = out[0], out[1]
        ws, n = _head_workspace(cfg, distill, False, dev)
        status = _status_word(dev)
        _check(getattr(moe.lib(), name)(ctypes.byref(cfg), X.data_ptr(), W.data_ptr(),
                                        *[t.data_ptr() for t in targets], loss.data_ptr(), lse.data_ptr(),
                                        ws.data_ptr(), n, status.data_ptr(), _stream(dev)), name)
    return loss, lse


def _head_backward(name, dloss, X, W, targets, lse, cfg, distill, need_dX, need_dW, stream):
    dev = X.device
    with _scope(dev, stream):
        dX = torch.empty_like(X) if need_dX else None
        dW = torch.empty_like(W) if need_dW else None
        ws, n = _head_workspace(cfg, distill, True, dev)
        status = _status_word(dev)
        _check(getattr(moe.lib(), name)(ctypes.byref(cfg), dloss.data_ptr(), X.data_ptr(), W.data_ptr(),
                                        *[t.data_ptr() for t in targets], lse.data_ptr(),
                                        dX.data_ptr() if need_dX else None, dW.data_ptr() if need_dW else None,
                                        ws.data_ptr(), n, status.data_ptr(), _stream(dev)), name)
    return dX, dW


def cross_entropy_forward(X, W, labels, stream=None, wait_timeout_ns: int = 0, debug_flags: int = 0):
    """(loss, lse), both fp32 [T]: loss_t = lse_t - z_t[labels_t] with z = X W^T.

    X bf16 [T, d], W bf16 [V, d], d a multiple of 8; labels int32 or int64
    [T].  A label outside [0, V) marks a token without a loss (0, and lse 0)."""
    T, d, V = _head_args(X, W)
    _ids_arg("labels", labels, (T,))
    dev = X.device
    _cuda(dev, X=X, W=W, labels=labels)
    cfg = _head_config(T, d, V, labels, wait_timeout_ns=wait_timeout_ns, debug_flags=debug_flags)
    return _head_forward("moe_cross_entropy_forward", X, W, (labels,), cfg, False, stream)


def cross_entropy_backward(dloss, X, W, labels, lse, need_dX: bool = True, need_dW: bool = True, piece: int = 0,
                           stream=None, wait_timeout_ns: int = 0, debug_flags: int = 0):
    """(dX, dW) bf16 for the upstream gradient dloss fp32 [T] and the forward's lse; None for what is not needed.

    `piece`: vocabulary columns handled at a time (0: a default that keeps
    the piece's workspace near 256 MB)."""
    T, d, V = _head_args(X, W)
    _ids_arg("labels", labels, (T,))
    _row_vector("dloss", dloss, T)
    _row_vector("lse", lse, T)
    _cuda(X.device, X=X, W=W, labels=labels)
    _rows_on(X.device, dloss=dloss, lse=lse)
    cfg = _head_config(T, d, V, labels, piece=piece, wait_timeout_ns=wait_timeout_ns, debug_flags=debug_flags)
    return _head_backward("moe_cross_entropy_backward", dloss, X, W, (labels,), lse, cfg, False, need_dX, need_dW,
                          stream)


def distill_forward(X, W, teacher_logits, teacher_ids, temperature: float = 1.0, stream=None,
                    wait_timeout_ns: int = 0, debug_flags: int = 0):
    """(loss, lse), both fp32 [T]: temperature^2 times the divergence of the student's softmax over the
    vocabulary from the teacher's softmax over its K entries, both at the temperature.

    teacher_logits fp32 or bf16 [T, K], teacher_ids int32 or int64 [T, K].  An
    entry whose id is outside [0, V) or whose logit is -inf is not in use."""
    T, d, V = _head_args(X, W)
    _teacher_args(teacher_logits, teacher_ids, T)
    _cuda(X.device, X=X, W=W, teacher_logits=teacher_logits, teacher_ids=teacher_ids)
    cfg = _head_config(T, d, V, teacher_ids, teacher_logits, temperature, wait_timeout_ns=wait_timeout_ns,
                       debug_flags=debug_flags)
    return _head_forward("moe_distill_forward", X, W, (teacher_logits, teacher_ids), cfg, True, stream)


def distill_backward(dloss, X, W, teacher_logits, teacher_ids, lse, temperature: float = 1.0, need_dX: bool = True,
                     need_dW: bool = True, piece: int = 0, stream=None, wait_timeout_ns: int = 0,
                     debug_flags: int = 0):
    """(dX, dW) bf16 of distill_forward for the upstream gradient dloss fp32 [T]; None for what is not needed."""
    T, d, V = _head_args(X, W)
    _teacher_args(teacher_logits, teacher_ids, T)
    _row_vector("dloss", dloss, T)
    _row_vector("lse", lse, T)
    _cuda(X.device, X=X, W=W, teacher_logits=teacher_logits, teacher_ids=teacher_ids)
    _rows_on(X.device, dloss=dloss, lse=lse)
    cfg = _head_config(T, d, V, teacher_ids, teacher_logits, temperature, piece, wait_timeout_ns, debug_flags)
    return _head_backward("moe_distill_backward", dloss, X, W, (teacher_logits, teacher_ids), lse, cfg, True, need_dX,
                          need_dW, stream)


def _rows_on(device, **vectors) -> None:
    """Row vectors need no more than their own alignment (a row of a larger tensor is fine)."""
    for name, t in vectors.items():
        _need(t.is_cuda and t.device == device and t.is_contiguous(), f"{name}: must be contiguous on {device}")


class _CrossEntropyFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, W, labels):
        X = X.contiguous()
        loss, lse = cross_entropy_forward(X, W, labels)
        ctx.save_for_backward(X, W, labels, lse)
        return loss

    @staticmethod
    def backward(ctx, dloss):
        X, W, labels, lse = ctx.saved_tensors
        dX, dW = cross_entropy_backward(dloss.contiguous(), X, W, labels, lse, need_dX=ctx.needs_input_grad[0],
                                        need_dW=ctx.needs_input_grad[1])
        return dX, dW, None


class _DistillFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, W, teacher_logits, teacher_ids, temperature):
        X = X.contiguous()
        loss, lse = distill_forward(X, W, teacher_logits, teacher_ids, temperature)
        ctx.temperature = temperature
        ctx.save_for_backward(X, W, teacher_logits, teacher_ids, lse)
        return loss

    @staticmethod
    def backward(ctx, dloss):
        X, W, teacher, ids, lse = ctx.saved_tensors
        dX, dW = distill_backward(dloss.contiguous(), X, W, teacher, ids, lse, ctx.temperature,
                                  need_dX=ctx.needs_input_grad[0], need_dW=ctx.needs_input_grad[1])
        return dX, dW, None, None, None


def linear_cross_entropy(X, W, labels) -> torch.Tensor:
    """Differentiable per-token loss fp32 [T] of the head W [V, d] on X [T, d]."""
    return _CrossEntropyFunction.apply(X, W, labels)


def linear_distillation(X, W, teacher_logits, teacher_ids, temperature: float = 1.0) -> torch.Tensor:
    """Differentiable per-token distillation loss fp32 [T] (the teacher gets no gradient)."""
    return _DistillFunction.apply(X, W, teacher_logits.detach(), teacher_ids, temperature)


class LMHead(torch.nn.Module):
    """The head's weight [V, d] (bf16, N(0, 1/d)) with its two losses."""

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
