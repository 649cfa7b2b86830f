"""Losses at the language-model head (tj2_linear_ce_*, tj2_distill_topk of include/tj2.h).

linear_ce_fwd / linear_ce_bwd: cross entropy of X W^T without the logits in memory; linear_cross_entropy
is the same as a differentiable function.  distill_topk: a student's logits against a teacher's top logits,
loss and gradient from one read; distillation_loss is its differentiable form.
"""
from __future__ import annotations

import ctypes

import torch
from torch.autograd.function import once_differentiable

from . import _BF16, _F32, _I32, _dense, _dtype_code, _ptr, check, lib, _stream
from .mx import _on

_OUT = (torch.bfloat16, torch.float32)
_I64 = (torch.int64,)


def _rows(t, name: str, dtypes, cols: int | None = None) -> int:
    """A matrix read with a leading dimension (unit column stride); returns the elements between rows."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in dtypes or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D CUDA (HIP) tensor of dtype {dtypes}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit column stride")
    if cols is not None and t.shape[1] != cols:
        raise ValueError(f"{name} has {t.shape[1]} columns, expected {cols}")
    # the stride of a single row is free: any pitch that holds it will do
    ld = t.stride(0) if t.shape[0] > 1 else max(t.shape[1], -(-t.shape[1] // 8) * 8)
    if ld < t.shape[1]:
        raise ValueError(f"{name} has rows that overlap")
    return ld


def _workspace(n: int, device) -> torch.Tensor:
    return torch.empty(max(int(n), 1), dtype=torch.uint8, device=device)


def linear_ce_fwd(X: torch.Tensor, W: torch.Tensor, targets: torch.Tensor, *, ignore_index: int = -100,
                  loss: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None):
    """Per-token (loss, lse) of the logits X W^T: X [T, K], W [V, K] bf16, targets int64 [T]; fp32 [T] results.

    The loss of a token with targets[t] == ignore_index is 0, of one outside the vocabulary NaN."""
    ldx = _rows(X, "X", _BF16)
    T, K = X.shape
    ldw = _rows(W, "W", _BF16, K)
    V = W.shape[0]
    _dense(targets, "targets", _I64, shape=(T,))
    if loss is None:
        loss = torch.empty(T, dtype=torch.float32, device=X.device)
    if lse is None:
        lse = torch.empty(T, dtype=torch.float32, device=X.device)
    _dense(loss, "loss", _F32, shape=(T,))
    _dense(lse, "lse", _F32, shape=(T,))
    if workspace is None:
        workspace = _workspace(lib().tj2_linear_ce_fwd_workspace_size(T, K, V), X.device)
    _dense(workspace, "workspace", (torch.uint8,))
    with _on(X, W, targets, loss, lse, workspace):
        st = lib().tj2_linear_ce_fwd(_ptr(X), ldx, _ptr(W), ldw, _ptr(targets), T, K, V, ignore_index, _ptr(loss), _ptr(lse),
                                     _ptr(workspace), workspace.numel(), _stream())
    check("tj2_linear_ce_fwd", st)
    return loss, lse


def linear_ce_bwd(X: torch.Tensor, W: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor, dloss: torch.Tensor, *,
                  ignore_index: int = -100, dx_dtype=torch.bfloat16, dw_dtype=torch.bfloat16,
                  dX: torch.Tensor | None = None, dW: torch.Tensor | None = None, need_dx: bool = True,
                  need_dw: bool = True, workspace: torch.Tensor | None = None):
    """(dX [T, K], dW [V, K]) for dloss, the gradient of each token's loss (fp32 [T]), with lse of linear_ce_fwd.

    need_dx / need_dw False leaves that gradient out (None)."""
    ldx = _rows(X, "X", _BF16)
    T, K = X.shape
    ldw = _rows(W, "W", _BF16, K)
    V = W.shape[0]
    _dense(targets, "targets", _I64, shape=(T,))
    _dense(lse, "lse", _F32, shape=(T,))
    _dense(dloss, "dloss", _F32, shape=(T,))
    if dX is None and need_dx:
        dX = torch.empty((T, K), dtype=dx_dtype, device=X.device)
    if dW is None and need_dw:
        dW = torch.empty((V, K), dtype=dw_dtype, device=X.device)
    _dense(dX, "dX", _OUT, shape=(T, K), optional=True)
    _dense(dW, "dW", _OUT, shape=(V, K), optional=True)
    if workspace is None:
        workspace = _workspace(lib().tj2_linear_ce_bwd_workspace_size(T, K, V), X.device)
    _dense(workspace, "workspace", (torch.uint8,))
    with _on(X, W, targets, lse, dloss, dX, dW, workspace):
        st = lib().tj2_linear_ce_bwd(_ptr(X), ldx, _ptr(W), ldw, _ptr(targets), T, K, V, ignore_index, _ptr(lse), _ptr(dloss),
                                     _ptr(dX), _dtype_code(dX) if dX is not None else 0, _ptr(dW),
                                     _dtype_code(dW) if dW is not None else 0, _ptr(workspace), workspace.numel(), _stream())
    check("tj2_linear_ce_bwd", st)
    return dX, dW


def _reduced(loss, targets, ignore_index, reduction):
    if reduction == "none":
        return loss
    if reduction == "sum":
        return loss.sum()
    return loss.sum() / (targets != ignore_index).sum()


class _LinearCe(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, W, targets, ignore_index):
        loss, lse = linear_ce_fwd(X, W, targets, ignore_index=ignore_index)
        ctx.save_for_backward(X, W, targets, lse)
        ctx.ignore_index = ignore_index
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss):
        X, W, targets, lse = ctx.saved_tensors
        if not (ctx.needs_input_grad[0] or ctx.needs_input_grad[1]):
            return None, None, None, None
        dX, dW = linear_ce_bwd(X, W, targets, lse, dloss.contiguous(), ignore_index=ctx.ignore_index,
                               need_dx=ctx.needs_input_grad[0], need_dw=ctx.needs_input_grad[1])
        return dX, dW, None, None


def linear_cross_entropy(X: torch.Tensor, W: torch.Tensor, targets: torch.Tensor, *, ignore_index: int = -100,
                         reduction: str = "mean") -> torch.Tensor:
    """Differentiable cross entropy of X W^T; reduction "mean" (over the tokens not ignored), "sum" or "none"."""
    if reduction not in ("mean", "sum", "none"):
        raise ValueError('reduction must be "mean", "sum" or "none"')
    return _reduced(_LinearCe.apply(X, W, targets, ignore_index), targets, ignore_index, reduction)


def distill_topk(logits: torch.Tensor, ids: torch.Tensor, teacher: torch.Tensor, *, temperature: float = 1.0,
                 alpha: float = 1.0, targets: torch.Tensor | None = None, ignore_index: int = -100,
                 weight: torch.Tensor | None = None, grad: bool = False, loss: torch.Tensor | None = None,
                 dlogits: torch.Tensor | None = None):
    """Per-token loss (fp32 [T]) of student logits [T, V] against a teacher's kept logits (ids int32 [T, k],
    teacher [T, k] of the logits' dtype): alpha * temperature^2 * KL(teacher || student) + (1 - alpha) * cross
    entropy with targets.  With grad (or dlogits given, which may be logits itself): (loss, dlogits), the
    gradient for `weight`, the gradient of each token's loss (fp32 [T], 1 if not given)."""
    ldl = _rows(logits, "logits", _OUT)
    T, V = logits.shape
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise ValueError("ids must be an int32 tensor [T, k]")
    k = ids.shape[1]
    _dense(ids, "ids", _I32, shape=(T, k))
    _dense(teacher, "teacher", (logits.dtype,), shape=(T, k))
    _dense(targets, "targets", _I64, shape=(T,), optional=True)
    _dense(weight, "weight", _F32, shape=(T,), optional=True)
    if loss is None:
        loss = torch.empty(T, dtype=torch.float32, device=logits.device)
    _dense(loss, "loss", _F32, shape=(T,))
    if dlogits is None and grad:
        dlogits = torch.empty((T, V), dtype=logits.dtype, device=logits.device)
    ldd = V
    if dlogits is not None:
        ldd = _rows(dlogits, "dlogits", (logits.dtype,), V)
        if dlogits.shape[0] != T:
            raise ValueError(f"dlogits has {dlogits.shape[0]} rows, expected {T}")
    with _on(logits, ids, teacher, targets, weight, loss, dlogits):
        st = lib().tj2_distill_topk(_ptr(logits), _dtype_code(logits), T, V, ldl, _ptr(ids), _ptr(teacher), k,
                                    ctypes.c_float(temperature), ctypes.c_float(alpha), _ptr(targets), ignore_index,
                                    _ptr(weight), _ptr(loss), _ptr(dlogits), ldd, _stream())
    check("tj2_distill_topk", st)
    return loss if dlogits is None else (loss, dlogits)


class _Distill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, teacher, temperature, alpha, targets, ignore_index):
        ctx.args = dict(temperature=temperature, alpha=alpha, targets=targets, ignore_index=ignore_index)
        ctx.save_for_backward(logits, ids, teacher)
        return distill_topk(logits, ids, teacher, **ctx.args)

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss):
        if not ctx.needs_input_grad[0]:
            return (None,) * 7
        logits, ids, teacher = ctx.saved_tensors
        _, dz = distill_topk(logits, ids, teacher, weight=dloss.contiguous(), grad=True, **ctx.args)
        return (dz,) + (None,) * 6


def distillation_loss(logits: torch.Tensor, ids: torch.Tensor, teacher: torch.Tensor, *, temperature: float = 1.0,
                      alpha: float = 1.0, targets: torch.Tensor | None = None, ignore_index: int = -100,
                      reduction: str = "mean") -> torch.Tensor:
    """Differentiable distill_topk; reduction "mean" (over the tokens not ignored), "sum" or "none"."""
    if reduction not in ("mean", "sum", "none"):
        raise ValueError('reduction must be "mean", "sum" or "none"')
    loss = _Distill.apply(logits, ids, teacher, temperature, alpha, targets, ignore_index)
    if targets is None and reduction == "mean":
        return loss.mean()
    return _reduced(loss, targets, ignore_index, reduction)
