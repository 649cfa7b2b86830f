"""Losses at the language-model head (tj2_linear_ce_*, tj2_distill_topk of include/tj2.h).

linear_ce_fwd / linear_ce_bwd: cross entropy of X W^T without the logits [T, V] in memory (the backward's
workspace holds their gradient a piece at a time); linear_cross_entropy is the same as a differentiable
function.  distill_topk: a student's logits against a teacher's top logits, loss and gradient from one read
(three above 106496 bf16 or 53248 fp32 entries); distillation_loss is its differentiable form, which takes one
pass for the loss and one in the backward.
"""
from __future__ import annotations

from functools import lru_cache

import torch
from torch.autograd.function import once_differentiable

from . import _BF16, _F32, _I32, lib
from .mx import _CODE, _OUT, _arg, _room, _run, _tensor

_I64 = (torch.int64,)


def _rows(t, name: str, dtypes, index: int, cols: int | None = None) -> int:
    """A matrix with a leading dimension (unit column stride); returns the elements between its rows."""
    if _tensor(t, name, 2) != index:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, other arguments on cuda:{index}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    rows, n = t.shape
    if cols is not None and n != cols:
        raise ValueError(f"{name} has {n} columns, expected {cols}")
    ld, unit = t.stride()
    if unit != 1 and n > 1:
        raise ValueError(f"{name} must have unit column stride")
    if rows <= 1:
        return -(-n // 8) * 8  # the stride of a single row is free: any pitch that holds it will do
    if ld < n:
        raise ValueError(f"{name} has rows that overlap")
    return ld


@lru_cache(maxsize=4096)
def _fwd_bytes(T: int, K: int, V: int) -> int:
    return max(1, int(lib().tj2_linear_ce_fwd_workspace_size(T, K, V)))


@lru_cache(maxsize=4096)
def _bwd_bytes(T: int, K: int, V: int) -> int:
    return max(1, int(lib().tj2_linear_ce_bwd_workspace_size(T, K, V)))


def linear_ce_fwd(X: torch.Tensor, W: torch.Tensor, targets: torch.Tensor, *, ignore_index: int = -100,
                  loss: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None):
    """Per-token (loss, lse) of the logits X W^T: X [T, K], W [V, K] bf16, targets int64 [T]; fp32 [T] results.

    The loss of a token with targets[t] == ignore_index is 0, of one outside the vocabulary NaN."""
    index = _tensor(X, "X", 2)
    ldx = _rows(X, "X", _BF16, index)
    T, K = X.shape
    ldw = _rows(W, "W", _BF16, index, K)
    V = W.shape[0]
    if loss is None:
        loss = torch.empty(T, dtype=torch.float32, device=index)
    if lse is None:
        lse = torch.empty(T, dtype=torch.float32, device=index)
    workspace, wp, wn = _room(workspace, _fwd_bytes(T, K, V), index)
    _run("tj2_linear_ce_fwd", index, X.data_ptr(), ldx, W.data_ptr(), ldw, _arg(targets, "targets", _I64, index, (T,)), T, K, V,
         ignore_index, _arg(loss, "loss", _F32, index, (T,)), _arg(lse, "lse", _F32, index, (T,)), wp, wn)
    return loss, lse


def linear_ce_bwd(X: torch.Tensor, W: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor, dloss: torch.Tensor, *,
                  ignore_index: int = -100, dx_dtype=torch.bfloat16, dw_dtype=torch.bfloat16,
                  dX: torch.Tensor | None = None, dW: torch.Tensor | None = None, need_dx: bool = True,
                  need_dw: bool = True, workspace: torch.Tensor | None = None):
    """(dX [T, K], dW [V, K]) for dloss, the gradient of each token's loss (fp32 [T]), with lse of linear_ce_fwd.

    need_dx / need_dw False leaves that gradient out (None).  dx_dtype and dw_dtype are the results' types; the
    logits' gradient that both are products of is bf16 (fp32 sums)."""
    index = _tensor(X, "X", 2)
    ldx = _rows(X, "X", _BF16, index)
    T, K = X.shape
    ldw = _rows(W, "W", _BF16, index, K)
    V = W.shape[0]
    if dX is None and need_dx:
        dX = torch.empty((T, K), dtype=dx_dtype, device=index)
    if dW is None and need_dw:
        dW = torch.empty((V, K), dtype=dw_dtype, device=index)
    workspace, wp, wn = _room(workspace, _bwd_bytes(T, K, V), index)
    _run("tj2_linear_ce_bwd", index, X.data_ptr(), ldx, W.data_ptr(), ldw, _arg(targets, "targets", _I64, index, (T,)), T, K, V,
         ignore_index, _arg(lse, "lse", _F32, index, (T,)), _arg(dloss, "dloss", _F32, index, (T,)),
         _arg(dX, "dX", _OUT, index, (T, K), optional=True), _CODE[dX.dtype] if dX is not None else 0,
         _arg(dW, "dW", _OUT, index, (V, K), optional=True), _CODE[dW.dtype] if dW is not None else 0, wp, wn)
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
    index = _tensor(logits, "logits", 2)
    ldl = _rows(logits, "logits", _OUT, index)
    T, V = logits.shape
    _tensor(ids, "ids", 2)
    k = ids.shape[1]
    if loss is None:
        loss = torch.empty(T, dtype=torch.float32, device=index)
    if dlogits is None and grad:
        dlogits = torch.empty((T, V), dtype=logits.dtype, device=index)
    ldd, dp = V, 0
    if dlogits is not None:
        ldd = ldl if dlogits is logits else _rows(dlogits, "dlogits", (logits.dtype,), index, V)
        if dlogits.shape[0] != T:
            raise ValueError(f"dlogits has {dlogits.shape[0]} rows, expected {T}")
        dp = dlogits.data_ptr()
    _run("tj2_distill_topk", index, logits.data_ptr(), _CODE[logits.dtype], T, V, ldl, _arg(ids, "ids", _I32, index, (T, k)),
         _arg(teacher, "teacher", (logits.dtype,), index, (T, k)), k, temperature, alpha,
         _arg(targets, "targets", _I64, index, (T,), optional=True), ignore_index,
         _arg(weight, "weight", _F32, index, (T,), optional=True), _arg(loss, "loss", _F32, index, (T,)), dp, ldd)
    return loss if dlogits is None else (loss, dlogits)


class _Distill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, teacher, temperature, alpha, targets, ignore_index):
        ctx.args = dict(temperature=temperature, alpha=alpha, ignore_index=ignore_index)
        ctx.save_for_backward(logits, ids, teacher, targets)
        return distill_topk(logits, ids, teacher, targets=targets, **ctx.args)

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss):
        if not ctx.needs_input_grad[0]:
            return (None,) * 7
        logits, ids, teacher, targets = ctx.saved_tensors
        _, dz = distill_topk(logits, ids, teacher, targets=targets, weight=dloss.contiguous(), grad=True, **ctx.args)
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
