"""Root-mean-square norm with the residual's addition (tj2_rms_norm_* of include/tj2.h).

rms_norm_fwd / rms_norm_bwd: s = x + residual, y = s weight / sqrt(mean(s^2) + eps) in the stream's type or as the FP8
operand of fp8_linear_fwd; rms_norm is the same as a differentiable function.
"""
from __future__ import annotations

from functools import lru_cache

import torch
from torch.autograd.function import once_differentiable

from . import _F32, FP8, QTensor, lib
from .fp8 import _q
from .losses import _rows
from .mx import _CODE, _OUT, _arg, _room, _run, _tensor


@lru_cache(maxsize=4096)
def _bwd_bytes(rows: int, cols: int) -> int:
    return max(1, int(lib().tj2_rms_norm_bwd_workspace_size(rows, cols)))


def _stream(t, name: str, index: int, like: torch.Tensor):
    """(pointer, pitch) of a matrix of like's type and shape with a pitch of its own; (0, 0) for None."""
    if t is None:
        return 0, 0
    if isinstance(t, torch.Tensor) and t.dtype is like.dtype and t.shape == like.shape and t.is_contiguous() and t.get_device() == index:
        return t.data_ptr(), like.shape[1]
    ld = _rows(t, name, (like.dtype,), index, like.shape[1])
    if t.shape[0] != like.shape[0]:
        raise ValueError(f"{name} has {t.shape[0]} rows, expected {like.shape[0]}")
    return t.data_ptr(), max(ld, like.shape[1])


def _like(x: torch.Tensor, index: int) -> torch.Tensor:
    """A contiguous tensor of x's shape and type."""
    return torch.empty_like(x) if x.is_contiguous() else torch.empty(x.shape, dtype=x.dtype, device=index)


def rms_norm_fwd(x: torch.Tensor, weight: torch.Tensor, *, residual: torch.Tensor | None = None, eps: float = 1e-6,
                 fp8: bool = False, sum: torch.Tensor | None = None, y=None, rstd: torch.Tensor | None = None):
    """(y, s, rstd) of x [rows, cols] (bf16 or fp32, unit column stride), weight [cols] (either type).

    s is x + residual in a contiguous `sum` (which may be x or residual), or x itself without a residual; y has x's type,
    or with fp8 (or a QTensor given for y) is an FP8 QTensor; rstd fp32 [rows]."""
    index = _tensor(x, "x", 2)
    if x.dtype not in _OUT:
        raise ValueError(f"x has dtype {x.dtype}, expected one of {_OUT}")
    rows, cols = x.shape
    if not rows or not cols:
        raise ValueError("x must not be empty")
    xp, ldx = _stream(x, "x", index, x)
    rp, ldr = _stream(residual, "residual", index, x)
    if residual is None and sum is not None:
        raise ValueError("sum needs a residual")
    if residual is not None and sum is None:
        sum = _like(x, index)
    if y is None:
        y = QTensor.packed(FP8, rows, cols, index) if fp8 else _like(x, index)
    elif fp8 and not isinstance(y, QTensor):
        raise ValueError("y must be an FP8 QTensor")
    if rstd is None:
        rstd = torch.empty(rows, dtype=torch.float32, device=index)
    q = isinstance(y, QTensor)
    _run("tj2_rms_norm_fwd", index, xp, ldx, rp, ldr, _CODE[x.dtype], rows, cols, _arg(weight, "weight", _OUT, index, (cols,)),
         _CODE[weight.dtype], eps, _arg(sum, "sum", (x.dtype,), index, (rows, cols), optional=True),
         0 if q else _arg(y, "y", (x.dtype,), index, (rows, cols)), _q(y, "y", index, rows, cols) if q else None,
         _arg(rstd, "rstd", _F32, index, (rows,)))
    return y, x if residual is None else sum, rstd


def rms_norm_bwd(dy: torch.Tensor, s: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor, *, dsum: torch.Tensor | None = None,
                 ds: torch.Tensor | None = None, dweight: torch.Tensor | None = None, need_ds: bool = True, need_dw: bool = True,
                 workspace: torch.Tensor | None = None):
    """(ds, dweight) of rms_norm_fwd's y for its gradient dy [rows, cols] of s's type; dsum, the gradient that comes in
    for s itself, is added to ds, which is the gradient of x and of residual (ds may be dy, s or dsum).  need_ds / need_dw
    False leaves that gradient out (None)."""
    index = _tensor(s, "s", 2)
    if s.dtype not in _OUT:
        raise ValueError(f"s has dtype {s.dtype}, expected one of {_OUT}")
    rows, cols = s.shape
    if not rows or not cols:
        raise ValueError("s must not be empty")
    sp, lds = _stream(s, "s", index, s)
    yp, lddy = _stream(dy, "dy", index, s)
    dp, ldd = _stream(dsum, "dsum", index, s)
    wp = _arg(weight, "weight", _OUT, index, (cols,))
    if ds is None and need_ds:
        ds = _like(s, index)
    if dweight is None and need_dw:
        dweight = torch.empty_like(weight)
    workspace, ws, wn = _room(workspace, _bwd_bytes(rows, cols) if dweight is not None else 0, index)
    _run("tj2_rms_norm_bwd", index, yp, lddy, sp, lds, _CODE[s.dtype], rows, cols, wp, _CODE[weight.dtype],
         _arg(rstd, "rstd", _F32, index, (rows,)), dp, ldd, _arg(ds, "ds", (s.dtype,), index, (rows, cols), optional=True),
         _arg(dweight, "dweight", (weight.dtype,), index, (cols,), optional=True), ws, wn)
    return ds, dweight


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        ctx.set_materialize_grads(False)
        y, s, rstd = rms_norm_fwd(x, weight, residual=residual, eps=eps)
        ctx.save_for_backward(s, weight, rstd)
        return y if residual is None else (y, s)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dsum=None):
        s, weight, rstd = ctx.saved_tensors
        need_x, need_w, need_r, _ = ctx.needs_input_grad
        if dy is None:  # s alone was used
            return dsum, None, dsum if need_r else None, None
        if not (need_x or need_w or need_r):
            return None, None, None, None
        dsum = None if dsum is None else dsum.contiguous()
        ds, dw = rms_norm_bwd(dy.contiguous(), s, weight, rstd, dsum=dsum, need_ds=need_x or need_r, need_dw=need_w)
        return ds if need_x else None, dw, ds if need_r else None, None


def rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, *, eps: float = 1e-6):
    """Differentiable rms_norm_fwd: y, or with a residual (y, s), s = x + residual."""
    return _RmsNorm.apply(x, weight, residual, eps)
