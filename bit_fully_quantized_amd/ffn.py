"""The gated feed-forward block (tj2_gated_ffn_* of include/tj2.h): Y = (act(X Wg^T) * (X Wu^T)) Wd^T in bf16.

gated_ffn_fwd / gated_ffn_bwd: both projections, the activation and the product in one kernel, then the output product;
the backward takes the forward's gates and factors and gives the gradients of X and the three weights.  gated_ffn is the
same as a differentiable function.
"""
from __future__ import annotations

from functools import lru_cache

import torch
from torch.autograd.function import once_differentiable

from . import _BF16, _lib, lib
from .losses import _rows
from .mx import _CODE, _OUT, _U8, _arg, _room, _run, _tensor

ACTIVATIONS = {"silu": _lib.SILU, "gelu": _lib.GELU, "gelu_tanh": _lib.GELU_TANH}


@lru_cache(maxsize=4096)
def _fwd_bytes(T: int, D: int, F: int) -> int:
    return max(1, int(lib().tj2_gated_ffn_fwd_workspace_size(T, D, F)))


@lru_cache(maxsize=4096)
def _bwd_bytes(T: int, D: int, F: int) -> int:
    return max(1, int(lib().tj2_gated_ffn_bwd_workspace_size(T, D, F)))


@lru_cache(maxsize=4096)
def gated_ffn_saved_size(T: int, F: int) -> int:
    """Bytes that gated_ffn_fwd keeps for gated_ffn_bwd: 6 of each feature of a token, in whole 64 x 64 of them."""
    return int(lib().tj2_gated_ffn_saved_size(T, F))


def _matrix(t, name: str, index: int, cols: int) -> int:
    """The row stride of a bf16 matrix of `cols` columns."""
    if isinstance(t, torch.Tensor) and t.dtype is torch.bfloat16 and t.dim() == 2 and t.is_contiguous() and t.get_device() == index and t.shape[1] == cols:
        return cols
    return _rows(t, name, _BF16, index, cols)


def _operands(X, Wg, Wu, Wd, activation: str):
    """(device index, T, D, F, the arguments that both passes share)."""
    index = _tensor(X, "X", 2)
    T, D = X.shape
    ldx = _matrix(X, "X", index, D)
    ldw = _matrix(Wg, "Wg", index, D)
    ldu = _matrix(Wu, "Wu", index, D)
    F = Wg.shape[0]
    ldd = _matrix(Wd, "Wd", index, F)
    if Wu.shape[0] != F or Wd.shape[0] != D:
        raise ValueError(f"Wg is [{F}, {D}]: Wu must be the same and Wd [{D}, {F}]")
    if ldu != ldw:
        raise ValueError("Wg and Wu must have the same row stride")
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}")
    return index, T, D, F, (X.data_ptr(), ldx, Wg.data_ptr(), Wu.data_ptr(), ldw, Wd.data_ptr(), ldd, T, D, F, act)


def gated_ffn_fwd(X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, Wd: torch.Tensor, *, activation: str = "silu",
                  save: bool = False, y_dtype=torch.bfloat16, Y: torch.Tensor | None = None, gu: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None):
    """(Y [T, D], saved) of X [T, D], Wg and Wu [F, D], Wd [D, F] (bf16, unit column stride, one row stride for Wg and Wu);
    saved = dict(gu) with save (or gu given): the gates and factors in 24 bits, uint8 [gated_ffn_saved_size(T, F)], that
    gated_ffn_bwd reads, else None.
    activation "silu", "gelu" (g Phi(g)) or "gelu_tanh"."""
    index, T, D, F, args = _operands(X, Wg, Wu, Wd, activation)
    if Y is None:
        Y = torch.empty((T, D), dtype=y_dtype, device=index)
    if gu is None and save:
        gu = torch.empty(gated_ffn_saved_size(T, F), dtype=torch.uint8, device=index)
    workspace, wp, wn = _room(workspace, _fwd_bytes(T, D, F), index)
    _run("tj2_gated_ffn_fwd", index, *args, _arg(gu, "gu", _U8, index, (gated_ffn_saved_size(T, F),), optional=True), _arg(Y, "Y", _OUT, index, (T, D)),
         _CODE[Y.dtype], wp, wn)
    return Y, None if gu is None else {"gu": gu}


def gated_ffn_bwd(dY: torch.Tensor, X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, Wd: torch.Tensor, saved: dict, *,
                  activation: str = "silu", dx_dtype=torch.bfloat16, dw_dtype=torch.bfloat16, dX: torch.Tensor | None = None,
                  dWg: torch.Tensor | None = None, dWu: torch.Tensor | None = None, dWd: torch.Tensor | None = None,
                  need=(True, True, True, True), workspace: torch.Tensor | None = None):
    """(dX, dWg, dWu, dWd) for dY [T, D] from gated_ffn_fwd's saved; `need` False leaves a gradient out (None).  The
    weights' gradients are of one type."""
    index, T, D, F, args = _operands(X, Wg, Wu, Wd, activation)
    ldy = _matrix(dY, "dY", index, D)
    if dY.shape[0] != T:
        raise ValueError(f"dY has {dY.shape[0]} rows, expected {T}")
    shapes = ((T, D), (F, D), (F, D), (D, F))
    outs = [torch.empty(sh, dtype=dt, device=index) if t is None and n else t
            for t, n, sh, dt in zip((dX, dWg, dWu, dWd), need, shapes, (dx_dtype, dw_dtype, dw_dtype, dw_dtype))]
    dw = {t.dtype for t in outs[1:] if t is not None}
    if len(dw) > 1:
        raise ValueError("dWg, dWu and dWd must have one dtype")
    px, pg, pu, pd = (_arg(t, n, _OUT, index, sh, optional=True) for t, n, sh in zip(outs, ("dX", "dWg", "dWu", "dWd"), shapes))
    workspace, wp, wn = _room(workspace, _bwd_bytes(T, D, F), index)
    _run("tj2_gated_ffn_bwd", index, dY.data_ptr(), ldy, *args, _arg(saved["gu"], "gu", _U8, index, (gated_ffn_saved_size(T, F),)),
         px, _CODE[outs[0].dtype] if px else 0, pg, pu, pd, _CODE[dw.pop()] if dw else 0, wp, wn)
    return tuple(outs)


class _GatedFfn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, Wg, Wu, Wd, activation):
        grad = any(ctx.needs_input_grad)
        Y, saved = gated_ffn_fwd(X, Wg, Wu, Wd, activation=activation, save=grad)
        ctx.activation = activation
        if grad:
            ctx.save_for_backward(X, Wg, Wu, Wd, saved["gu"])
        return Y

    @staticmethod
    @once_differentiable
    def backward(ctx, dY):
        X, Wg, Wu, Wd, gu = ctx.saved_tensors
        dY = dY.contiguous()
        if dY.data_ptr() % 16:  # a view into a longer gradient
            dY = dY.clone()
        return (*gated_ffn_bwd(dY, X, Wg, Wu, Wd, {"gu": gu}, activation=ctx.activation, need=ctx.needs_input_grad[:4]), None)


def gated_ffn(X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, Wd: torch.Tensor, *, activation: str = "silu") -> torch.Tensor:
    """Differentiable gated_ffn_fwd: Y [T, D] in bf16."""
    if not torch.is_grad_enabled():  # (what leaves ask for is not withdrawn then: the function would keep the gates)
        return gated_ffn_fwd(X, Wg, Wu, Wd, activation=activation)[0]
    return _GatedFfn.apply(X, Wg, Wu, Wd, activation)
