"""MXFP4 operands and the linear layer on them (the mxfp4_ entry points of include/tj2.h).

MXFP4 stores E2M1 elements under one power-of-two scale per 32, the form gfx950's scaled matrix
instructions take as it is.  Names and arguments follow the NVFP4 functions of the package; work runs on
the current stream of the tensors' device.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import (_BF16, _F32, GROUP_COL, GROUP_ROW, MXFP4, RTN, SR, QTensor, _dense, _dtype_code, _matrix_out, _ptr,
               _stream, check, lib)

_OUT = (torch.bfloat16, torch.float32)


def _on(*tensors):
    """The device all `tensors` (Nones aside) are on, made current for a call where it is not."""
    dev = None
    for t in tensors:
        if t is None:
            continue
        d = (t.codes if isinstance(t, QTensor) else t).device
        if dev is not None and d != dev:
            raise ValueError(f"tensors on different devices: {dev} and {d}")
        dev = d
    return contextlib.nullcontext() if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)


def _mx(q, name: str, rows: int | None = None, length: int | None = None) -> None:
    if not isinstance(q, QTensor) or q.fmt != MXFP4:
        raise ValueError(f"{name} must be an MXFP4 QTensor")
    if not q.codes.is_cuda:
        raise ValueError(f"{name} must be on a CUDA (HIP) device")
    if (rows is not None and q.rows != rows) or (length is not None and q.len != length):
        raise ValueError(f"{name} is [{q.rows}, {q.len}], expected [{rows}, {length}]")


def mx_quantize(x, *, grouping: int = GROUP_ROW, rounding: int = RTN, rht: bool = False, signs: int = 0, seed: int = 0,
                offset: int = 0, out: QTensor | None = None) -> QTensor:
    """Quantize a dense bf16/fp32 tensor [rows, cols], or regroup an MXFP4 QTensor (GROUP_COL), to MXFP4.

    GROUP_ROW groups along cols; GROUP_COL along rows, stored transposed as [cols, rows].  RTN takes the
    scale 2^(floor(log2 amax) - 2); SR the smallest one that saturates nothing, with Philox draws of
    (seed, offset).  rht applies the 16-wide Hadamard transform with the sign mask `signs` first."""
    if isinstance(x, QTensor):
        _mx(x, "x")
        rows, cols, xp, xd, xq = x.rows, x.len, None, MXFP4, ctypes.byref(x.c())
        dev = x.codes.device
    else:
        _dense(x, "x", _OUT)
        if x.dim() != 2:
            raise ValueError("x must be 2-D")
        rows, cols = x.shape
        xp, xd, xq, dev = x, _dtype_code(x), None, x.device
    if out is None:
        if rows <= 0 or cols <= 0:
            raise ValueError("x must not be empty")
        out = QTensor(MXFP4, rows, cols, dev) if grouping == GROUP_ROW else QTensor(MXFP4, cols, rows, dev)
    _mx(out, "out")
    with _on(x, out):
        st = lib().mxfp4_quantize(_ptr(xp), xd, xq, rows, cols, grouping, rounding, 1 if rht else 0, signs, seed, offset,
                                  ctypes.byref(out.c()), _stream())
    check("mxfp4_quantize", st)
    return out


def mx_dequantize(q: QTensor, *, dtype=torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """The values of an MXFP4 QTensor as a dense [rows, len] tensor (bf16 holds them exactly)."""
    _mx(q, "q")
    if out is None:
        out = torch.empty((q.rows, q.len), dtype=dtype, device=q.codes.device)
    _dense(out, "out", _OUT, shape=(q.rows, q.len))
    with _on(q, out):
        st = lib().mxfp4_dequantize(ctypes.byref(q.c()), _ptr(out), _dtype_code(out), _stream())
    check("mxfp4_dequantize", st)
    return out


def mx_gemm_workspace(I: int, J: int, K: int, device="cuda") -> torch.Tensor | None:
    """Workspace of an I x J product over K, or None where none is needed."""
    n = int(lib().mxfp4_gemm_workspace_size(I, J, K))
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def mx_gemm(A: QTensor, B: QTensor, *, out: torch.Tensor | None = None, out_dtype=torch.float32, accumulate: bool = False,
            workspace: torch.Tensor | None = None) -> torch.Tensor:
    """C = A B^T (accumulate: added into a float32 `out`) on MXFP4 operands grouped along the reduction."""
    _mx(A, "A")
    _mx(B, "B", B.rows, A.len)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = torch.empty((A.rows, B.rows), dtype=out_dtype, device=A.codes.device)
    _matrix_out(out, "out", _OUT, A.rows, B.rows)
    if workspace is None:
        workspace = mx_gemm_workspace(A.rows, B.rows, A.len, A.codes.device)
    _dense(workspace, "workspace", (torch.uint8,), optional=True)
    with _on(A, B, out, workspace):
        st = lib().mxfp4_gemm(ctypes.byref(A.c()), ctypes.byref(B.c()), _ptr(out), _dtype_code(out),
                              max(out.stride(0), B.rows), 1 if accumulate else 0, _ptr(workspace),
                              0 if workspace is None else workspace.numel(), _stream())
    check("mxfp4_gemm", st)
    return out


def mx_linear_fwd(X: torch.Tensor, W_master: torch.Tensor | None, N: int, *, Wq: QTensor | None = None,
                  y_dtype=torch.bfloat16, Y: torch.Tensor | None = None, Xq: QTensor | None = None,
                  workspace: torch.Tensor | None = None):
    """Y = X W^T with MXFP4 operands; returns (Y, saved) with saved = dict(Xq, Wq).

    W_master (fp32 [N, K]) is quantized into Wq; without it Wq is used as given.  X has any number of rows."""
    _dense(X, "X", _BF16)
    if X.dim() != 2:
        raise ValueError("X must be 2-D")
    M, K = X.shape
    _dense(W_master, "W_master", _F32, shape=(N, K), optional=True)
    if W_master is None and Wq is None:
        raise ValueError("W_master or Wq is required")
    if Wq is None:
        Wq = QTensor(MXFP4, N, K, X.device)
    if Xq is None:
        Xq = QTensor(MXFP4, M, K, X.device)
    _mx(Wq, "Wq", N, K)
    _mx(Xq, "Xq", M, K)
    if Y is None:
        Y = torch.empty((M, N), dtype=y_dtype, device=X.device)
    _dense(Y, "Y", _OUT, shape=(M, N))
    if workspace is None:
        workspace = mx_gemm_workspace(M, N, K, X.device)
    _dense(workspace, "workspace", (torch.uint8,), optional=True)
    with _on(X, W_master, Wq, Xq, Y, workspace):
        st = lib().mxfp4_linear_fwd(_ptr(X), M, K, N, _ptr(W_master), ctypes.byref(Wq.c()), ctypes.byref(Xq.c()), _ptr(Y),
                                    _dtype_code(Y), _ptr(workspace), 0 if workspace is None else workspace.numel(),
                                    _stream())
    check("mxfp4_linear_fwd", st)
    return Y, {"Xq": Xq, "Wq": Wq}


def mx_linear_bwd_workspace(M: int, N: int, K: int, device="cuda") -> torch.Tensor:
    return torch.empty(int(lib().mxfp4_linear_bwd_workspace_size(M, N, K)), dtype=torch.uint8, device=device)


def mx_linear_bwd(dY: torch.Tensor, saved: dict, K: int, *, seed: int, offset: int, rht: bool = True, rounding: int = SR,
                  dx_dtype=torch.bfloat16, dX: torch.Tensor | None = None, dW: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None):
    """(dX, dW) of mx_linear_fwd from its saved operands: dY, W-hat and X-hat regrouped to MXFP4 along each
    product's reduction, stochastically rounded and Hadamard-transformed unless told otherwise."""
    _dense(dY, "dY", _BF16)
    if dY.dim() != 2:
        raise ValueError("dY must be 2-D")
    M, N = dY.shape
    Xq, Wq = saved["Xq"], saved["Wq"]
    _mx(Xq, "Xq", M, K)
    _mx(Wq, "Wq", N, K)
    if dX is None:
        dX = torch.empty((M, K), dtype=dx_dtype, device=dY.device)
    if dW is None:
        dW = torch.empty((N, K), dtype=torch.float32, device=dY.device)
    _dense(dX, "dX", _OUT, shape=(M, K))
    _dense(dW, "dW", _F32, shape=(N, K))
    if workspace is None:
        workspace = mx_linear_bwd_workspace(M, N, K, dY.device)
    _dense(workspace, "workspace", (torch.uint8,))
    with _on(dY, Xq, Wq, dX, dW, workspace):
        st = lib().mxfp4_linear_bwd(_ptr(dY), M, N, K, ctypes.byref(Xq.c()), ctypes.byref(Wq.c()), rounding,
                                    1 if rht else 0, seed, offset, _ptr(dX), _dtype_code(dX), _ptr(dW), _ptr(workspace),
                                    workspace.numel(), _stream())
    check("mxfp4_linear_bwd", st)
    return dX, dW
