"""FP8 operands and the linear layer on them (the fp8_ entry points of include/tj2.h).

E4M3 elements under one fp32 scale per 128 of a row (FP8: activations and gradients) or per 128 x 128 (FP8_BLOCK:
weights), multiplied by gfx950's 8-bit matrix instructions as they are stored (fp32 results: decoded, as exact
products).  Names and arguments follow the MXFP4 functions of the package; work runs on the current stream of the
tensors' device.
"""
from __future__ import annotations

from functools import lru_cache

import torch

from . import _BF16, _F32, FP8, FP8_BLOCK, GROUP_COL, GROUP_ROW, QTensor, _matrix_out, lib
from .mx import _CODE, _OUT, _arg, _byref, _room, _run, _tensor


def _q(q, name: str, index: int, rows: int | None = None, length: int | None = None, fmts=(FP8,)):
    """The descriptor of an FP8 argument on device `index`."""
    if not isinstance(q, QTensor) or q.fmt not in fmts:
        raise ValueError(f"{name} must be a QTensor of format {' or '.join({FP8: 'FP8', FP8_BLOCK: 'FP8_BLOCK'}[f] for f in fmts)}")
    if (rows is not None and q.rows != rows) or (length is not None and q.len != length):
        raise ValueError(f"{name} is [{q.rows}, {q.len}], expected [{rows}, {length}]")
    t = q.storage()
    if t.get_device() != index or (t is not q.buffer and q.scale128.get_device() != index):
        raise ValueError(f"{name} must be on cuda:{index}, with the other arguments")
    return _byref(q.c())


def fp8_quantize(x, *, grouping: int = GROUP_ROW, block: bool = False, out: QTensor | None = None) -> QTensor:
    """Quantize a dense bf16/fp32 tensor [rows, cols] to FP8, or regroup an FP8 QTensor (GROUP_COL).

    GROUP_ROW: a scale per 128 of a row, or with block (or an FP8_BLOCK `out`) per 128 x 128.  GROUP_COL: a scale per
    128 of a column, stored transposed as [cols, rows]."""
    if isinstance(x, QTensor):
        index = _tensor(x.storage(), "x")
        rows, cols, xp, xd, xq = x.rows, x.len, 0, FP8, _q(x, "x", index)
    else:
        index = _tensor(x, "x", 2)
        xp, xd, xq = _arg(x, "x", _OUT, index), _CODE[x.dtype], None
        rows, cols = x.shape
    if out is None:
        if block and grouping != GROUP_ROW:
            raise ValueError("block needs GROUP_ROW")
        fmt = FP8_BLOCK if block else FP8
        out = QTensor.packed(fmt, rows, cols, index) if grouping == GROUP_ROW else QTensor.packed(fmt, cols, rows, index)
    elif block and isinstance(out, QTensor) and out.fmt != FP8_BLOCK:
        raise ValueError("block needs an FP8_BLOCK out")
    _run("fp8_quantize", index, xp, xd, xq, rows, cols, grouping, _q(out, "out", index, fmts=(FP8, FP8_BLOCK)))
    return out


def fp8_dequantize(q: QTensor, *, dtype=torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """The values of an FP8 or FP8_BLOCK QTensor as a dense [rows, len] tensor (fp32 as the products take them, or
    rounded to bf16)."""
    if not isinstance(q, QTensor):
        raise ValueError("q must be an FP8 or FP8_BLOCK QTensor")
    index = _tensor(q.storage(), "q")
    desc = _q(q, "q", index, fmts=(FP8, FP8_BLOCK))
    if out is None:
        out = torch.empty((q.rows, q.len), dtype=dtype, device=index)
    _run("fp8_dequantize", index, desc, _arg(out, "out", _OUT, index, (q.rows, q.len)), _CODE[out.dtype])
    return out


@lru_cache(maxsize=4096)
def _gemm_bytes(I: int, J: int, K: int) -> int:
    return int(lib().fp8_gemm_workspace_size(I, J, K))


@lru_cache(maxsize=4096)
def _fwd_bytes(M: int, N: int, K: int) -> int:
    return int(lib().fp8_linear_fwd_workspace_size(M, N, K))


@lru_cache(maxsize=4096)
def fp8_linear_bwd_workspace_size(M: int, N: int, K: int) -> int:
    """Bytes of the workspace of fp8_linear_bwd."""
    return int(lib().fp8_linear_bwd_workspace_size(M, N, K))


def fp8_gemm_workspace(I: int, J: int, K: int, device="cuda") -> torch.Tensor | None:
    """Workspace of an I x J product over K, or None where none is needed."""
    n = _gemm_bytes(I, J, K)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def fp8_gemm(A: QTensor, B: QTensor, *, out: torch.Tensor | None = None, out_dtype=torch.float32, accumulate: bool = False,
             workspace: torch.Tensor | None = None) -> torch.Tensor:
    """C = A B^T (accumulate: added into a float32 `out`), A FP8, B FP8 or FP8_BLOCK, grouped along the reduction."""
    if not isinstance(A, QTensor) or not isinstance(B, QTensor):
        raise ValueError("A and B must be FP8 QTensors")
    index = _tensor(A.storage(), "A")
    a, b = _q(A, "A", index), _q(B, "B", index, B.rows, A.len, fmts=(FP8, FP8_BLOCK))
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = torch.empty((A.rows, B.rows), dtype=out_dtype, device=index)
    _matrix_out(out, "out", _OUT, A.rows, B.rows)
    if out.get_device() != index:
        raise ValueError(f"out is on cuda:{out.get_device()}, other arguments on cuda:{index}")
    workspace, wp, wn = _room(workspace, _gemm_bytes(A.rows, B.rows, A.len), index)
    _run("fp8_gemm", index, a, b, out.data_ptr(), _CODE[out.dtype], max(out.stride(0), B.rows), 1 if accumulate else 0, wp, wn)
    return out


def fp8_linear_fwd(X, W_master: torch.Tensor | None, N: int, *, Wq: QTensor | None = None, y_dtype=torch.bfloat16,
                   Y: torch.Tensor | None = None, Xq: QTensor | None = None, workspace: torch.Tensor | None = None):
    """Y = X W^T with FP8 operands; returns (Y, saved) with saved = dict(Xq, Wq).

    X: bf16 [M, K], quantized (into Xq), or an FP8 QTensor, taken as it is (rms_norm_fwd writes one).  W_master (fp32
    [N, K]) is quantized into Wq (FP8_BLOCK); without it Wq is used as given.  X has any number of rows."""
    if isinstance(X, QTensor):
        if Xq is not None and Xq is not X:
            raise ValueError("X is quantized already: Xq has nothing to receive")
        index = _tensor(X.storage(), "X")
        xp, M, K, Xq = 0, X.rows, X.len, X
    else:
        index = _tensor(X, "X", 2)
        xp = _arg(X, "X", _BF16, index)
        M, K = X.shape
    if W_master is None and Wq is None:
        raise ValueError("W_master or Wq is required")
    wp = _arg(W_master, "W_master", _F32, index, (N, K), optional=True)
    if Wq is None:
        Wq = QTensor.packed(FP8_BLOCK, N, K, index)
    if Xq is None:
        Xq = QTensor.packed(FP8, M, K, index)
    if Y is None:
        Y = torch.empty((M, N), dtype=y_dtype, device=index)
    workspace, sp, sn = _room(workspace, _fwd_bytes(M, N, K), index)
    _run("fp8_linear_fwd", index, xp, M, K, N, wp, _q(Wq, "Wq", index, N, K, (FP8_BLOCK,)), _q(Xq, "Xq", index, M, K),
         _arg(Y, "Y", _OUT, index, (M, N)), _CODE[Y.dtype], sp, sn)
    return Y, {"Xq": Xq, "Wq": Wq}


def fp8_linear_bwd_workspace(M: int, N: int, K: int, device="cuda") -> torch.Tensor:
    return torch.empty(fp8_linear_bwd_workspace_size(M, N, K), dtype=torch.uint8, device=device)


def fp8_linear_bwd(dY: torch.Tensor, saved: dict, K: int, *, dx_dtype=torch.bfloat16, dX: torch.Tensor | None = None,
                   dW: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """(dX, dW) of fp8_linear_fwd from its saved operands: dY quantized along the features and along the tokens, W-hat
    as it is and X-hat regrouped along the tokens."""
    index = _tensor(dY, "dY", 2)
    yp = _arg(dY, "dY", _BF16, index)
    M, N = dY.shape
    if dX is None:
        dX = torch.empty((M, K), dtype=dx_dtype, device=index)
    if dW is None:
        dW = torch.empty((N, K), dtype=torch.float32, device=index)
    workspace, sp, sn = _room(workspace, fp8_linear_bwd_workspace_size(M, N, K), index)
    _run("fp8_linear_bwd", index, yp, M, N, K, _q(saved["Xq"], "Xq", index, M, K), _q(saved["Wq"], "Wq", index, N, K, (FP8_BLOCK,)),
         _arg(dX, "dX", _OUT, index, (M, K)), _CODE[dX.dtype], _arg(dW, "dW", _F32, index, (N, K)), sp, sn)
    return dX, dW
