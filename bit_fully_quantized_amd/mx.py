"""MXFP4 operands and the linear layer on them (the mxfp4_ entry points of include/tj2.h).

MXFP4 stores E2M1 elements under one power-of-two scale per 32, the form gfx950's scaled matrix
instructions take as it is.  Names and arguments follow the NVFP4 functions of the package; work runs on
the current stream of the tensors' device.

Decoding calls these functions once a token and layer, so a call costs about what its launches do: one
pass over the arguments that yields their pointers, and the reason of a refusal only where there is one.
"""
from __future__ import annotations

import ctypes
from functools import lru_cache

import torch

from . import _BF16, _F32, GROUP_COL, GROUP_ROW, MXFP4, RTN, SR, QTensor, _dense, _matrix_out, check, lib
from ._lib import BF16, F32

_OUT = (torch.bfloat16, torch.float32)
_U8 = (torch.uint8,)
_CODE = {torch.bfloat16: BF16, torch.float32: F32}
_byref = ctypes.byref
_FN: dict = {}  # entry points by name
_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _tensor(t, name: str, dim: int | None = None) -> int:
    """The device index of tensor argument `name`, which is on a GPU."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA (HIP) tensor")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name} must be {dim}-D")
    return t.get_device()


def _arg(t, name: str, dtypes, index: int, shape=None, optional: bool = False) -> int:
    """The pointer of a dense argument on device `index` (0 for None where that may be)."""
    if t is None and optional:
        return 0
    if (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.is_contiguous() and t.get_device() == index
            and (shape is None or t.shape == shape)):
        return t.data_ptr()
    _dense(t, name, dtypes, shape)
    raise ValueError(f"{name} is on cuda:{t.get_device()}, other arguments on cuda:{index}")


def _q(q, name: str, index: int, rows: int | None = None, length: int | None = None):
    """The descriptor of an MXFP4 argument on device `index`."""
    if not isinstance(q, QTensor) or q.fmt != MXFP4:
        raise ValueError(f"{name} must be an MXFP4 QTensor")
    if (rows is not None and q.rows != rows) or (length is not None and q.len != length):
        raise ValueError(f"{name} is [{q.rows}, {q.len}], expected [{rows}, {length}]")
    t = q.storage()
    if t.get_device() != index or (t is not q.buffer and q.scale16.get_device() != index):
        raise ValueError(f"{name} must be on cuda:{index}, with the other arguments")
    return _byref(q.c())


def _run(name: str, index: int, *args) -> None:
    """Entry point `name` on the current stream of device `index`, made current for the call if it is not."""
    fn = _FN.get(name) or _FN.setdefault(name, getattr(lib(), name))
    if _device() == index:
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status:
        check(name, status)


def _room(workspace, size: int, index: int):
    """(workspace, its pointer, its bytes); allocated if not given and size is not 0."""
    if workspace is None:
        if not size:
            return None, 0, 0
        workspace = torch.empty(size, dtype=torch.uint8, device=index)
    return workspace, _arg(workspace, "workspace", _U8, index), workspace.numel()


def mx_quantize(x, *, grouping: int = GROUP_ROW, rounding: int = RTN, rht: bool = False, signs: int = 0, seed: int = 0,
                offset: int = 0, out: QTensor | None = None) -> QTensor:
    """Quantize a dense bf16/fp32 tensor [rows, cols], or regroup an MXFP4 QTensor (GROUP_COL), to MXFP4.

    GROUP_ROW groups along cols; GROUP_COL along rows, stored transposed as [cols, rows].  RTN takes the
    scale 2^(floor(log2 amax) - 2); SR the smallest one that saturates nothing, with Philox draws of
    (seed, offset).  rht applies the 16-wide Hadamard transform with the sign mask `signs` first."""
    if isinstance(x, QTensor):
        index = _tensor(x.storage(), "x")
        rows, cols, xp, xd, xq = x.rows, x.len, 0, MXFP4, _q(x, "x", index)
    else:
        index = _tensor(x, "x", 2)
        xp, xd, xq = _arg(x, "x", _OUT, index), _CODE[x.dtype], None
        rows, cols = x.shape
    if out is None:
        if rows <= 0 or cols <= 0:
            raise ValueError("x must not be empty")
        out = QTensor(MXFP4, rows, cols, index) if grouping == GROUP_ROW else QTensor(MXFP4, cols, rows, index)
    _run("mxfp4_quantize", index, xp, xd, xq, rows, cols, grouping, rounding, 1 if rht else 0, signs, seed, offset,
         _q(out, "out", index))
    return out


def mx_dequantize(q: QTensor, *, dtype=torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """The values of an MXFP4 QTensor as a dense [rows, len] tensor (bf16 holds them exactly)."""
    if not isinstance(q, QTensor):
        raise ValueError("q must be an MXFP4 QTensor")
    index = _tensor(q.storage(), "q")
    desc = _q(q, "q", index)
    if out is None:
        out = torch.empty((q.rows, q.len), dtype=dtype, device=index)
    _run("mxfp4_dequantize", index, desc, _arg(out, "out", _OUT, index, (q.rows, q.len)), _CODE[out.dtype])
    return out


@lru_cache(maxsize=4096)
def _gemm_bytes(I: int, J: int, K: int) -> int:
    return int(lib().mxfp4_gemm_workspace_size(I, J, K))


@lru_cache(maxsize=4096)
def mx_linear_bwd_workspace_size(M: int, N: int, K: int) -> int:
    """Bytes of the workspace of mx_linear_bwd."""
    return int(lib().mxfp4_linear_bwd_workspace_size(M, N, K))


def mx_gemm_workspace(I: int, J: int, K: int, device="cuda") -> torch.Tensor | None:
    """Workspace of an I x J product over K, or None where none is needed."""
    n = _gemm_bytes(I, J, K)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def mx_gemm(A: QTensor, B: QTensor, *, out: torch.Tensor | None = None, out_dtype=torch.float32, accumulate: bool = False,
            workspace: torch.Tensor | None = None) -> torch.Tensor:
    """C = A B^T (accumulate: added into a float32 `out`) on MXFP4 operands grouped along the reduction."""
    if not isinstance(A, QTensor) or not isinstance(B, QTensor):
        raise ValueError("A and B must be MXFP4 QTensors")
    index = _tensor(A.storage(), "A")
    a, b = _q(A, "A", index), _q(B, "B", index, B.rows, A.len)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = torch.empty((A.rows, B.rows), dtype=out_dtype, device=index)
    _matrix_out(out, "out", _OUT, A.rows, B.rows)
    if out.get_device() != index:
        raise ValueError(f"out is on cuda:{out.get_device()}, other arguments on cuda:{index}")
    workspace, wp, wn = _room(workspace, _gemm_bytes(A.rows, B.rows, A.len), index)
    _run("mxfp4_gemm", index, a, b, out.data_ptr(), _CODE[out.dtype], max(out.stride(0), B.rows), 1 if accumulate else 0, wp, wn)
    return out


def mx_linear_fwd(X: torch.Tensor, W_master: torch.Tensor | None, N: int, *, Wq: QTensor | None = None,
                  y_dtype=torch.bfloat16, Y: torch.Tensor | None = None, Xq: QTensor | None = None,
                  workspace: torch.Tensor | None = None):
    """Y = X W^T with MXFP4 operands; returns (Y, saved) with saved = dict(Xq, Wq).

    W_master (fp32 [N, K]) is quantized into Wq; without it Wq is used as given.  X has any number of rows."""
    index = _tensor(X, "X", 2)
    xp = _arg(X, "X", _BF16, index)
    M, K = X.shape
    if W_master is None and Wq is None:
        raise ValueError("W_master or Wq is required")
    wp = _arg(W_master, "W_master", _F32, index, (N, K), optional=True)
    if Wq is None:
        Wq = QTensor(MXFP4, N, K, index)
    if Xq is None:
        Xq = QTensor(MXFP4, M, K, index)
    if Y is None:
        Y = torch.empty((M, N), dtype=y_dtype, device=index)
    workspace, sp, sn = _room(workspace, _gemm_bytes(M, N, K), index)
    _run("mxfp4_linear_fwd", index, xp, M, K, N, wp, _q(Wq, "Wq", index, N, K), _q(Xq, "Xq", index, M, K),
         _arg(Y, "Y", _OUT, index, (M, N)), _CODE[Y.dtype], sp, sn)
    return Y, {"Xq": Xq, "Wq": Wq}


def mx_linear_bwd_workspace(M: int, N: int, K: int, device="cuda") -> torch.Tensor:
    return torch.empty(mx_linear_bwd_workspace_size(M, N, K), dtype=torch.uint8, device=device)


def mx_linear_bwd(dY: torch.Tensor, saved: dict, K: int, *, seed: int, offset: int, rht: bool = True, rounding: int = SR,
                  dx_dtype=torch.bfloat16, dX: torch.Tensor | None = None, dW: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None):
    """(dX, dW) of mx_linear_fwd from its saved operands: dY, W-hat and X-hat regrouped to MXFP4 along each
    product's reduction, stochastically rounded and Hadamard-transformed unless told otherwise."""
    index = _tensor(dY, "dY", 2)
    yp = _arg(dY, "dY", _BF16, index)
    M, N = dY.shape
    if dX is None:
        dX = torch.empty((M, K), dtype=dx_dtype, device=index)
    if dW is None:
        dW = torch.empty((N, K), dtype=torch.float32, device=index)
    workspace, sp, sn = _room(workspace, mx_linear_bwd_workspace_size(M, N, K), index)
    _run("mxfp4_linear_bwd", index, yp, M, N, K, _q(saved["Xq"], "Xq", index, M, K), _q(saved["Wq"], "Wq", index, N, K),
         rounding, 1 if rht else 0, seed, offset, _arg(dX, "dX", _OUT, index, (M, K)), _CODE[dX.dtype],
         _arg(dW, "dW", _F32, index, (N, K)), sp, sn)
    return dX, dW
