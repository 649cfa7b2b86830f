"""The FP8 and norm entry points refuse bad arguments on the host, before any device work (CPU)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from bit_fully_quantized_amd import _lib
    return _lib


def q(lib, fmt, rows, length, codes=0x100000, scale=0x200000):
    return lib.QTensorC(codes, 0, scale, rows, length, fmt, 0)


def test_sizes(lib):
    L = lib.lib()
    c, s, t = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    assert L.tj2_qtensor_bytes(lib.FP8_BLOCK, 300, 272, ctypes.byref(c), ctypes.byref(s), ctypes.byref(t)) == 0
    assert (c.value, s.value, t.value) == (300 * 3 * 128, 0, 3 * 3 * 4)
    assert L.tj2_qtensor_bytes(lib.FP8_BLOCK, 300, 40, ctypes.byref(c), ctypes.byref(s), ctypes.byref(t)) == lib.TJ2_ERR_SHAPE
    for f in (L.fp8_gemm_workspace_size, L.fp8_linear_fwd_workspace_size, L.fp8_linear_bwd_workspace_size):
        assert f(0, 16, 16) == 0 and f(16, -1, 16) == 0 and f(16, 16, 0) == 0
    assert L.tj2_rms_norm_bwd_workspace_size(0, 5) == 0 and L.tj2_rms_norm_bwd_workspace_size(7, 5) > 0
    # one token needs no workspace, and a reduction that is split its partial sums
    assert L.fp8_linear_fwd_workspace_size(1, 4096, 1024) == 0
    assert L.fp8_gemm_workspace_size(128, 128, 16384) % (128 * 128 * 4) == 0 and L.fp8_gemm_workspace_size(128, 128, 16384) > 0


def test_quantize(lib):
    L = lib.lib()
    ARG, SHAPE, ALIGN, NO = lib.TJ2_ERR_ARG, lib.TJ2_ERR_SHAPE, lib.TJ2_ERR_ALIGN, lib.TJ2_ERR_UNSUPPORTED

    def run(x=0x1000, dt=lib.F32, xq=None, rows=32, cols=64, grouping=0, out=None):
        out = q(lib, lib.FP8, rows, cols) if out is None else out
        return L.fp8_quantize(x, dt, xq, rows, cols, grouping, ctypes.byref(out) if out else None, None)
    assert run(x=None) == ARG and run(x=0x1008) == ALIGN and run(dt=lib.NVFP4) == ARG and run(grouping=2) == ARG and run(out=0) == ARG
    assert run(rows=0) == SHAPE and run(cols=0) == SHAPE and run(cols=40) == SHAPE and run(cols=(1 << 22) + 16) == SHAPE
    assert run(rows=1 << 27) == SHAPE and run(rows=-5) == SHAPE
    assert run(out=q(lib, lib.NVFP4, 32, 64)) == ARG and run(out=q(lib, lib.FP8, 32, 80)) == SHAPE
    assert run(grouping=1) == SHAPE  # [cols, rows] expected
    assert run(grouping=1, out=q(lib, lib.FP8_BLOCK, 64, 32)) == ARG
    assert run(grouping=1, rows=40, out=q(lib, lib.FP8, 64, 40)) == SHAPE
    assert run(out=q(lib, lib.FP8, 32, 64, codes=0x100008)) == ALIGN and run(out=q(lib, lib.FP8, 32, 64, scale=0)) == ARG
    src = q(lib, lib.FP8, 32, 64)
    assert run(x=None, dt=lib.FP8, xq=ctypes.byref(src)) == NO
    assert run(x=None, dt=lib.FP8, xq=None, grouping=1, out=q(lib, lib.FP8, 64, 32)) == ARG
    assert run(x=None, dt=lib.FP8, xq=ctypes.byref(src), grouping=1, out=q(lib, lib.FP8, 64, 32)) == ARG  # its own arrays
    blk = q(lib, lib.FP8_BLOCK, 32, 64)
    assert run(x=None, dt=lib.FP8, xq=ctypes.byref(blk), grouping=1, out=q(lib, lib.FP8, 64, 32, 0x300000, 0x400000)) == ARG
    good = q(lib, lib.FP8, 32, 64)
    assert L.fp8_dequantize(None, 0x1000, lib.F32, None) == ARG and L.fp8_dequantize(ctypes.byref(good), None, lib.F32, None) == ARG
    assert L.fp8_dequantize(ctypes.byref(good), 0x1000, lib.FP8, None) == ARG
    assert L.fp8_dequantize(ctypes.byref(good), 0x1004, lib.F32, None) == ALIGN


def test_products(lib):
    L = lib.lib()
    ARG, SHAPE, ALIGN, NO = lib.TJ2_ERR_ARG, lib.TJ2_ERR_SHAPE, lib.TJ2_ERR_ALIGN, lib.TJ2_ERR_UNSUPPORTED
    A, B = q(lib, lib.FP8, 32, 256), q(lib, lib.FP8_BLOCK, 48, 256)

    def run(a=A, b=B, C=0x1000, dt=lib.F32, ldc=48, acc=0, ws=None, n=0):
        return L.fp8_gemm(ctypes.byref(a) if a else None, ctypes.byref(b) if b else None, C, dt, ldc, acc, ws, n, None)
    assert run(a=None) == ARG and run(b=None) == ARG and run(C=None) == ARG and run(dt=lib.FP8) == ARG
    assert run(a=B) == ARG and run(b=q(lib, lib.NVFP4, 48, 256)) == ARG
    assert run(b=q(lib, lib.FP8, 48, 272)) == SHAPE and run(ldc=47) == SHAPE and run(dt=lib.BF16, acc=1) == NO
    assert run(C=0x1002) == ALIGN and run(dt=lib.BF16, C=0x1001) == ALIGN
    big, other = q(lib, lib.FP8, 128, 16384), q(lib, lib.FP8, 128, 16384)
    need = L.fp8_gemm_workspace_size(128, 128, 16384)
    assert run(a=big, b=other, ldc=128, ws=0x10000, n=need - 1) == ARG and b"needed" in L.tj2_last_error()
    assert run(a=big, b=other, ldc=128, ws=0x10008, n=need) == ALIGN

    Xq, Wq = q(lib, lib.FP8, 3, 64), q(lib, lib.FP8_BLOCK, 48, 64)

    def fwd(X=0x1000, M=3, K=64, N=48, W=None, wq=Wq, xq=Xq, Y=0x2000, dt=lib.BF16):
        return L.fp8_linear_fwd(X, M, K, N, W, ctypes.byref(wq) if wq else None, ctypes.byref(xq) if xq else None, Y, dt, None, 0, None)
    assert fwd(Y=None) == ARG and fwd(wq=None) == ARG and fwd(xq=None) == ARG and fwd(dt=lib.MXFP4) == ARG
    assert fwd(M=0) == SHAPE and fwd(K=40) == SHAPE and fwd(N=40) == SHAPE and fwd(M=4) == SHAPE
    assert fwd(wq=q(lib, lib.FP8, 48, 64)) == ARG and fwd(xq=q(lib, lib.FP8_BLOCK, 3, 64)) == ARG
    assert fwd(X=0x1002) == ALIGN and fwd(W=0x3004) == ALIGN and fwd(Y=0x2008) == ALIGN
    need = L.fp8_linear_bwd_workspace_size(3, 48, 64)

    def bwd(dY=0x1000, dX=0x2000, dt=lib.BF16, dW=0x3000, ws=0x10000, n=need, M=3, xq=Xq):
        return L.fp8_linear_bwd(dY, M, 48, 64, ctypes.byref(xq), ctypes.byref(Wq), dX, dt, dW, ws, n, None)
    assert bwd(dY=None) == ARG and bwd(dX=None) == ARG and bwd(dW=None) == ARG and bwd(ws=None) == ARG and bwd(n=need - 1) == ARG
    assert bwd(dt=lib.FP8) == ARG and bwd(M=0) == SHAPE and bwd(M=5) == SHAPE
    assert bwd(dY=0x1008) == ALIGN and bwd(dX=0x2002) == ALIGN and bwd(dW=0x3004) == ALIGN and bwd(ws=0x10004) == ALIGN
    long = (1 << 22) + 16  # tokens that a transposed operand could not hold
    assert bwd(M=long, xq=q(lib, lib.FP8, long, 64), n=1 << 62) == SHAPE


def test_norm(lib):
    L = lib.lib()
    ARG, SHAPE, ALIGN = lib.TJ2_ERR_ARG, lib.TJ2_ERR_SHAPE, lib.TJ2_ERR_ALIGN

    def fwd(x=0x1000, ldx=64, res=None, ldr=64, dt=lib.BF16, rows=3, cols=64, w=0x2000, wd=lib.F32, eps=1e-6, s=None, y=0x4000,
            yq=None, rstd=0x5000):
        return L.tj2_rms_norm_fwd(x, ldx, res, ldr, dt, rows, cols, w, wd, ctypes.c_float(eps), s, y, ctypes.byref(yq) if yq else None,
                                  rstd, None)
    assert fwd(x=None) == ARG and fwd(w=None) == ARG and fwd(y=None) == ARG and fwd(dt=lib.FP8) == ARG and fwd(wd=9) == ARG
    assert fwd(res=0x6000) == ARG and fwd(s=0x6000) == ARG
    for eps in (-1.0, float("nan"), float("inf")):
        assert fwd(eps=eps) == ARG
    assert fwd(rows=0) == SHAPE and fwd(cols=0) == SHAPE and fwd(cols=(1 << 22) + 1, ldx=1 << 23) == SHAPE and fwd(ldx=63) == SHAPE
    assert fwd(res=0x6000, s=0x7000, ldr=60) == SHAPE
    assert fwd(x=0x1001) == ALIGN and fwd(dt=lib.F32, x=0x1002) == ALIGN and fwd(w=0x2002) == ALIGN and fwd(rstd=0x5002) == ALIGN
    yq = q(lib, lib.FP8, 3, 64)
    assert fwd(yq=yq) == ARG  # y too
    assert fwd(y=None, yq=q(lib, lib.FP8, 4, 64)) == SHAPE and fwd(y=None, yq=q(lib, lib.FP8_BLOCK, 3, 64)) == ARG
    assert fwd(y=None, yq=yq, x=0x1008) == ALIGN and fwd(y=None, yq=yq, ldx=68) == ALIGN and fwd(y=None, yq=yq, w=0x2004) == ALIGN
    assert fwd(y=None, yq=yq, res=0x6000, s=0x7002) == ALIGN and fwd(y=None, yq=yq, res=0x6000, s=0x7000, ldr=66) == ALIGN
    need = L.tj2_rms_norm_bwd_workspace_size(3, 64)

    def bwd(dy=0x1000, lddy=64, s=0x2000, lds=64, dt=lib.F32, rows=3, w=0x3000, wd=lib.F32, rstd=0x4000, dsum=None, ldd=64, ds=0x5000,
            dw=0x6000, ws=0x10000, n=need):
        return L.tj2_rms_norm_bwd(dy, lddy, s, lds, dt, rows, 64, w, wd, rstd, dsum, ldd, ds, dw, ws, n, None)
    assert bwd(dy=None) == ARG and bwd(s=None) == ARG and bwd(w=None) == ARG and bwd(rstd=None) == ARG and bwd(ds=None, dw=None) == ARG
    assert bwd(ws=None) == ARG and bwd(n=need - 1) == ARG and bwd(dt=lib.NVFP4) == ARG
    assert bwd(rows=0) == SHAPE and bwd(lddy=60) == SHAPE and bwd(lds=60) == SHAPE and bwd(dsum=0x7000, ldd=63) == SHAPE
    assert bwd(dy=0x1002) == ALIGN and bwd(dw=0x6002) == ALIGN and bwd(rstd=0x4001) == ALIGN and bwd(ws=0x10008) == ALIGN
    assert bwd(ds=0x5002) == ALIGN


def test_binding():
    import bit_fully_quantized_amd as tj2
    x, w = torch.zeros(2, 16), torch.zeros(16)
    for f in (lambda: tj2.rms_norm_fwd(x, w), lambda: tj2.rms_norm(x, w), lambda: tj2.rms_norm_bwd(x, x, w, w), lambda: tj2.fp8_quantize(x),
              lambda: tj2.fp8_linear_fwd(x.bfloat16(), x, 16), lambda: tj2.fp8_gemm(x, x), lambda: tj2.fp8_dequantize(x)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(ValueError):
        tj2.QTensor(tj2.FP8_BLOCK, 4, 40)
    with pytest.raises(ValueError):
        tj2.QTensor.packed(tj2.NVFP4, 4, 32)


def test_results_in_an_inputs_place(lib):
    """A dense result over an input of another pitch, or over another result, is refused."""
    L, ARG = lib.lib(), lib.TJ2_ERR_ARG

    def fwd(x=0x1000, ldx=64, res=0x6000, ldr=64, s=0x7000, y=0x4000):
        return L.tj2_rms_norm_fwd(x, ldx, res, ldr, lib.BF16, 3, 64, 0x2000, lib.F32, ctypes.c_float(1e-6), s, y, None, 0x5000, None)
    assert fwd(s=0x1000, ldx=72) == ARG and fwd(s=0x6000, ldr=72) == ARG and fwd(y=0x7000) == ARG
    assert fwd(y=0x1000, ldx=72) == ARG and fwd(y=0x6000, ldr=72) == ARG
    assert fwd(res=None, s=None, y=0x1000, ldx=72) == ARG
    need = L.tj2_rms_norm_bwd_workspace_size(3, 64)

    def bwd(dy=0x1000, lddy=64, s=0x2000, lds=64, dsum=0x8000, ldd=64, ds=0x5000):
        return L.tj2_rms_norm_bwd(dy, lddy, s, lds, lib.F32, 3, 64, 0x3000, lib.F32, 0x4000, dsum, ldd, ds, 0x6000, 0x10000, need, None)
    assert bwd(ds=0x1000, lddy=72) == ARG and bwd(ds=0x2000, lds=72) == ARG and bwd(ds=0x8000, ldd=72) == ARG
    Xq, Wq, need = q(lib, lib.FP8, 3, 64), q(lib, lib.FP8_BLOCK, 48, 64), L.fp8_linear_bwd_workspace_size(3, 48, 64)
    assert L.fp8_linear_bwd(0x1000, 3, 48, 64, ctypes.byref(Xq), ctypes.byref(Wq), 0x2000, lib.BF16, 0x2000, 0x10000, need, None) == ARG
