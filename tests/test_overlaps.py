"""Results that lie partly over one another or over an input are refused on the host, before any device work (CPU)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from bit_fully_quantized_amd import _lib
    return _lib


def refused(lib, status):
    return status == lib.TJ2_ERR_ARG and b"overlap" in lib.lib().tj2_last_error()


def q(lib, fmt, rows, length, codes, scale):
    return ctypes.byref(lib.QTensorC(codes, 0, scale, rows, length, fmt, 0))


def test_norm(lib):
    L, row = lib.lib(), 64 * 2  # 3 rows of 64 bf16, 72 apart where a pitch is given

    def fwd(x=0x100000, ldx=72, res=0x200000, ldr=72, w=0x300000, s=0x400000, y=0x500000, yq=None, rstd=0x600000):
        return L.tj2_rms_norm_fwd(x, ldx, res, ldr, lib.BF16, 3, 64, w, lib.F32, ctypes.c_float(1e-6), s, y, yq, rstd, None)
    end = 2 * 144 + row  # of x and residual
    for at in (0, 2, row - 2, 144, -3 * row + 2, end - 2):
        assert refused(lib, fwd(s=0x100000 + at)) and refused(lib, fwd(s=0x200000 + at)), at
        assert refused(lib, fwd(y=0x100000 + at)) and refused(lib, fwd(y=0x200000 + at)), at
    for at in (2, 3 * row - 2, -3 * row + 2):  # dense inputs may be replaced whole, not in part
        assert refused(lib, fwd(ldx=64, s=0x100000 + at)) and refused(lib, fwd(ldr=64, y=0x200000 + at)), at
        assert refused(lib, fwd(y=0x400000 + at)), at
    assert refused(lib, fwd(y=0x400000))
    for at in (-3 * row + 2, 64 * 4 - 2):
        assert refused(lib, fwd(s=0x300000 + at)) and refused(lib, fwd(y=0x300000 + at)), at
    for at in (0x100000, 0x200000 + 2 * 144 + row - 4, 0x300000 + 252, 0x400000 + 3 * row - 4, 0x500000 - 8):
        assert refused(lib, fwd(rstd=at)), hex(at)
    for codes, scale in ((0x100000, 0x700000), (0x200100, 0x700000), (0x400010, 0x700000), (0x700000, 0x300010), (0x700000, 0x600000)):
        assert refused(lib, fwd(y=None, yq=q(lib, lib.FP8, 3, 64, codes, scale))), (hex(codes), hex(scale))
    need = L.tj2_rms_norm_bwd_workspace_size(3, 64)

    def bwd(dy=0x100000, lddy=72, s=0x200000, lds=72, w=0x300000, rstd=0x400000, dsum=0x500000, ldd=72, ds=0x600000, dw=0x700000):
        return L.tj2_rms_norm_bwd(dy, lddy, s, lds, lib.BF16, 3, 64, w, lib.BF16, rstd, dsum, ldd, ds, dw, 0x800000, need, None)
    for base in (0x100000, 0x200000, 0x500000):
        for at in (0, 2, 144, -3 * row + 2, end - 2):
            assert refused(lib, bwd(ds=base + at)), (hex(base), at)
        for at in (0, -row + 2, end - 2):
            assert refused(lib, bwd(dw=base + at)), (hex(base), at)
    assert refused(lib, bwd(dw=0x600000)) and refused(lib, bwd(dw=0x600000 + 3 * row - 2)) and refused(lib, bwd(dw=0x600000 - row + 2))
    assert refused(lib, bwd(ds=0x300000)) and refused(lib, bwd(ds=0x400004)) and refused(lib, bwd(dw=0x300002)) and refused(lib, bwd(dw=0x400008))
    assert refused(lib, bwd(dy=0x100000, lddy=64, ds=0x100002)) and refused(lib, bwd(lds=1 << 61, ds=0x200000 + row - 2))


def test_fp8(lib):
    L = lib.lib()

    def quantize(x=0x100000, dt=lib.F32, xq=None, grouping=0, codes=0x200000, scale=0x300000, fmt=lib.FP8):  # 32 x 64
        out = q(lib, fmt, *((32, 64) if grouping == 0 else (64, 32)), codes, scale)
        return L.fp8_quantize(x, dt, xq, 32, 64, grouping, out, None)
    size = 32 * 64 * 4
    for at in (0, 16, size - 16, -32 * 128 + 16):
        assert refused(lib, quantize(codes=0x100000 + at)) and refused(lib, quantize(codes=0x100000 + at, fmt=lib.FP8_BLOCK)), at
    assert refused(lib, quantize(scale=0x100000 + size - 16)) and refused(lib, quantize(scale=0x100000 - 32 * 4 + 16))
    src = dict(x=None, dt=lib.FP8, xq=q(lib, lib.FP8, 32, 64, 0x100000, 0x400000), grouping=1)
    for kw in (dict(codes=0x100000), dict(codes=0x100000 + 32 * 128 - 16), dict(codes=0x400000), dict(scale=0x100010), dict(scale=0x400070)):
        assert refused(lib, quantize(**src, **kw)), kw
    good = q(lib, lib.FP8, 32, 64, 0x100000, 0x400000)
    for at in (0x100000, 0x100000 + 32 * 128 - 16, 0x100000 - size + 16, 0x400000 + 112):
        assert refused(lib, L.fp8_dequantize(good, at, lib.F32, None)), hex(at)

    A, B = q(lib, lib.FP8, 32, 256, 0x100000, 0x200000), q(lib, lib.FP8_BLOCK, 48, 256, 0x300000, 0x400000)
    for C in (0x100000, 0x100000 + 32 * 256 - 4, 0x200000, 0x300000 - 31 * 200 * 4, 0x300000 + 48 * 256 - 4, 0x400004):
        assert refused(lib, L.fp8_gemm(A, B, C, lib.F32, 200, 0, None, 0, None)), hex(C)

    def fwd(X=0x100000, W=0x200000, Y=0x300000, xc=0x400000, xs=0x500000, wc=0x600000, ws=0x700000):  # M 3, K 64, N 48
        return L.fp8_linear_fwd(X, 3, 64, 48, W, q(lib, lib.FP8_BLOCK, 48, 64, wc, ws), q(lib, lib.FP8, 3, 64, xc, xs), Y, lib.BF16, None, 0,
                                None)
    places = dict(X=(0x100000, 3 * 64 * 2), W=(0x200000, 48 * 64 * 4), Y=(0x300000, 3 * 48 * 2), xc=(0x400000, 3 * 128), xs=(0x500000, 12),
                  wc=(0x600000, 48 * 128), ws=(0x700000, 4))
    for a in ("Y", "xc", "xs", "wc", "ws"):
        for b in places:
            if a != b and {a, b} not in ({"xc", "xs"}, {"wc", "ws"}):
                at, n = places[b]
                for to in {at, at + (n - 1) // 16 * 16}:
                    assert refused(lib, fwd(**{a: to})), (a, b, hex(to))
    need = L.fp8_linear_bwd_workspace_size(3, 48, 64)

    def bwd(dX=0x300000, dW=0x800000, dt=lib.BF16):
        return L.fp8_linear_bwd(0x100000, 3, 48, 64, q(lib, lib.FP8, 3, 64, 0x400000, 0x500000), q(lib, lib.FP8_BLOCK, 48, 64, 0x600000, 0x700000),
                                dX, dt, dW, 0x900000, need, None)
    for at, n in ((0x100000, 3 * 48 * 2), (0x400000, 3 * 128), (0x500000, 12), (0x600000, 48 * 128), (0x700000, 4)):
        for to in {at, at + (n - 1) // 16 * 16}:
            assert refused(lib, bwd(dX=to)) and refused(lib, bwd(dW=to)), hex(to)
    assert refused(lib, bwd(dX=0x800000)) and refused(lib, bwd(dX=0x800000 + 48 * 64 * 4 - 16)) and refused(lib, bwd(dW=0x300000 + 3 * 64 * 2 - 16))


def test_feed_forward_block(lib):
    L, T, D, F = lib.lib(), 5, 64, 96
    need, saved = L.tj2_gated_ffn_fwd_workspace_size(T, D, F), L.tj2_gated_ffn_saved_size(T, F)

    def fwd(X=0x100000, Wg=0x200000, Wu=0x300000, Wd=0x400000, gu=0x500000, Y=0x600000):
        return L.tj2_gated_ffn_fwd(X, 72, Wg, Wu, 72, Wd, 104, T, D, F, 0, gu, Y, lib.F32, 0x900000, need, None)
    wd_end = 0x400000 + (D - 1) * 104 * 2 + F * 2
    for Y in (0x400000, 0x400000 + 112, wd_end - 16, 0x400000 - T * D * 4 + 16, 0x500000, 0x500000 + saved - 16):
        assert refused(lib, fwd(Y=Y)), hex(Y)
    for gu in (0x100000, 0x200000, 0x300000 - saved + 16, wd_end - 16, 0x600000 + T * D * 4 - 16):
        assert refused(lib, fwd(gu=gu)), hex(gu)
    need = L.tj2_gated_ffn_bwd_workspace_size(T, D, F)

    def bwd(dX=0x700000, dWg=0x800000, dWu=0x900000, dWd=0xA00000):
        return L.tj2_gated_ffn_bwd(0x600000, 72, 0x100000, 72, 0x200000, 0x300000, 72, 0x400000, 104, T, D, F, 0, 0x500000, dX, lib.F32, dWg,
                                   dWu, dWd, lib.F32, 0xB00000, need, None)
    for k in ("dX", "dWg", "dWu", "dWd"):
        for at in (0x600000, 0x600000 + 4 * 144 + 112, 0x100000, 0x200000 + 95 * 144 + 112, 0x300000 + 16, wd_end - 16, 0x500000 + saved - 16):
            assert refused(lib, bwd(**{k: at})), (k, hex(at))
    whole = F * D * 4
    for a, b, at in (("dX", "dWg", 0x800000), ("dWg", "dWu", 0x900000), ("dWu", "dWd", 0xA00000), ("dWg", "dWd", 0xA00000)):
        for to in (at, at + 16, at + whole - 16):
            assert refused(lib, bwd(**{a: to})), (a, b)
