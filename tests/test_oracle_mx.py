"""The MXFP4 oracle against brute force and closed forms (CPU), and the refusals of its entry points."""
import ctypes

import numpy as np
import pytest

from oracle import formats, mx

RNG = np.random.default_rng(0)
GRID = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])


def test_scale_rules_at_the_borders():
    for e in (-120, -3, 0, 5, 120):
        s = 2.0 ** e
        assert mx.scale_byte(4.0 * s, "rtn") == e + 127          # 4 is E2M1's top binade
        assert mx.scale_byte(np.nextafter(np.float32(8.0 * s), np.float32(0)), "rtn") == e + 127
        assert mx.scale_byte(6.0 * s, "sr") == e + 127           # 6 still fits
        assert mx.scale_byte(float(np.nextafter(np.float32(6.0 * s), np.float32(np.inf))), "sr") == e + 128
    assert mx.scale_byte(0.0, "rtn") == 0 and mx.scale_byte(2.0 ** -149, "sr") == 0
    assert mx.scale_byte(np.inf, "rtn") == 255 and mx.scale_byte(np.nan, "sr") == 255


@pytest.mark.parametrize("L", [1, 31, 32, 33, 100, 128])
def test_rtn_takes_a_nearest_grid_value(L):
    x = (RNG.standard_normal((5, L)) * np.exp2(RNG.integers(-30, 30, (5, 1)))).astype(np.float32)
    q = mx.quantize(x)
    v = mx.dequantize(q)
    s = np.repeat(np.ldexp(1.0, q.scale.astype(int) - 127), 32, axis=1)[:, :L]
    a = np.minimum(np.abs(x) / s, 6.0)
    best = np.abs(a[..., None] - GRID).min(axis=-1)
    np.testing.assert_array_equal(np.abs(np.abs(v) / s - a), best)
    assert ((np.abs(x) / s).max(axis=1) < 8.0).all()


def test_sr_is_unbiased_and_never_saturates():
    x = np.linspace(-6.4, 6.4, 96, dtype=np.float32)[None, :].repeat(4096, axis=0)
    q = mx.quantize(x, rounding="sr", seed=3, offset=9)
    v = mx.dequantize(q)
    s = np.repeat(np.ldexp(1.0, q.scale[0].astype(int) - 127), 32)
    # draws have 16 bits (bias below a gap / 65536); the mean of 4096 roundings is within 6 standard
    # deviations, each at most half a gap (2 s) / sqrt(4096)
    assert (np.abs(v.mean(axis=0) - x[0]) <= 6 * 0.5 * 2 * s / 64 + 2 * s / 65536).all()


def test_special_groups_and_codes():
    x = np.zeros((3, 64), dtype=np.float32)
    x[0, 5] = np.nan
    x[1, 40] = np.inf
    x[1, 41] = 3.0
    x[2, 3] = -0.0
    q = mx.quantize(x)
    assert q.scale.tolist() == [[255, 0], [0, 255], [0, 0]]
    v = mx.dequantize(q)
    assert np.isnan(v[0, :32]).all() and (v[0, 32:] == 0).all() and np.isnan(v[1, 32:]).all()
    assert formats.e2m1_decode(q.codes[2, 1] >> 4) == 0.0 and np.signbit(v[2, 3])


def test_transform_cancels_in_a_product_with_a_ragged_end():
    a, b = RNG.standard_normal((3, 37)).astype(np.float32), RNG.standard_normal((4, 37)).astype(np.float32)
    ta, tb = mx.transform(a, 0xBEEF), mx.transform(b, 0xBEEF)
    # fp32 butterflies: 5 roundings of half a step (2^-24) a value, relative to the row norms
    bound = 10 * 2.0 ** -24 * np.linalg.norm(a, axis=1)[:, None] * np.linalg.norm(b, axis=1)[None, :] * 4
    assert (np.abs(ta.astype(np.float64) @ tb.T - a.astype(np.float64) @ b.T) <= bound).all()
    np.testing.assert_array_equal(ta[:, 32:], a[:, 32:])


def fake(rows, length, fmt=5, base=0x10000):
    from bit_fully_quantized_amd import _lib
    return _lib.QTensorC(base, base + 0x1000, 0, rows, length, fmt, 0)


def test_entry_points_refuse_on_the_host():
    from bit_fully_quantized_amd import _lib
    L = _lib.lib()
    ref = ctypes.byref
    ARG, SHAPE, ALIGN, UNS = _lib.TJ2_ERR_ARG, _lib.TJ2_ERR_SHAPE, _lib.TJ2_ERR_ALIGN, _lib.TJ2_ERR_UNSUPPORTED

    def quant(x=0x1000, dt=_lib.BF16, xq=None, rows=32, cols=64, grouping=0, rounding=0, out=None):
        return L.mxfp4_quantize(x, dt, xq, rows, cols, grouping, rounding, 0, 0, 0, 0, out, None)
    out, outt = fake(32, 64), fake(64, 32)
    assert quant(out=None) == ARG
    assert quant(x=None, out=ref(out)) == ARG
    assert quant(x=0x1002, out=ref(out)) == ALIGN
    assert quant(cols=40, out=ref(out)) == SHAPE
    assert quant(rows=31, out=ref(out)) == SHAPE
    assert quant(grouping=1, out=ref(out)) == SHAPE          # transposed output expected
    assert quant(grouping=2, out=ref(out)) == ARG
    assert quant(rounding=2, out=ref(out)) == ARG
    assert quant(dt=_lib.NVFP4, out=ref(out)) == ARG
    assert quant(out=ref(fake(32, 64, _lib.NVFP4))) == ARG
    assert quant(dt=_lib.MXFP4, xq=ref(out), out=ref(out)) == UNS  # rows of a quantized input
    assert quant(dt=_lib.MXFP4, xq=ref(fake(32, 48)), grouping=1, out=ref(outt)) == SHAPE
    assert quant(rows=0, out=ref(out)) == SHAPE
    big = fake(1 << 21, 1 << 15)
    assert quant(rows=1 << 21, cols=1 << 15, out=ref(big)) == SHAPE and b"too many" in L.tj2_last_error()
    long = fake(16, (1 << 23) + 16)
    assert quant(rows=16, cols=(1 << 23) + 16, out=ref(long)) == SHAPE and b"2^23" in L.tj2_last_error()

    A, B = fake(3, 64), fake(5, 64)
    gemm = lambda a, b, c=0x5000, dt=_lib.F32, ldc=5, acc=0, ws=None, n=0: L.mxfp4_gemm(a, b, c, dt, ldc, acc, ws, n, None)
    assert gemm(None, ref(B)) == ARG
    assert gemm(ref(A), ref(fake(5, 96))) == SHAPE
    assert gemm(ref(A), ref(B), c=None) == ARG
    assert gemm(ref(A), ref(B), dt=7) == ARG
    assert gemm(ref(A), ref(B), ldc=4) == SHAPE
    assert gemm(ref(A), ref(B), dt=_lib.BF16, acc=1) == UNS
    assert gemm(ref(A), ref(B), ws=0x9001, n=1 << 20) == ALIGN
    a2, b2 = fake(64, 65536), fake(64, 65536)
    need = L.mxfp4_gemm_workspace_size(64, 64, 65536)
    assert need > 0 and gemm(ref(a2), ref(b2), ldc=64, ws=0x9000, n=need - 1) == ARG
    # the double block's products refuse the format
    assert L.nvfp4_gemm(ref(A), ref(B), None, None, 0x5000, _lib.F32, 5, None, 0, None, 0, None) != 0

    assert L.mxfp4_dequantize(None, 0x1000, _lib.BF16, None) == ARG
    assert L.mxfp4_dequantize(ref(A), None, _lib.BF16, None) == ARG
    assert L.mxfp4_dequantize(ref(A), 0x1001, _lib.BF16, None) == ALIGN
    assert L.mxfp4_dequantize(ref(A), 0x1000, _lib.NVFP4, None) == ARG

    fwd = lambda M, K, N, wq, xq, y=0x7000: L.mxfp4_linear_fwd(0x1000, M, K, N, None, wq, xq, y, _lib.BF16, None, 0, None)
    assert fwd(3, 64, 48, ref(fake(48, 64)), None) == ARG
    assert fwd(0, 64, 48, ref(fake(48, 64)), ref(A)) == SHAPE
    assert fwd(3, 60, 48, ref(fake(48, 60)), ref(fake(3, 60))) == SHAPE
    assert fwd(3, 64, 40, ref(fake(40, 64)), ref(A)) == SHAPE
    assert fwd(3, 64, 48, ref(fake(48, 64)), ref(A), y=None) == ARG
    bwd = lambda ws, n, rounding=1: L.mxfp4_linear_bwd(0x1000, 3, 48, 64, ref(A), ref(fake(48, 64)), rounding, 1, 0, 0, 0x2000,
                                                       _lib.BF16, 0x3000, ws, n, None)
    need = L.mxfp4_linear_bwd_workspace_size(3, 48, 64)
    assert need > 0 and L.mxfp4_linear_bwd_workspace_size(0, 48, 64) == 0
    assert bwd(None, 0) == ARG and bwd(0x9000, need - 1) == ARG and bwd(0x9004, need) == ALIGN
    assert bwd(0x9000, need, rounding=5) == ARG


def test_storage_size():
    from bit_fully_quantized_amd import _lib
    L = _lib.lib()
    c, s, s128 = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    assert L.tj2_qtensor_bytes(_lib.MXFP4, 3, 131, ctypes.byref(c), ctypes.byref(s), ctypes.byref(s128)) == 0
    assert (c.value, s.value, s128.value) == (3 * 2 * 64, 3 * 2 * 4, 0)
    assert L.tj2_qtensor_bytes(_lib.MXFP4, 3, 0, None, None, None) == _lib.TJ2_ERR_SHAPE
