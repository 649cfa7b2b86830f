"""Weights' gradients of the norm, the FP8 linear and the feed-forward block over tokens whose offsets pass 32 bits,
against 64-bit sums.  No token repeats, so those past the border count as the others do: were a 256th of them wrong, the
gradients would be off by a sixteenth of their norm."""
import pytest
import torch

from test_gpu_ffn import Exact
from test_gpu_fp8_tiles import values
from test_gpu_norm import stat

pytestmark = pytest.mark.gpu

tj2 = pytest.importorskip("bit_fully_quantized_amd")
BF = torch.bfloat16
H24, H8 = 2.0 ** -24, 2.0 ** -8


def normal(rows, cols, seed, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    out = torch.empty(rows, cols, device="cuda", dtype=BF)
    for r in range(0, rows, 1 << 17):
        n = min(1 << 17, rows - r)
        out[r:r + n] = (torch.randn(n, cols, generator=g, device="cuda") * std).to(BF)
    return out


def off(got, ref):
    return float((got.double() - ref).norm() / ref.norm())


def test_norm():
    rows, cols = (1 << 20) + 77, 2064  # 2.16e9 elements
    x, dy, w = normal(rows, cols, 1), normal(rows, cols, 2), torch.linspace(0.5, 1.5, cols, device="cuda")
    rstd = tj2.rms_norm_fwd(x, w)[2]
    dw = tj2.rms_norm_bwd(dy, x, w, rstd, need_ds=False)[1]
    ref = torch.zeros(cols, device="cuda", dtype=torch.float64)
    for r in range(0, rows, 1 << 16):
        s = x[r:r + (1 << 16)].double()
        ref += (dy[r:r + (1 << 16)].double() * s / torch.sqrt((s * s).mean(1, keepdim=True) + 1e-6)).sum(0)
    # a thread's sum over some 1024 rows and two sums of 32 of those: 33 half steps, were each of the sum so far; rstd's
    # error; a few operations an element
    assert off(dw, ref) <= 40 * H24 + stat(cols)


def test_fp8_linear():
    M, K, N = (1 << 20) + 256, 128, 2064  # dY has 2.16e9 elements
    X, W, dY = normal(M, K, 1), normal(N, K, 2, 0.1).float(), normal(M, N, 3, 1e-3)
    _, saved = tj2.fp8_linear_fwd(X, W, N)
    dX, dW = tj2.fp8_linear_bwd(dY, saved, K)
    xt = tj2.fp8_quantize(tj2.fp8_dequantize(saved["Xq"], dtype=torch.float32), grouping=tj2.GROUP_COL)
    w = values(saved["Wq"])
    ref = torch.zeros(N, K, device="cuda", dtype=torch.float64)
    step = 1 << 15  # tokens: whole groups
    for r in range(0, M, step):
        part = dY[r:r + step].contiguous()
        n = part.shape[0]
        a = values(tj2.fp8_quantize(part, grouping=tj2.GROUP_COL))
        b = values(tj2.QTensor.wrap(tj2.FP8, K, n, xt.codes[:, r:r + n].contiguous(), None,
                                    xt.scale128[:, r // 128:(r + n + 127) // 128].contiguous()))
        ref += a @ b.T
        d = values(tj2.fp8_quantize(part))
        want = d @ w
        assert ((dX[r:r + n].double() - want).abs() <= H8 * want.abs() + 2.0 ** -10 * (d.abs() @ w.abs())).all(), r
    # 8194 chunks in 16 splits, 7 roundings a chunk and those of the splits: 60 half steps, were each of the sum so far
    assert off(dW, ref) <= 256 * H24


def test_feed_forward_block():
    T, D, F = (1 << 19) + 130, 16, 4112  # G has 2.16e9 elements
    X, dY = normal(T, D, 1), normal(T, D, 5, 1e-2)
    Wg, Wu, Wd = normal(F, D, 2, 0.2), normal(F, D, 3, 0.2), normal(D, F, 4, 0.02)
    Y, saved = tj2.gated_ffn_fwd(X, Wg, Wu, Wd, save=True)
    grads = tj2.gated_ffn_bwd(dY, X, Wg, Wu, Wd, saved, dw_dtype=torch.float32)
    sums = [0.0, 0.0, 0.0]
    for r in range(0, T, 1 << 14):
        e = Exact(X[r:r + (1 << 14)], Wg, Wu, Wd, "silu", dY[r:r + (1 << 14)])
        assert off(Y[r:r + (1 << 14)], e.Y[0]) <= 2 * H8 and off(grads[0][r:r + (1 << 14)], e.dX[0]) <= 2 * H8, r
        sums = [a + b[0] for a, b in zip(sums, (e.dWg, e.dWu, e.dWd))]
    # dG, dU and H rounded to bf16: half a step of each term, as of the norm
    for g, want in zip(grads[1:], sums):
        assert off(g, want) <= 2 * H8
