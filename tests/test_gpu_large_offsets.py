"""Norm, FP8 linear and feed-forward block where offsets pass 32 bits: the last rows are what they are alone."""
import pytest
import torch

pytestmark = pytest.mark.gpu

tj2 = pytest.importorskip("bit_fully_quantized_amd")
BF = torch.bfloat16


def tiled(rows, cols, seed, std=1.0):
    """rows x cols whose every 1024 rows repeat but for a few at the end."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = (torch.randn(1024, cols, generator=g, device="cuda") * std).to(BF).repeat(-(-rows // 1024), 1)[:rows]
    x[-7:] = (torch.randn(7, cols, generator=g, device="cuda") * std).to(BF)
    return x


def test_norm():
    rows, cols = (1 << 20) + 77, 2064  # 2.16e9 elements
    x, r = tiled(rows, cols, 1), tiled(rows, cols, 2)
    w = torch.linspace(0.5, 1.5, cols, device="cuda")
    y, s, rstd = tj2.rms_norm_fwd(x, w, residual=r)
    ds, _ = tj2.rms_norm_bwd(x, s, w, rstd, dsum=r)
    ay, a_s, ar = tj2.rms_norm_fwd(x[-300:].contiguous(), w, residual=r[-300:].contiguous())
    assert torch.equal(y[-300:], ay) and torch.equal(s[-300:], a_s) and torch.equal(rstd[-300:], ar)
    assert torch.equal(ds[-300:], tj2.rms_norm_bwd(x[-300:].contiguous(), a_s, w, ar, dsum=r[-300:].contiguous(), need_dw=False)[0])
    del y, ds
    q = tj2.rms_norm_fwd(x, w, residual=r, fp8=True)[0]
    a = tj2.rms_norm_fwd(x[-300:].contiguous(), w, residual=r[-300:].contiguous(), fp8=True)[0]
    assert torch.equal(tj2.fp8_dequantize(q)[-300:], tj2.fp8_dequantize(a))


def test_fp8_linear():
    M, K, N = (1 << 20) + 256, 128, 2064  # Y has 2.16e9 elements
    X, W = tiled(M, K, 1), tiled(N, K, 2, 0.1).float()
    Y, saved = tj2.fp8_linear_fwd(X, W, N)
    alone = tj2.fp8_linear_fwd(X[-256:].contiguous(), W, N)[0]
    assert float((Y[-256:].double() - alone.double()).norm() / alone.double().norm()) <= 2.0 ** -8
    q = tj2.fp8_quantize(X[-7:].contiguous())
    x, w = (tj2.fp8_dequantize(t, dtype=torch.float32).double() for t in (q, saved["Wq"]))
    ref, top = x @ w.T, x.abs() @ w.abs().T
    # bf16's half step, and the instruction's sums, which keep 14 bits of their largest product
    assert ((Y[-7:].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -13 * top).all()
    dX, dW = tj2.fp8_linear_bwd(Y, saved, K)
    small = tj2.fp8_linear_fwd(X[-256:].contiguous(), W, N)[1]
    dXa = tj2.fp8_linear_bwd(Y[-256:].contiguous(), small, K)[0]
    assert float((dX[-256:].double() - dXa.double()).norm() / dXa.double().norm()) <= 2.0 ** -8
    assert torch.isfinite(dW).all()


def test_feed_forward_block():
    T, D, F = (1 << 19) + 130, 16, 4112  # G has 2.16e9 elements
    X = tiled(T, D, 1)
    Wg, Wu, Wd = tiled(F, D, 2, 0.2), tiled(F, D, 3, 0.2), tiled(D, F, 4, 0.02)
    Y, saved = tj2.gated_ffn_fwd(X, Wg, Wu, Wd, save=True)
    Xa = X[-130:].contiguous()
    Ya, saved_a = tj2.gated_ffn_fwd(Xa, Wg, Wu, Wd, save=True)
    assert float((Y[-130:].double() - Ya.double()).norm() / Ya.double().norm()) <= 2.0 ** -8
    dX = tj2.gated_ffn_bwd(X, X, Wg, Wu, Wd, saved, need=(True, False, False, False))[0]
    dXa = tj2.gated_ffn_bwd(Xa, Xa, Wg, Wu, Wd, saved_a, need=(True, False, False, False))[0]
    assert float((dX[-130:].double() - dXa.double()).norm() / dXa.double().norm()) <= 2.0 ** -8
