"""Results between an input's rows and right beside inputs and other results: what they are elsewhere."""
import pytest
import torch

pytestmark = pytest.mark.gpu

tj2 = pytest.importorskip("bit_fully_quantized_amd")
BF = torch.bfloat16


def normal(shape, seed, dtype=BF, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def test_norm_in_the_gaps_of_its_input():
    rows, cols = 5, 64
    buf = torch.zeros(rows, 16 * cols, device="cuda", dtype=BF)
    x, w = buf[:, :cols], 1.0 + normal(cols, 2, torch.float32, 0.1)
    x.copy_(normal((rows, cols), 1))
    res, dy = normal((rows, cols), 3), normal((rows, cols), 4)
    want = tj2.rms_norm_fwd(x.contiguous(), w, residual=res)
    back = tj2.rms_norm_bwd(dy, want[1], w, want[2], dsum=x.contiguous())
    gap = [buf.view(-1)[i * 16 * cols + cols:][: rows * cols].view(rows, cols) for i in range(2)]  # after the first two rows
    after = buf.view(-1)[16 * cols + 6 * cols:][: rows * cols].view(rows, cols)
    y, s, rstd = tj2.rms_norm_fwd(x, w, residual=res, y=gap[0], sum=gap[1])
    assert y is gap[0] and torch.equal(y, want[0]) and torch.equal(s, want[1]) and torch.equal(rstd, want[2])
    ds, _ = tj2.rms_norm_bwd(dy, s, w, rstd, dsum=x, ds=after)
    assert ds is after and torch.equal(ds, back[0])
    assert torch.equal(s, want[1])


def test_results_side_by_side():
    M, K, N = 16, 128, 48
    X, W, dY = normal((M, K), 1), normal((N, K), 2, torch.float32, 0.1), normal((M, N), 3)
    Y, saved = tj2.fp8_linear_fwd(X, W, N)
    dX, dW = tj2.fp8_linear_bwd(dY, saved, K, dx_dtype=torch.float32)
    flat = torch.empty(M * N + M * K * 2 + N * K * 4, device="cuda")
    parts = flat.split((M * N, M * K * 2, N * K * 4))
    y, dx, dw = parts[0].view(M, N), parts[1][: M * K].view(M, K), parts[2][: N * K].view(N, K)
    assert torch.equal(tj2.fp8_linear_fwd(X, W, N, Y=y)[0].to(BF), Y)
    assert all(torch.equal(a, b) for a, b in zip(tj2.fp8_linear_bwd(dY, saved, K, dX=dx, dW=dw), (dX, dW)))
    T, D, F = 20, 64, 96
    X, Wg, Wu, Wd, dY = normal((T, D), 1), normal((F, D), 2, BF, 0.1), normal((F, D), 3, BF, 0.1), normal((D, F), 4, BF, 0.1), normal((T, D), 5)
    Y, kept = tj2.gated_ffn_fwd(X, Wg, Wu, Wd, save=True)
    want = tj2.gated_ffn_bwd(dY, X, Wg, Wu, Wd, kept)
    into = torch.empty(T * D + 3 * F * D, dtype=BF, device="cuda").split((T * D, F * D, F * D, F * D))
    got = tj2.gated_ffn_bwd(dY, X, Wg, Wu, Wd, kept, dX=into[0].view(T, D), dWg=into[1].view(F, D), dWu=into[2].view(F, D), dWd=into[3].view(D, F))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # X has been read when Y is written
    x = X.clone()
    assert torch.equal(tj2.gated_ffn_fwd(x, Wg, Wu, Wd, Y=x)[0], Y) and torch.equal(x, Y)
