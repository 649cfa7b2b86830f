"""FP8 products and linears of sizes that take the larger tiles, with remainders on every side: all elements against
64-bit products of the operands' values."""
import pytest
import torch

from test_gpu_fp8 import H8, H24, normal

pytestmark = pytest.mark.gpu

tj2 = pytest.importorskip("bit_fully_quantized_amd")
BF = torch.bfloat16


def values(q):
    """Codes times scales in 64 bits (on the GPU), element by element from the format's definition."""
    c = q.codes[:, : q.len].to(torch.int32)
    e, m = c >> 3 & 15, (c & 7).double()
    v = torch.where(e > 0, (1 + m / 8) * torch.exp2((e - 7).double()), m / 8 * 2.0 ** -6)
    v = torch.where(c & 128 > 0, -v, v)
    s = q.scale128.double().repeat_interleave(128, 1)[:, : q.len]
    return v * (s if q.fmt == tj2.FP8 else s.repeat_interleave(128, 0)[: q.rows])


def close(got, a, b, start=None, what=""):
    """got against a b^T in 64 bits: fp32 results as sums of exact products (a rounding a product, three a chunk and
    those of up to 32 partial sums), bf16 ones as the 8-bit instruction's (14 bits of what 8 neighbours add to their
    largest product: 2^-10 of the magnitudes), then half a step of bf16."""
    K = a.shape[1]
    for r in range(0, a.shape[0], 4096):
        x = a[r:r + 4096]
        ref, mag = x @ b.T, x.abs() @ b.abs().T
        if start is not None:
            ref, mag = ref + start[r:r + 4096], mag + start[r:r + 4096].abs()
        if got.dtype == torch.float32:
            tol = (K + 3 * (K // 128 + 1) + 32) * H24 * mag
        else:
            tol = H8 * ref.abs() + 2.0 ** -10 * mag
        err = (got[r:r + 4096].double() - ref).abs()
        assert (err <= tol + 1e-42).all(), (what, r, float((err / (tol + 1e-42)).max()))
        # the bounds add magnitudes; of independent errors the norm is the root of the sum of squares: some 7 roundings a
        # chunk, each of at most half a step of the sum so far, 22 half steps for 64 chunks (64 are asked)
        assert float(err.norm() / ref.norm()) <= (H8 if got.dtype == BF else 64 * H24), (what, r)


# bf16 results take tiles of 128, 256, 256 and 128 (in 2 splits), fp32 ones of 128
GEMMS = [(2050, 2064, 272), (4100, 2064, 1040), (8200, 4112, 400), (1030, 2063, 8208)]


@pytest.mark.parametrize("block", [False, True])
@pytest.mark.parametrize("I,J,K", GEMMS)
def test_products(I, J, K, block):
    A, B = tj2.fp8_quantize(normal(I, K, 1)), tj2.fp8_quantize(normal(J, K, 3, 0.02), block=block)
    a, b = values(A), values(B)
    for dt in (torch.float32, BF):
        wide = torch.full((I, J + 13), 7.0, device="cuda", dtype=dt)
        tj2.fp8_gemm(A, B, out=wide)
        close(wide[:, :J], a, b, what=dt)
        assert (wide[:, J:] == 7.0).all()
        C = tj2.fp8_gemm(A, B, out_dtype=dt)
        close(C, a, b, what=dt)
        assert torch.equal(C, wide[:, :J])
    before = wide[:, :J].float()
    C = before.clone()
    tj2.fp8_gemm(A, B, out=C, accumulate=True)
    close(C, a, b, before.double(), "accumulate")


# tiles of the forward, of dX in bf16 (in fp32 of 128 at most) and of dW: 128, 128 and 128 in one launch; 256, 128 and 128
# in 4 splits, in one launch; 128, 128 and 64 in 4 splits, apart; 256, 256 and 128 in 2 splits, apart
LINEARS = [(4100, 1040, 4112), (8200, 1040, 4112), (8100, 1008, 1008), (8100, 2032, 2032)]


@pytest.mark.parametrize("M,K,N", LINEARS)
def test_linear(M, K, N):
    X, W, dY = normal(M, K, 1, dtype=BF), normal(N, K, 2, 0.02), normal(M, N, 3, 1e-3, BF)
    Y, saved = tj2.fp8_linear_fwd(X, W, N)
    x, w = values(saved["Xq"]), values(saved["Wq"])
    close(Y, x, w, what="Y")
    close(tj2.fp8_linear_fwd(X, None, N, Wq=saved["Wq"], y_dtype=torch.float32)[0], x, w, what="Y fp32")
    # the backward's operands by the quantizers, which have tests of their own; columns grouped along the tokens
    dy, wt = values(tj2.fp8_quantize(dY)), w.T.contiguous()

    def turned(t):
        pad = torch.zeros(-(-M // 16) * 16, t.shape[1], dtype=t.dtype, device="cuda")
        pad[:M] = t
        return values(tj2.fp8_quantize(pad, grouping=tj2.GROUP_COL))[:, :M]
    dyt, xt = turned(dY), turned(tj2.fp8_dequantize(saved["Xq"], dtype=torch.float32))
    for dt in (BF, torch.float32):
        dX, dW = tj2.fp8_linear_bwd(dY, saved, K, dx_dtype=dt)
        close(dX, dy, wt, what=("dX", dt))
        close(dW, dyt, xt, what=("dW", dt))
        again = tj2.fp8_linear_bwd(dY, saved, K, dx_dtype=dt)
        assert torch.equal(again[0], dX) and torch.equal(again[1], dW)


def test_gradients_follow_the_differences():
    """With operands on the grid, sum(Y * dY) is linear in X and in W: its difference along a direction is the
    gradient's product with it, up to dY's rounding (2^-4 of an element at most, and X's once more in dW: a vector whose
    norm is at most 2^-4, or 2 * 2^-4 + 2^-8, of what the product would be of the magnitudes).  Along the gradient
    itself the difference is its squared norm, so a gradient of another size or sign, or none, fails."""
    M, K, N = 200, 192, 160
    X, W, dY = normal(M, K, 1, dtype=BF), normal(N, K, 2, 0.02), normal(M, N, 3, 1e-3, BF)
    _, saved = tj2.fp8_linear_fwd(X, W, N)
    got = [t.double() for t in tj2.fp8_linear_bwd(dY, saved, K, dx_dtype=torch.float32)]
    x, w, d = values(saved["Xq"]), values(saved["Wq"]), dY.double()

    def f(x, w):
        return ((x @ w.T) * d).sum()
    # an element's rounding is at most half a step; those of a sum of n are independent of one another, so the error of a
    # sum is of the order of the root of the sum of their squares, of which 8 times is asked
    e = 2.0 ** -4
    spread = (e * torch.sqrt(d ** 2 @ w ** 2), (2 * e + 2.0 ** -8) * torch.sqrt((d ** 2).T @ x ** 2))
    for i, g in enumerate(got):
        assert ((g - (d @ w if i == 0 else d.T @ x)).abs() <= 8 * spread[i]).all()
        ways = [g / g.norm()] + [torch.randn(g.shape, generator=torch.Generator("cuda").manual_seed(s), device="cuda", dtype=torch.float64) for s in range(4)]
        for k, way in enumerate(ways):
            diff = f(x + way, w) - f(x, w) if i == 0 else f(x, w + way) - f(x, w)  # linear: the difference is exact
            tol = 8 * float((spread[i] * way).norm()) + 1e-9 * float(f(x.abs(), w.abs()).abs())
            assert abs(float((g * way).sum() - diff)) <= tol, (i, k)
            if k == 0:
                assert tol < 0.5 * float(diff)
