"""FP8 operands (a scale per 128 of a row, or per 128 x 128), their product and the linear layer on them, against the
definition: quantizers bit for bit, products in 64 bits."""
import numpy as np
import pytest
import torch

from oracle import formats

pytestmark = pytest.mark.gpu

tj2 = pytest.importorskip("bit_fully_quantized_amd")

H24, H8 = 2.0 ** -24, 2.0 ** -8  # half a step of fp32 and of bf16, relative


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(rows, cols, seed=0, std=1.0, dtype=torch.float32):
    x = torch.randn(rows, cols, generator=gen(seed), device="cuda") * std
    return (x * torch.where(torch.rand(cols, generator=gen(seed + 1), device="cuda") < 0.05, 8.0, 1.0)).to(dtype)


def ref_tiles(x, tr, tc):
    """Codes [rows, cols] and fp32 scales [tiles of rows, tiles of cols] of fp32 x by the definition (numpy)."""
    x = np.asarray(x, dtype=np.float32)
    rows, cols = x.shape
    nr, nc = -(-rows // tr), -(-cols // tc)
    p = np.zeros((nr * tr, nc * tc), np.float32)
    p[:rows, :cols] = x
    p = p.reshape(nr, tr, nc, tc)
    amax = np.abs(p).max(axis=(1, 3))
    bad = ~np.isfinite(p).all(axis=(1, 3))
    with np.errstate(all="ignore"):
        S = np.where(amax < np.float32(2.0 ** -100), np.float32(0), amax / np.float32(448)).astype(np.float32)
        inv = np.where(S > 0, np.float32(1) / S, np.float32(0)).astype(np.float32)
        v = np.clip(p * inv[:, None, :, None], np.float32(-448), np.float32(448))
    v = np.where(bad[:, None, :, None], np.float32(0), v)
    S = np.where(bad, np.float32(np.nan), S)
    return formats.e4m3_rne(v).reshape(nr * tr, nc * tc)[:rows, :cols], S


def same(q, codes, S):
    got = q.codes.cpu().numpy()
    np.testing.assert_array_equal(got[:, : q.len], codes)
    assert not got[:, q.len:].any()
    np.testing.assert_array_equal(q.scale128.cpu().numpy().view(np.uint32) & 0x7FC00000 if np.isnan(S).any() else 0,
                                  S.view(np.uint32) & 0x7FC00000 if np.isnan(S).any() else 0)
    np.testing.assert_array_equal(q.scale128.cpu().numpy(), S)  # (NaNs compare equal here)


def values(q):
    """fp64 values code * scale."""
    v = formats.e4m3_decode(q.codes.cpu().numpy()[:, : q.len]).astype(np.float64)
    s = q.scale128.cpu().numpy().astype(np.float64)
    s = np.repeat(s, 128, 1)[:, : q.len]
    return v * (s if q.fmt == tj2.FP8 else np.repeat(s, 128, 0)[: q.rows])


def awkward(rows, cols, dtype, seed=0):
    """Groups of zeros, of tiny, subnormal and huge values, and negative zeros among ordinary ones."""
    x = normal(rows, cols, seed, dtype=torch.float32)
    x[0] = 0.0
    if rows > 3:
        x[1] *= 2.0 ** -104
        x[2] *= 2.0 ** 120
        x[3] *= 2.0 ** -130
    x[:, 0] = -0.0
    return x.to(dtype)


SHAPES = [(1, 16), (3, 48), (5, 128), (16, 144), (37, 256), (128, 128), (129, 272), (300, 1040)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize_rows_and_blocks(rows, cols, dtype):
    x = awkward(rows, cols, dtype)
    h = x.float().cpu().numpy()
    q = tj2.fp8_quantize(x)
    same(q, *ref_tiles(h, 1, 128))
    old = tj2.quantize(x, out_fmt=tj2.FP8)  # the forward's outlier channels have the same format
    assert torch.equal(old.codes, q.codes) and torch.equal(old.scale128, q.scale128)
    b = tj2.fp8_quantize(x, block=True)
    assert b.fmt == tj2.FP8_BLOCK and b.scale128.shape == (-(-rows // 128), -(-cols // 128))
    same(b, *ref_tiles(h, 128, 128))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(16, 16), (48, 112), (128, 64), (144, 128), (272, 208), (1040, 144)])
def test_quantize_columns(rows, cols, dtype):
    x = awkward(rows, cols, dtype)
    q = tj2.fp8_quantize(x, grouping=tj2.GROUP_COL)
    same(q, *ref_tiles(x.float().cpu().numpy().T.copy(), 1, 128))
    r = tj2.fp8_quantize(x)  # its codes grouped anew
    same(tj2.fp8_quantize(r, grouping=tj2.GROUP_COL), *ref_tiles(tj2.fp8_dequantize(r, dtype=torch.float32).cpu().numpy().T.copy(), 1, 128))


def test_infinities_and_nans_stay_in_their_group():
    x = normal(260, 400)
    x[3, 7], x[200, 130], x[5, 399] = float("inf"), float("nan"), float("-inf")
    h = x.cpu().numpy()
    for kw, tiles, m in ((dict(), (1, 128), h), (dict(block=True), (128, 128), h)):
        q = tj2.fp8_quantize(x, **kw)
        codes, S = ref_tiles(m, *tiles)
        np.testing.assert_array_equal(q.codes.cpu().numpy()[:, :400], codes)
        np.testing.assert_array_equal(q.scale128.cpu().numpy(), S)
        v = tj2.fp8_dequantize(q, dtype=torch.float32)
        assert torch.isnan(v[3, :128]).all() and torch.isnan(v).sum() >= 3 * 16 and not torch.isinf(v).any()
    q = tj2.fp8_quantize(x[:256].contiguous(), grouping=tj2.GROUP_COL)
    codes, S = ref_tiles(h[:256].T.copy(), 1, 128)
    np.testing.assert_array_equal(q.codes.cpu().numpy(), codes)
    np.testing.assert_array_equal(q.scale128.cpu().numpy(), S)
    # a product: the row of a NaN group is NaN, the others are what they were
    B = tj2.fp8_quantize(normal(48, 400, 9))
    y = normal(260, 400)
    q, clean = tj2.fp8_quantize(x), tj2.fp8_quantize(y)
    for dt in (torch.float32, torch.bfloat16):
        C, D = tj2.fp8_gemm(q, B, out_dtype=dt), tj2.fp8_gemm(clean, B, out_dtype=dt)
        bad = torch.tensor([3, 5, 200], device="cuda")
        assert torch.isnan(C[bad]).all()
        keep = torch.ones(260, dtype=torch.bool, device="cuda")
        keep[bad] = False
        assert torch.equal(C[keep], D[keep])


@pytest.mark.parametrize("block", [False, True])
def test_values(block):
    q = tj2.fp8_quantize(awkward(137, 208, torch.float32), block=block)
    ref = values(q).astype(np.float32)  # one rounding of an exact product
    assert np.array_equal(tj2.fp8_dequantize(q, dtype=torch.float32).cpu().numpy(), ref)
    assert torch.equal(tj2.fp8_dequantize(q).cpu(), torch.from_numpy(ref).bfloat16())


def check(C, A, B, start=None):
    """A result against the operands' values in 64 bits."""
    a, b = values(A), values(B)
    ref, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    if start is not None:
        ref, mag = ref + start, mag + np.abs(start)
    got = C.double().cpu().numpy()
    K = A.len
    if C.dtype == torch.float32:
        # exact products; an fp32 sum of K of them, a scale's product and a multiplication per 128, splits and start
        tol = (K + 3 * (K // 128 + 1) + 32) * H24 * mag
    else:
        # the 8-bit instruction keeps 14 bits of what up to 8 neighbours add to their largest product: 8 * 2^-13 of the
        # magnitudes; then half a step of bf16
        tol = H8 * np.abs(ref) + 2.0 ** -10 * mag
    err = np.abs(got - ref)
    assert (err <= tol + 1e-42).all(), float((err / (tol + 1e-42)).max())


GEMMS = [(1, 16, 16), (1, 48, 1024), (5, 33, 144), (16, 130, 2048), (17, 64, 256), (31, 256, 640), (64, 200, 1024),
         (65, 65, 128), (100, 70, 4096), (129, 257, 400), (256, 512, 384), (300, 515, 2000), (515, 300, 272)]


@pytest.mark.parametrize("block", [False, True])
@pytest.mark.parametrize("I,J,K", GEMMS)
def test_products(I, J, K, block):
    A = tj2.fp8_quantize(normal(I, K, 1))
    B = tj2.fp8_quantize(normal(J, K, 3, 0.02), block=block)
    check(tj2.fp8_gemm(A, B), A, B)
    check(tj2.fp8_gemm(A, B, out_dtype=torch.bfloat16), A, B)
    # into part of a wider matrix, whose other columns stay; and added to it
    wide = torch.full((I, J + 13), 7.0, device="cuda")
    tj2.fp8_gemm(A, B, out=wide)
    check(wide[:, :J], A, B)
    assert (wide[:, J:] == 7.0).all()
    tj2.fp8_gemm(A, B, out=wide, accumulate=True)
    check(wide[:, :J], A, B, values(A) @ values(B).T)
    assert (wide[:, J:] == 7.0).all()


@pytest.mark.parametrize("block", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_split_reduction_repeats_bit_for_bit(block, dtype):
    A = tj2.fp8_quantize(normal(130, 16384, 1))
    B = tj2.fp8_quantize(normal(100, 16384, 2), block=block)
    assert tj2.fp8_gemm_workspace(130, 100, 16384) is not None
    C = tj2.fp8_gemm(A, B, out_dtype=dtype)
    check(C, A, B)
    for _ in range(3):
        assert torch.equal(tj2.fp8_gemm(A, B, out_dtype=dtype), C)


def test_padding_beyond_a_row_is_not_read():
    """Stored weights whose padding holds anything."""
    A, B = tj2.fp8_quantize(normal(40, 144, 1)), tj2.fp8_quantize(normal(33, 144, 2), block=True)
    C = [tj2.fp8_gemm(A, B, out_dtype=dt) for dt in (torch.float32, torch.bfloat16)]
    one = tj2.fp8_quantize(normal(1, 144, 3))
    D = tj2.fp8_gemm(one, B)
    codes = B.codes.clone()
    codes[:, 144:] = 0x7F
    W = tj2.QTensor.wrap(tj2.FP8_BLOCK, 33, 144, codes, None, B.scale128)
    assert torch.equal(tj2.fp8_gemm(A, W), C[0]) and torch.equal(tj2.fp8_gemm(A, W, out_dtype=torch.bfloat16), C[1])
    assert torch.equal(tj2.fp8_gemm(one, W), D)


LINEARS = [(1, 1024, 256), (2, 48, 16), (16, 4096, 64), (17, 144, 320), (24, 1024, 528), (48, 1024, 272), (64, 1040, 128),
           (77, 656, 400), (128, 128, 128), (200, 272, 1040), (515, 528, 304), (1100, 2064, 656)]


@pytest.mark.parametrize("M,K,N", LINEARS)
def test_linear(M, K, N):
    X, W, dY = normal(M, K, 1, dtype=torch.bfloat16), normal(N, K, 2, 0.02), normal(M, N, 3, 1e-3, torch.bfloat16)
    X[M // 2] = 0.0 if M > 4 else X[M // 2]
    Y, saved = tj2.fp8_linear_fwd(X, W, N)
    Xq, Wq = saved["Xq"], saved["Wq"]
    ref_x, ref_w = tj2.fp8_quantize(X), tj2.fp8_quantize(W, block=True)
    for a, b in ((Xq, ref_x), (Wq, ref_w)):
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scale128, b.scale128)
    check(Y, Xq, Wq)
    check(tj2.fp8_linear_fwd(X, None, N, Wq=Wq, y_dtype=torch.float32)[0], Xq, Wq)
    assert torch.equal(tj2.fp8_linear_fwd(Xq, None, N, Wq=Wq)[0], Y)  # an operand that is quantized already
    dX, dW = tj2.fp8_linear_bwd(dY, saved, K)
    # dX: Q(dY) W-hat; the weights' codes turned, a block's scale the same
    h = dY.float().cpu().numpy()
    codes, S = ref_tiles(h, 1, 128)
    dyv = formats.e4m3_decode(codes).astype(np.float64) * np.repeat(S.astype(np.float64), 128, 1)[:, :N]
    w = values(Wq)
    ref, mag = dyv @ w, np.abs(dyv) @ np.abs(w)
    assert (np.abs(dX.double().cpu().numpy() - ref) <= H8 * np.abs(ref) + 2.0 ** -10 * mag + 1e-42).all()
    dX32, _ = tj2.fp8_linear_bwd(dY, saved, K, dx_dtype=torch.float32)
    assert (np.abs(dX32.double().cpu().numpy() - ref) <= (N + 3 * (N // 128 + 1) + 32) * H24 * mag + 1e-42).all()
    # dW: both operands grouped along the tokens
    codes, S = ref_tiles(h.T.copy(), 1, 128)
    a = formats.e4m3_decode(codes).astype(np.float64) * np.repeat(S.astype(np.float64), 128, 1)[:, :M]
    xh = tj2.fp8_dequantize(Xq, dtype=torch.float32).cpu().numpy()
    codes, S = ref_tiles(xh.T.copy(), 1, 128)
    b = formats.e4m3_decode(codes).astype(np.float64) * np.repeat(S.astype(np.float64), 128, 1)[:, :M]
    ref, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    assert (np.abs(dW.double().cpu().numpy() - ref) <= (M + 3 * (M // 128 + 1) + 32) * H24 * mag + 1e-42).all()


def test_gradients_against_differences():
    """With weights and inputs on the grid the layer is linear in both: differences of sum(Y * dY) in W and X give its
    gradients, up to dY's and X's rounding to FP8 (half a step, 2^-4 of each element)."""
    M, K, N = 40, 64, 48
    X, W = normal(M, K, 1, dtype=torch.bfloat16), normal(N, K, 2, 0.02)
    dY = normal(M, N, 3, 1e-3, torch.bfloat16)
    _, saved = tj2.fp8_linear_fwd(X, W, N)
    dX, dW = tj2.fp8_linear_bwd(dY, saved, K, dx_dtype=torch.float32)
    x, w, d = values(saved["Xq"]), values(saved["Wq"]), dY.double().cpu().numpy()

    def f(x, w):
        return float(((x @ w.T) * d).sum())
    rng = np.random.default_rng(0)
    for _ in range(8):
        ex, ew = rng.standard_normal(x.shape), rng.standard_normal(w.shape)
        dx = f(x + ex, w) - f(x, w)  # linear in each: the difference is exact
        dw = f(x, w + ew) - f(x, w)
        tx = 2.0 ** -4 * (np.abs(ex) @ np.abs(w).T * np.abs(d)).sum() * 1.01
        tw = (2 * 2.0 ** -4 + 2.0 ** -8) * (np.abs(x) @ np.abs(ew).T * np.abs(d)).sum() * 1.01
        assert abs(float((dX.double().cpu().numpy() * ex).sum()) - dx) <= tx
        assert abs(float((dW.double().cpu().numpy() * ew).sum()) - dw) <= tw


def test_given_buffers_streams_and_graphs():
    M, K, N = 150, 272, 400
    W = normal(N, K, 2, 0.02)
    xs = [normal(M, K, s, dtype=torch.bfloat16) for s in (1, 4)]
    ds = [normal(M, N, s, 1e-3, torch.bfloat16) for s in (5, 6)]
    want = []
    for x, d in zip(xs, ds):
        Y, saved = tj2.fp8_linear_fwd(x, W, N)
        want.append((Y, *tj2.fp8_linear_bwd(d, saved, K)))
    # two streams at once, each with its own buffers
    streams, got = [torch.cuda.Stream() for _ in xs], []
    torch.cuda.synchronize()
    for st, x, d in zip(streams, xs, ds):
        with torch.cuda.stream(st):
            Y, saved = tj2.fp8_linear_fwd(x, W, N)
            got.append((Y, *tj2.fp8_linear_bwd(d, saved, K)))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    # captured, two graphs that share a workspace, replayed in turn with eager work between
    x, d = xs[0].clone(), ds[0].clone()
    Xq, Wq = tj2.QTensor.packed(tj2.FP8, M, K), tj2.QTensor(tj2.FP8_BLOCK, N, K)
    Y, dX, dW = torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), torch.empty(M, K, dtype=torch.bfloat16, device="cuda"), torch.empty(N, K, device="cuda")
    ws = tj2.fp8_linear_bwd_workspace(M, N, K)
    side, graphs = torch.cuda.Stream(), []
    with torch.cuda.stream(side):
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                _, saved = tj2.fp8_linear_fwd(x, W, N, Xq=Xq, Wq=Wq, Y=Y)
                tj2.fp8_linear_bwd(d, saved, K, dX=dX, dW=dW, workspace=ws)
            graphs.append(g)
    torch.cuda.synchronize()
    for i in range(6):
        x.copy_(xs[i % 2])
        d.copy_(ds[i % 2])
        ws.fill_(255)
        graphs[i // 2 % 2].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(want[i % 2], (Y, dX, dW))), i
        tj2.fp8_linear_fwd(xs[1], W, N)
