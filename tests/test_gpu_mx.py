"""MXFP4 on the GPU: codes and scales bit for bit against the oracle, products against fp64, the linear layer's
two passes, and what a caller may do around them (streams, graphs, wrapped weights, masked rows)."""
import numpy as np
import pytest
import torch

from oracle import mx

import _helpers as H

pytestmark = pytest.mark.gpu

tj2 = pytest.importorskip("bit_fully_quantized_amd")


def data(rows, cols, seed, spread=3, dtype=np.float32):
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-spread, spread + 1, (rows, 1)))).astype(np.float32)
    x[rng.random((rows, cols)) < 0.02] = 0.0
    return x


def to_gpu(x, dtype):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda().to(dtype)
    return t, t.float().cpu().numpy()


def same(got, ref, what=""):
    codes, scale, _ = got.host()
    np.testing.assert_array_equal(scale, ref.scale, err_msg=f"{what} scales")
    np.testing.assert_array_equal(codes, ref.codes, err_msg=f"{what} codes")
    full, sfull = got.codes.cpu().numpy(), got.scale16.cpu().numpy()
    assert not full[:, (ref.L + 1) // 2:].any() and not sfull[:, ref.scale.shape[1]:].any(), f"{what} padding"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 48), (37, 128), (130, 144), (257, 1040)])
@pytest.mark.parametrize("grouping", ["row", "col"])
@pytest.mark.parametrize("rounding,rht", [("rtn", False), ("rtn", True), ("sr", False), ("sr", True)])
def test_quantize_matches_the_oracle(dtype, rows, cols, grouping, rounding, rht):
    t, x = to_gpu(data(rows, cols, rows + cols), dtype)
    mask = 0xA53C if rht else 0
    q = tj2.mx_quantize(t, grouping=tj2.GROUP_COL if grouping == "col" else tj2.GROUP_ROW,
                        rounding=tj2.SR if rounding == "sr" else tj2.RTN, rht=rht, signs=mask, seed=77, offset=2 ** 33 + 5)
    ref = mx.quantize(x, grouping=grouping, rounding=rounding, rht_mask=mask if rht else None, seed=77, offset=2 ** 33 + 5)
    same(q, ref)
    for dt in (torch.bfloat16, torch.float32):
        np.testing.assert_array_equal(tj2.mx_dequantize(q, dtype=dt).double().cpu().numpy(), mx.dequantize(ref))


@pytest.mark.parametrize("rounding", ["rtn", "sr"])
def test_quantize_regroups_quantized_input(rounding):
    t, x = to_gpu(data(99, 176, 5), torch.float32)
    q, ref = tj2.mx_quantize(t), mx.quantize(x)
    got = tj2.mx_quantize(q, grouping=tj2.GROUP_COL, rounding=tj2.SR if rounding == "sr" else tj2.RTN, rht=True, signs=9,
                          seed=1, offset=2)
    same(got, mx.quantize(mx.dequantize(ref), grouping="col", rounding=rounding, rht_mask=9, seed=1, offset=2))


@pytest.mark.parametrize("rounding", ["rtn", "sr"])
@pytest.mark.parametrize("grouping", ["row", "col"])
def test_quantize_extremes(grouping, rounding):
    x = np.zeros((64, 64), dtype=np.float32)
    x[:, 0] = np.float32(2.0 ** -149)
    x[0, :32] = 3.4e38
    x[1, :] = np.float32(2.0 ** -126) * np.arange(64, dtype=np.float32) / 8
    x[2, 7] = np.nan
    x[3, 60] = -np.inf
    x[4, :] = np.float32(2.0 ** -128)
    x[5, :] = np.arange(64) / 8.0           # every tie of the grid
    x[6, :] = -np.arange(64) / 8.0
    x[40, 33] = -0.0
    t = torch.from_numpy(x).cuda()
    q = tj2.mx_quantize(t, grouping=tj2.GROUP_COL if grouping == "col" else tj2.GROUP_ROW,
                        rounding=tj2.SR if rounding == "sr" else tj2.RTN, seed=5)
    ref = mx.quantize(x, grouping=grouping, rounding=rounding, seed=5)
    same(q, ref)
    # 3.4e38 rounds up to 4 * 2^126 = 2^128 (SR) or down: 2^128 is beyond bf16 and fp32, whose nearest value of it is inf
    with np.errstate(over="ignore"):
        want = mx.dequantize(ref).astype(np.float32)
    np.testing.assert_array_equal(tj2.mx_dequantize(q).float().cpu().numpy(), want)


def test_values_of_odd_lengths():
    t, x = to_gpu(data(45, 80, 6), torch.bfloat16)  # 45 along the rows of the transposed operand
    q = tj2.mx_quantize(t, grouping=tj2.GROUP_COL)
    ref = mx.dequantize(mx.quantize(x, grouping="col"))
    for dt in (torch.bfloat16, torch.float32):
        np.testing.assert_array_equal(tj2.mx_dequantize(q, dtype=dt).double().cpu().numpy(), ref)


def operands(I, J, K, seed):
    a, x = to_gpu(data(I, K, seed), torch.bfloat16)
    b, w = to_gpu(data(J, K, seed + 1) * np.float32(0.02), torch.float32)
    return tj2.mx_quantize(a), tj2.mx_quantize(b), mx.dequantize(mx.quantize(x)), mx.dequantize(mx.quantize(w))


def close(got, A, B, bf16, base=None):
    """|error| <= the fp32 sums' (K half steps of 2^-24 on the sum of magnitudes) + half a step of a bf16 result."""
    ref = A @ B.T + (0 if base is None else base)
    mags = np.abs(A) @ np.abs(B).T + (0 if base is None else np.abs(base))
    tol = (A.shape[1] + 16) * 2.0 ** -24 * mags + (np.abs(ref) * 2.0 ** -8 if bf16 else 0)
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= tol).all(), (float((err - tol).max()), np.argwhere(err > tol)[:4])


@pytest.mark.parametrize("I,J,K", [(1, 16, 16), (1, 1, 32), (5, 7, 48), (16, 48, 128), (17, 300, 400), (64, 1000, 1024),
                                   (65, 129, 1040), (130, 515, 272), (300, 260, 2064), (513, 512, 512)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gemm(I, J, K, dtype):
    qa, qb, A, B = operands(I, J, K, I + J + K)
    close(tj2.mx_gemm(qa, qb, out_dtype=dtype), A, B, dtype == torch.bfloat16)


@pytest.mark.parametrize("I,J,K", [(40, 96, 16384), (260, 130, 8208), (1, 64, 65536)])
def test_gemm_split_reduction(I, J, K):
    assert tj2.lib().mxfp4_gemm_workspace_size(256, 256, 16384) > 0
    qa, qb, A, B = operands(I, J, K, 3)
    first = tj2.mx_gemm(qa, qb)
    close(first, A, B, False)
    assert torch.equal(first, tj2.mx_gemm(qa, qb))  # the order of the sums is fixed


def test_gemm_strided_accumulate_and_neighbours():
    qa, qb, A, B = operands(37, 83, 176, 8)
    for cols in (83, 84, 96):
        buf = torch.randn(37, cols, device="cuda")
        base = buf.clone()
        tj2.mx_gemm(qa, qb, out=buf, accumulate=True)
        close(buf[:, :83], A, B, False, base[:, :83].double().cpu().numpy())
        assert torch.equal(buf[:, 83:], base[:, 83:])
    rows = torch.full((39, 96), 7.0, device="cuda", dtype=torch.bfloat16)
    tj2.mx_gemm(qa, qb, out=rows[1:38, :])
    close(rows[1:38, :83], A, B, True)
    assert (rows[0] == 7).all() and (rows[38] == 7).all() and (rows[:, 83:] == 7).all()


def test_gemm_zero_rows_and_nan_rows_stay_apart():
    t, x = to_gpu(data(20, 96, 2), torch.bfloat16)
    t[3] = 0.0
    t[5, 40] = float("inf")
    w, wv = to_gpu(data(24, 96, 3), torch.float32)
    C = tj2.mx_gemm(tj2.mx_quantize(t), tj2.mx_quantize(w)).cpu()
    assert (C[3] == 0).all() and torch.isnan(C[5]).all()
    keep = [i for i in range(20) if i not in (3, 5)]
    assert torch.isfinite(C[keep]).all()


@pytest.mark.parametrize("M,K,N", [(1, 16, 16), (7, 144, 80), (77, 272, 528), (300, 512, 256)])
@pytest.mark.parametrize("rounding,rht", [("sr", True), ("rtn", False)])
def test_linear_forward_and_backward(M, K, N, rounding, rht):
    x, X = to_gpu(data(M, K, 1), torch.bfloat16)
    w, W = to_gpu(data(N, K, 2, spread=1) * np.float32(0.02), torch.float32)
    dy, dY = to_gpu(data(M, N, 3) * np.float32(1e-3), torch.bfloat16)
    Y, saved = tj2.mx_linear_fwd(x, w, N, y_dtype=torch.float32)
    same(saved["Xq"], mx.quantize(X), "Xq")
    same(saved["Wq"], mx.quantize(W), "Wq")
    dX, dW = tj2.mx_linear_bwd(dy, saved, K, seed=11, offset=16, rht=rht, dx_dtype=torch.float32,
                               rounding=tj2.SR if rounding == "sr" else tj2.RTN)
    ref = mx.linear(X, W, dY, rounding=rounding, rht=rht, seed=11, offset=16)
    for name, got, r, k in (("Y", Y, ref[0], K), ("dX", dX, ref[1], N), ("dW", dW, ref[2], M)):
        # fp32 sums over k terms: k half steps, each of a partial sum that random signs keep near the result's norm
        assert H.rel_fro(got.cpu().numpy(), r) <= (k + 16) * 2.0 ** -24 * 4, name
    # from given codes, as serving and a master pass have them
    Y2, _ = tj2.mx_linear_fwd(x, None, N, Wq=saved["Wq"], y_dtype=torch.float32)
    assert torch.equal(Y, Y2)


def test_backward_gradient_is_unbiased():
    """The mean of many stochastic backwards approaches the exact products of the quantized forward tensors."""
    M, K, N, n = 48, 64, 32, 256
    x, X = to_gpu(data(M, K, 4, spread=1), torch.bfloat16)
    w, W = to_gpu(data(N, K, 5, spread=1) * np.float32(0.1), torch.float32)
    dy, dY = to_gpu(data(M, N, 6, spread=1), torch.bfloat16)
    _, saved = tj2.mx_linear_fwd(x, w, N)
    xh, wh = mx.dequantize(mx.quantize(X)), mx.dequantize(mx.quantize(W))
    refs = dY.astype(np.float64) @ wh, dY.T.astype(np.float64) @ xh
    sums, one = [0.0, 0.0], None
    for i in range(n):
        got = [g.double().cpu().numpy() for g in tj2.mx_linear_bwd(dy, saved, K, seed=0, offset=8 * i, dx_dtype=torch.float32)]
        one = one or [H.rel_fro(g, r) for g, r in zip(got, refs)]
        sums = [s + g for s, g in zip(sums, got)]
    for s, r, o in zip(sums, refs, one):
        assert H.rel_fro(s / n, r) <= 2.0 * o / np.sqrt(n)  # twice the standard error of a mean of n


def test_wrapped_weights_streams_and_graph():
    x, _ = to_gpu(data(9, 160, 7), torch.bfloat16)
    w, _ = to_gpu(data(64, 160, 8), torch.float32)
    Wq = tj2.mx_quantize(w)
    wrapped = tj2.QTensor.wrap(tj2.MXFP4, 64, 160, Wq.codes.clone(), Wq.scale16.clone())
    want, _ = tj2.mx_linear_fwd(x, None, 64, Wq=Wq)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, _ = tj2.mx_linear_fwd(x, None, 64, Wq=wrapped)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    Y, Xq = torch.empty_like(want), tj2.QTensor(tj2.MXFP4, 9, 160)
    static = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tj2.mx_linear_fwd(static, None, 64, Wq=wrapped, Y=Y, Xq=Xq)
    for k in range(3):
        static.copy_(x * (k + 1))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, tj2.mx_linear_fwd(static.clone(), None, 64, Wq=Wq)[0])


def values(q):
    return tj2.mx_dequantize(q, dtype=torch.float32).double()


def near(got, A, B):
    """close() on the GPU: K + 16 half steps of fp32 on the sum of magnitudes and half a step of a bf16 result."""
    ref, mags = A @ B.T, A.abs() @ B.abs().T
    tol = (A.shape[1] + 16) * 2.0 ** -24 * mags + (ref.abs() * 2.0 ** -8 if got.dtype == torch.bfloat16 else 0)
    assert ((got.double() - ref).abs() <= tol).all(), float(((got.double() - ref).abs() - tol).max())


@pytest.mark.parametrize("I,J,K", [(2100, 1500, 2064), (3000, 2600, 1040), (2048, 4096, 256), (16384, 1024, 528), (1100, 9001, 272),
                                   (129, 50304, 144), (33, 17, 4096), (2049, 65, 16400)])
def test_gemm_of_every_tile_and_split(I, J, K):
    t, _ = to_gpu(data(I, K, 1, spread=1), torch.bfloat16)
    w, _ = to_gpu(data(J, K, 2, spread=1), torch.float32)
    qa, qb = tj2.mx_quantize(t), tj2.mx_quantize(w)
    A, B = values(qa), values(qb)
    near(tj2.mx_gemm(qa, qb, out_dtype=torch.bfloat16), A, B)
    near(tj2.mx_gemm(qa, qb), A, B)


@pytest.mark.parametrize("M,K,N", [(1, 16, 16), (16, 16, 4096), (17, 48, 16), (8192, 64, 128), (300, 1024, 8192), (2100, 1040, 1488),
                                   (5, 4096, 16), (127, 128, 129 * 16), (4097, 272, 32)])
@pytest.mark.parametrize("rht", [True, False])
def test_backward_products_of_every_shape(M, K, N, rht):
    """Both products against their operands, which mx_quantize gives bit for bit as the oracle does."""
    x, _ = to_gpu(data(M, K, 1), torch.bfloat16)
    w, _ = to_gpu(data(N, K, 2, spread=1), torch.float32)
    dy, _ = to_gpu(data(M, N, 3) * np.float32(1e-3), torch.bfloat16)
    Y, saved = tj2.mx_linear_fwd(x, w, N)
    near(Y, values(tj2.mx_quantize(x)), values(tj2.mx_quantize(w)))
    seed, offset = 9, 24
    for dt in (torch.bfloat16, torch.float32):
        dX, dW = tj2.mx_linear_bwd(dy, saved, K, seed=seed, offset=offset, rht=rht, dx_dtype=dt)
        sx, sw = (tj2.lib().tj2_rht_signs(seed, offset + o) if rht else 0 for o in (0, 2))
        opt = dict(rounding=tj2.SR, rht=rht, seed=seed)
        near(dX, values(tj2.mx_quantize(dy, signs=sx, offset=offset, **opt)),
             values(tj2.mx_quantize(saved["Wq"], grouping=tj2.GROUP_COL, signs=sx, offset=offset + 1, **opt)))
        near(dW, values(tj2.mx_quantize(dy, grouping=tj2.GROUP_COL, signs=sw, offset=offset + 2, **opt)),
             values(tj2.mx_quantize(saved["Xq"], grouping=tj2.GROUP_COL, signs=sw, offset=offset + 3, **opt)))


def test_backward_graphs_share_a_workspace():
    """Two captured backward passes with one workspace, replayed in turns among eager calls that use it too."""
    cases, ws = [], None
    for seed, (M, K, N) in ((1, (300, 1024, 8192)), (2, (70, 48, 96))):
        x, _ = to_gpu(data(M, K, seed), torch.bfloat16)
        w, _ = to_gpu(data(N, K, seed + 1), torch.float32)
        dy, _ = to_gpu(data(M, N, seed + 2), torch.bfloat16)
        ws = tj2.mx_linear_bwd_workspace(M, N, K) if ws is None else ws
        cases.append((dy, tj2.mx_linear_fwd(x, w, N)[1], K))
    opt = dict(seed=3, offset=8)
    want = [tj2.mx_linear_bwd(*c, **opt) for c in cases]
    graphs, held = [], [tuple(torch.empty_like(t) for t in w) for w in want]
    for c, (dX, dW) in zip(cases, held):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tj2.mx_linear_bwd(*c, **opt, dX=dX, dW=dW, workspace=ws)
        graphs.append(g)
    for k in (0, 1, 0, 0, 1):
        for t in held[k]:
            t.fill_(float("nan"))
        graphs[k].replay()
        other = tj2.mx_linear_bwd(*cases[1 - k], **opt, workspace=ws)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held[k], want[k]))
        assert all(torch.equal(a, b) for a, b in zip(other, want[1 - k]))


def test_operand_arrays_may_be_looked_at_and_replaced():
    """An operand's arrays are views of its storage; one that a caller puts in their place is what is used."""
    t, x = to_gpu(data(20, 272, 4), torch.bfloat16)
    q = tj2.mx_quantize(t)
    want = tj2.mx_dequantize(q)
    assert q.codes.shape == (20, 3 * 64) and q.scale16.shape == (20, 3 * 4)
    same(q, mx.quantize(x))
    assert torch.equal(tj2.mx_dequantize(q), want)
    other = tj2.mx_quantize(t)
    other.codes = torch.zeros_like(q.codes)
    assert (tj2.mx_dequantize(other) == 0).all() and torch.equal(other.scale16, q.scale16)
    other.codes, other.scale16 = q.codes.clone(), q.scale16.clone()
    assert torch.equal(tj2.mx_dequantize(other), want) and torch.equal(tj2.mx_dequantize(q.clone()), want)
    with pytest.raises(AttributeError):
        q.scale64


def test_binding_refuses():
    x = torch.zeros(4, 32, device="cuda", dtype=torch.bfloat16)
    w = torch.zeros(16, 32, device="cuda")
    q4 = tj2.quantize(x)
    for bad in (lambda: tj2.mx_quantize(x.half()), lambda: tj2.mx_quantize(x.t()), lambda: tj2.mx_quantize(x.cpu()),
                lambda: tj2.mx_quantize(x[:0]), lambda: tj2.mx_quantize(q4), lambda: tj2.mx_dequantize(q4),
                lambda: tj2.mx_gemm(q4, q4), lambda: tj2.mx_linear_fwd(x, None, 16), lambda: tj2.mx_linear_fwd(x, w, 8),
                lambda: tj2.mx_linear_fwd(x.float(), w, 16),
                lambda: tj2.QTensor.wrap(tj2.MXFP4, 4, 32, torch.zeros(4, 16, dtype=torch.uint8, device="cuda"), None)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(tj2.Tj2Error):
        tj2.mx_quantize(torch.zeros(4, 40, device="cuda"))
