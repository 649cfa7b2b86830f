"""Root-mean-square norm with the residual's addition, its FP8 result and its gradients, against the formulas in 64 bits."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

tj2 = pytest.importorskip("bit_fully_quantized_amd")

H24, H8 = 2.0 ** -24, 2.0 ** -8
EPS = 1e-6
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {torch.bfloat16: H8, torch.float32: H24}


def normal(shape, seed, std=1.0, dtype=torch.float32):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def plain(x, w, res, eps=EPS):
    """(y, s, rstd) in 64 bits, s rounded to x's type as the definition says."""
    s = x.double() if res is None else (x.double() + res.double()).to(x.dtype).double()
    r = 1.0 / torch.sqrt((s * s).mean(1, keepdim=True) + eps)
    return s * r * w.double(), s, r[:, 0]


def stat(cols):
    """fp32 relative error of rstd: a sum of cols squares (threads add 32 at most, or cols / 256 of long rows, then 6 to
    8 levels), half of it through the root, the division, addition and roots' half steps."""
    return (max(32, cols / 256) + 8 + 6) * H24


SIZES = [(1, 1), (1, 7), (3, 16), (2, 33), (5, 511), (4, 512), (7, 513), (1, 1024), (300, 1003), (9, 1024), (5, 2048), (3, 2056),
         (6, 4096), (2, 4104), (3, 8192), (2, 8193), (3, 20000), (2, 8200), (4500, 64), (2100, 2100)]


@pytest.mark.parametrize("dtype,wtype", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("residual", [False, True])
def test_forward_and_backward(rows, cols, residual, dtype, wtype):
    T = DT[dtype]
    x, w = normal((rows, cols), 1, 0.7, T), (1.0 + normal(cols, 2, 0.1)).to(DT[wtype])
    res = normal((rows, cols), 3, 1.5, T) if residual else None
    y, s, rstd = tj2.rms_norm_fwd(x, w, residual=res, eps=EPS)
    ry, rs, rr = plain(x, w, res)
    assert y.dtype == T and y.shape == x.shape
    if residual:
        # bf16 sums of bf16 numbers: fp32 holds them up to 2^-24, which can move a tie
        exact = (x.float() + res.float()).to(T)
        assert torch.equal(s, exact)
        rs = exact.double()
        rr = 1.0 / torch.sqrt((rs * rs).mean(1) + EPS)
        ry = rs * rr[:, None] * w.double()
    else:
        assert s is x
    e = stat(cols)
    assert ((rstd.double() - rr).abs() <= e * rr).all()
    assert ((y.double() - ry).abs() <= (HALF[T] + e + 4 * H24) * ry.abs() * 1.001).all()
    # backward, with and without what comes in for s
    dy = normal((rows, cols), 4, 1e-2, T)
    for dsum in (None, normal((rows, cols), 5, 1e-2, T)):
        ds, dw = tj2.rms_norm_bwd(dy, s, w, rstd, dsum=dsum)
        assert ds.dtype == T and dw.dtype == DT[wtype]
        g, wd, r = dy.double(), w.double(), rr[:, None]
        xh = rs * r
        c = (g * wd * xh).mean(1, keepdim=True)
        ref = r * (g * wd - xh * c)
        # magnitudes that enter: each fp32 operation's half step, the mean's sum and rstd's error
        mag = r * ((g * wd).abs() + xh.abs() * (g * wd * xh).abs().mean(1, keepdim=True))
        if dsum is not None:
            ref, mag = ref + dsum.double(), mag + dsum.double().abs()
        tol = HALF[T] * ref.abs() + (4 * e + 8 * H24) * mag
        assert ((ds.double() - ref).abs() <= tol * 1.001).all()
        rw, mw = (g * xh).sum(0), (g * xh).abs().sum(0)
        tol = HALF[DT[wtype]] * rw.abs() + (rows + 64 + 8) * H24 * mw + 2 * e * mw
        assert ((dw.double() - rw).abs() <= tol).all()
    only, none = tj2.rms_norm_bwd(dy, s, w, rstd, need_dw=False)
    assert none is None and torch.equal(only, tj2.rms_norm_bwd(dy, s, w, rstd)[0])
    none, dw = tj2.rms_norm_bwd(dy, s, w, rstd, need_ds=False)
    assert none is None and torch.equal(dw, tj2.rms_norm_bwd(dy, s, w, rstd)[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 1024), (5, 144), (130, 528), (7, 2048), (3, 4112), (5, 8192), (2, 8208), (2, 20000), (9000, 48)])
@pytest.mark.parametrize("residual", [False, True])
def test_fp8_result(rows, cols, residual, dtype):
    T = DT[dtype]
    x, w = normal((rows, cols), 1, 0.7, T), 1.0 + normal(cols, 2, 0.1)
    res = normal((rows, cols), 3, 1.5, T) if residual else None
    if rows > 2:
        x[1] = 0.0
        if residual:
            res[1] = 0.0
    q, s, rstd = tj2.rms_norm_fwd(x, w, residual=res, eps=EPS, fp8=True)
    y32, s2, rstd2 = tj2.rms_norm_fwd(x, w, residual=res, eps=EPS)
    assert torch.equal(s, s2) and torch.equal(rstd, rstd2)
    rs = s.double()
    ref = rs * (1.0 / torch.sqrt((rs * rs).mean(1, keepdim=True) + EPS)) * w.double()
    if T == torch.float32:  # the same numbers, quantized as fp8_quantize does
        p = tj2.fp8_quantize(y32)
        assert torch.equal(p.codes, q.codes) and torch.equal(p.scale128, q.scale128)
    e = stat(cols) + 4 * H24
    pad = torch.nn.functional.pad(ref, (0, -cols % 128)).view(rows, -1, 128)
    S = pad.abs().amax(2) / 448.0
    assert ((q.scale128.double() - S).abs() <= (e + 2 * H24) * S).all()
    v = tj2.fp8_dequantize(q, dtype=torch.float32).double()
    # half a step of E4M3: 2^-4 of the value, or 2^-10 of the scale where it is subnormal
    tol = torch.maximum(2.0 ** -4 * ref.abs(), 2.0 ** -10 * S.repeat_interleave(128, 1)[:, :cols])
    assert ((v - ref).abs() <= tol * 1.0001 + e * ref.abs()).all()
    assert not q.codes[:, cols:].any()


def test_pitches_and_results_in_place():
    rows, cols = 37, 200
    for T in (torch.bfloat16, torch.float32):
        X, R = normal((rows, 3 * cols), 1, 1.0, T), normal((rows, 2 * cols + 8), 2, 1.0, T)
        w = 1.0 + normal(cols, 3, 0.1)
        for a, b in ((0, 0), (cols, cols), (3, 5)):  # the last: no row is aligned
            x, r = X[:, a:a + cols], R[:, b:b + cols]
            want = tj2.rms_norm_fwd(x.contiguous(), w, residual=r.contiguous())
            got = tj2.rms_norm_fwd(x, w, residual=r)
            # another way through a row is another order of its sum
            assert torch.equal(got[1], want[1])
            assert ((got[0].double() - want[0].double()).abs() <= (2 * HALF[T] + 2 * stat(cols)) * want[0].double().abs()).all()
            dy, dsum = X[:, a + 5:a + 5 + cols], R[:, b + 1:b + 1 + cols]
            ds, dw = tj2.rms_norm_bwd(dy, got[1], w, got[2], dsum=dsum)
            ds2, dw2 = tj2.rms_norm_bwd(dy.contiguous(), got[1], w, got[2], dsum=dsum.contiguous())
            assert float((ds.double() - ds2.double()).norm() / ds2.double().norm()) <= 2 * HALF[T]
            assert float((dw - dw2).norm() / dw2.norm()) <= 64 * H24
        for cols2 in (cols, 2048, 9000):
            x, r = normal((rows, cols2), 1, 1.0, T), normal((rows, cols2), 2, 1.0, T)
            w2 = 1.0 + normal(cols2, 3, 0.1)
            want = tj2.rms_norm_fwd(x, w2, residual=r)
            for into in (x.clone(), r.clone()):
                same_x = torch.equal(into, x)
                got = tj2.rms_norm_fwd(into if same_x else x, w2, residual=r if same_x else into, sum=into)
                assert got[1] is into and torch.equal(into, want[1]) and torch.equal(got[0], want[0])
            dy, dsum = normal((rows, cols2), 4, 1.0, T), normal((rows, cols2), 5, 1.0, T)
            ds = tj2.rms_norm_bwd(dy, want[1], w2, want[2], dsum=dsum)[0]
            for into in (dy.clone(), dsum.clone()):
                first = torch.equal(into, dy)
                got = tj2.rms_norm_bwd(into if first else dy, want[1], w2, want[2], dsum=dsum if first else into, ds=into)[0]
                assert got is into and torch.equal(into, ds)


def test_rows_of_zeros_infinities_and_nans():
    for T in (torch.bfloat16, torch.float32):
        x, w = normal((6, 256), 1, 1.0, T), torch.ones(256, device="cuda")
        x[1], x[2, 9], x[3, 200] = 0.0, float("inf"), float("nan")
        y, _, rstd = tj2.rms_norm_fwd(x, w)
        assert (y[1] == 0).all() and torch.isfinite(y[[0, 4, 5]].float()).all()
        assert torch.isnan(y[3].float()).all() and torch.isnan(y[2, 9].float()) and (y[2, :9] == 0).all()
        q, _, _ = tj2.rms_norm_fwd(x, w, fp8=True)
        v = tj2.fp8_dequantize(q)
        assert torch.isnan(v[3].float()).all() and torch.isnan(v[2, :128].float()).all() and torch.isfinite(v[[0, 1, 4, 5]].float()).all()
        ok = [0, 1, 4, 5]
        dy = normal((6, 256), 2, 1.0, T)
        ds, _ = tj2.rms_norm_bwd(dy, x, w, rstd)
        alone, _ = tj2.rms_norm_bwd(dy[ok].contiguous(), x[ok].contiguous(), w, rstd[ok].contiguous())
        assert torch.equal(ds[ok], alone) and torch.isnan(ds[3].float()).all()


@pytest.mark.parametrize("residual", [False, True])
def test_differentiable(residual):
    """Gradients of a scalar of y and s against torch's own of the formula in 64 bits, and against differences."""
    rows, cols = 21, 304
    x, w = normal((rows, cols), 1, 0.7).requires_grad_(), (1.0 + normal(cols, 2, 0.1)).requires_grad_()
    res = normal((rows, cols), 3, 1.5).requires_grad_() if residual else None
    a, b = normal((rows, cols), 4).double(), normal((rows, cols), 5).double()

    def f(x, w, r):
        s = x if r is None else x + r
        y = s * torch.rsqrt((s * s).mean(1, keepdim=True) + EPS) * w
        return (y * a).sum() + (0 if r is None else (s * b).sum())
    out = tj2.rms_norm(x, w, res, eps=EPS)
    loss = (out[0] * a).sum() + (out[1] * b).sum() if residual else (out * a).sum()
    leaves = [x, w] + ([res] if residual else [])
    got = torch.autograd.grad(loss, leaves)
    d = [t.detach().double().requires_grad_() for t in leaves]
    want = torch.autograd.grad(f(*d, *([None] if not residual else [])), d)
    for p, q in zip(got, want):
        assert float((p.double() - q).norm() / q.norm()) <= 8 * stat(cols)
    for i in range(len(d)):
        e = normal(d[i].shape, 9 + i).double()
        h = 1e-5
        up, down = [[t.detach() + (sign * h * e if j == i else 0) for j, t in enumerate(d)] for sign in (1, -1)]
        diff = (f(*up, *([None] if not residual else [])) - f(*down, *([None] if not residual else []))) / (2 * h)
        # the third derivative's h^2 and 64-bit rounding over h are far below the fp32 gradients' own error
        assert abs(float((got[i].double() * e).sum() - diff)) <= 8 * stat(cols) * float(got[i].double().norm() * e.norm())


def test_differentiable_parts():
    x, r = normal((5, 64), 1).requires_grad_(), normal((5, 64), 2).requires_grad_()
    w = torch.ones(64, device="cuda", requires_grad=True)
    y, s = tj2.rms_norm(x, w, r)
    gx, gr = torch.autograd.grad(s.sum(), [x, r], retain_graph=True)  # s alone
    assert (gx == 1).all() and (gr == 1).all()
    gw, = torch.autograd.grad(y.sum(), [w], retain_graph=True)
    gx, = torch.autograd.grad(y.sum(), [x])
    assert torch.isfinite(gw).all() and torch.isfinite(gx).all()
    y, s = tj2.rms_norm(x.detach(), w, r.detach())
    assert not s.requires_grad or torch.autograd.grad(y.sum() + s.sum(), [w])[0].shape == (64,)
    (2 * tj2.rms_norm(x, w)).sum().backward()
    (2 * tj2.rms_norm(x, w)).sum().backward()  # adds up
    one = x.grad.clone()
    x.grad = None
    (2 * tj2.rms_norm(x, w)).sum().backward()
    assert torch.equal(one, 2 * x.grad)


def test_streams_graphs_and_order():
    rows, cols = 5000, 520
    x, w, r = normal((rows, cols), 1, 1.0, torch.bfloat16), 1.0 + normal(cols, 2, 0.1), normal((rows, cols), 3, 1.0, torch.bfloat16)
    dy = normal((rows, cols), 4, 1.0, torch.bfloat16)
    y, s, rstd = tj2.rms_norm_fwd(x, w, residual=r)
    ds, dw = tj2.rms_norm_bwd(dy, s, w, rstd)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(3):
            y2, s2, rstd2 = tj2.rms_norm_fwd(x, w, residual=r)
            ds2, dw2 = tj2.rms_norm_bwd(dy, s2, w, rstd2)
    side.synchronize()
    assert torch.equal(y, y2) and torch.equal(ds, ds2) and torch.equal(dw, dw2)
    ins = (x.clone(), dy.clone())
    outs = dict(y=torch.empty_like(y), sum=torch.empty_like(s), rstd=torch.empty_like(rstd))
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    gs, gw = torch.empty_like(ds), torch.empty_like(dw)
    graphs = []
    with torch.cuda.stream(side):
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                tj2.rms_norm_fwd(ins[0], w, residual=r, **outs)
                tj2.rms_norm_bwd(ins[1], outs["sum"], w, outs["rstd"], ds=gs, dweight=gw, workspace=ws)
            graphs.append(g)
    torch.cuda.synchronize()
    for i in range(4):
        ws.fill_(255)
        k = -1.0 if i % 2 else 1.0
        ins[1].copy_(dy * k)
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs["y"], y) and torch.equal(gs, ds * k) and torch.equal(gw, dw * k)
        tj2.rms_norm_bwd(dy, s, w, rstd)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [1000, 1003, 9000, 9001])
def test_gradient_over_its_inputs(cols, dtype):
    """ds in dy's, s' or dsum's place: both gradients are what they are apart."""
    T = DT[dtype]
    dy, s, dsum = (normal((130, cols), i, 1.0, T) for i in (1, 2, 3))
    w = 1.0 + normal(cols, 4, 0.1)
    rstd = tj2.rms_norm_fwd(s, w)[2]
    want = tj2.rms_norm_bwd(dy, s, w, rstd, dsum=dsum)
    for i in range(3):
        a = [dy.clone(), s.clone(), dsum.clone()]
        ds, dw = tj2.rms_norm_bwd(a[0], a[1], w, rstd, dsum=a[2], ds=a[i])
        assert ds is a[i] and torch.equal(ds, want[0]) and torch.equal(dw, want[1])


@pytest.mark.parametrize("cols", [*range(1, 26), 63, 127, 129, 255, 505, 520, 1017, 1031, 2041, 2047, 4095, 4097, 8185, 8191])
def test_lengths_about_the_vectors(cols):
    """Rows that end within a vector, at every place of one, between others' rows that are not to be read or written."""
    for T in (torch.bfloat16, torch.float32):
        X = torch.full((5, cols + 16), float("nan"), device="cuda", dtype=T)
        X[:, 8:8 + cols] = normal((5, cols), 1, 1.0, T)
        x, w = X[:, 8:8 + cols], (1.0 + normal(cols, 2, 0.1)).to(T)
        out = torch.full((7, cols), 5.0, device="cuda", dtype=T)
        y, _, rstd = tj2.rms_norm_fwd(x, w, y=out[1:6])
        ry, rs, rr = plain(x, w, None)
        e = stat(cols)
        assert ((rstd.double() - rr).abs() <= e * rr).all()
        assert ((y.double() - ry).abs() <= (HALF[T] + e + 4 * H24) * ry.abs() * 1.001).all()
        assert (out[0] == 5.0).all() and (out[6] == 5.0).all()
        dy = normal((5, cols), 3, 1.0, T)
        out.fill_(5.0)
        ds, dw = tj2.rms_norm_bwd(dy, x, w, rstd, ds=out[1:6])
        assert (out[0] == 5.0).all() and (out[6] == 5.0).all()
        xr = x.double() * rstd.double()[:, None]
        g = dy.double() * w.double()
        full = rstd.double()[:, None] * (g - xr * (g * xr).mean(1, keepdim=True))
        # the terms that cancel count: r |g| and r |x r| mean |g x r|, each step half of one, the mean a sum as rstd's
        top = rstd.double()[:, None] * (g.abs() + xr.abs() * (g * xr).abs().mean(1, keepdim=True))
        assert ((ds.double() - full).abs() <= HALF[T] * full.abs() * 1.001 + (e + 8 * H24) * top).all()
        rw, tw = (dy.double() * xr).sum(0), (dy.double() * xr).abs().sum(0)
        assert ((dw.double() - rw).abs() <= HALF[T] * rw.abs() * 1.001 + 16 * H24 * tw).all()
