"""The gated feed-forward block and its gradients against the formulas in 64 bits."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

tj2 = pytest.importorskip("bit_fully_quantized_amd")

H24, H8 = 2.0 ** -24, 2.0 ** -8  # half a step of fp32 and of bf16, relative
BF = torch.bfloat16
ACTS = ["silu", "gelu", "gelu_tanh"]


def normal(shape, seed, std=1.0, dtype=BF):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def make(T, D, F, seed=0):
    X = normal((T, D), seed)
    if D > 32:
        X[:, 5] *= 8
    return X, normal((F, D), seed + 1, 0.7 / math.sqrt(D)), normal((F, D), seed + 2, 0.7 / math.sqrt(D)), normal((D, F), seed + 3, 0.7 / math.sqrt(F))


def act64(name, g):
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * (1 - s)
    if name == "gelu":
        c = 0.5 * torch.special.erfc(-g / math.sqrt(2))
        return g * c, c + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)


class Exact:
    """Values and bounds of the error of each, from the roundings that the operator makes: fp32 sums of n products
    ((n + 8) half steps of their magnitudes), G and U kept in 24 bits (2^-17), activations within 2^-20 (exponential,
    reciprocal and a few operations; slopes below 1.2 in the next derivative), bf16 H, dG, dU and results."""

    def __init__(self, X, Wg, Wu, Wd, act, dY=None):
        X, Wg, Wu, Wd = (t.double() for t in (X, Wg, Wu, Wd))
        D, F = X.shape[1], Wg.shape[0]
        G, U = X @ Wg.T, X @ Wu.T
        eG, eU = (D + 8) * H24 * (X.abs() @ Wg.abs().T), (D + 8) * H24 * (X.abs() @ Wu.abs().T)
        a, da = act64(act, G)
        H = a * U
        ea = 1.2 * eG + 2.0 ** -20 * (a.abs() + G.abs())
        eH = ea * U.abs() + a.abs() * eU + ea * eU + 2.0 ** -20 * H.abs()
        eHr = eH + H8 * (H.abs() + eH)
        self.Y = H @ Wd.T, eHr @ Wd.abs().T + (F + 16) * H24 * (H.abs() @ Wd.abs().T)
        if dY is None:
            return
        dY = dY.double()
        dH, edH = dY @ Wd, (D + 8) * H24 * (dY.abs() @ Wd.abs())
        eG, eU = eG + 2.0 ** -16 * G.abs(), eU + 2.0 ** -16 * U.abs()
        ea = 1.2 * eG + 2.0 ** -20 * (a.abs() + G.abs())
        eda = 1.2 * eG + 2.0 ** -19 * (1 + G.abs())
        eHr = ea * U.abs() + a.abs() * eU + ea * eU + 2.0 ** -20 * H.abs()
        eHr = eHr + H8 * (H.abs() + eHr)
        dG, dU = dH * U * da, dH * a
        edG = edH * (U * da).abs() + dH.abs() * (eU * da.abs() + U.abs() * eda) + 2.0 ** -20 * dG.abs()
        edG = edG + H8 * (dG.abs() + edG)
        edU = edH * a.abs() + dH.abs() * ea + 2.0 ** -20 * dU.abs()
        edU = edU + H8 * (dU.abs() + edU)
        T = X.shape[0]

        def product(a, ea, b, n):
            return a @ b, ea @ b.abs() + (n + 40) * H24 * (a.abs() @ b.abs())
        g, u = product(dG, edG, Wg, 2 * F), product(dU, edU, Wu, 2 * F)
        self.dX = g[0] + u[0], g[1] + u[1]
        self.dWg, self.dWu = product(dG.T, edG.T, X, T), product(dU.T, edU.T, X, T)
        self.dWd = dY.T @ H, dY.abs().T @ eHr + (T + 40) * H24 * (dY.abs().T @ H.abs())


def check(got, ref, what=""):
    v, e = ref
    tol = e * 1.01 + (H8 if got.dtype == BF else H24) * (v.abs() + e) + 1e-38
    d = (got.double() - v).abs()
    assert (d <= tol).all(), (what, float((d / tol).max()))
    # the bounds add magnitudes; an error of the norm is far below them: roundings of the result and of two factors
    if v.numel() > 4096:
        assert float(d.norm() / v.norm()) <= 2 * H8, what


SIZES = [(1, 16, 16), (1, 1024, 4096), (2, 48, 80), (5, 144, 208), (16, 2048, 144), (17, 528, 320), (30, 1024, 176), (64, 512, 96),
         (64, 1040, 64), (65, 80, 144), (130, 128, 128), (200, 272, 528), (300, 96, 1040), (515, 656, 272), (1235, 528, 1552)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,D,F", SIZES)
def test_forward_and_backward(T, D, F, act):
    X, Wg, Wu, Wd = make(T, D, F)
    dY = normal((T, D), 9, 1e-2)
    ref = Exact(X, Wg, Wu, Wd, act, dY)
    Y, saved = tj2.gated_ffn_fwd(X, Wg, Wu, Wd, activation=act)
    assert saved is None
    check(Y, ref.Y, "Y")
    Y2, saved = tj2.gated_ffn_fwd(X, Wg, Wu, Wd, activation=act, save=True)
    assert torch.equal(Y, Y2)
    check(tj2.gated_ffn_fwd(X, Wg, Wu, Wd, activation=act, y_dtype=torch.float32)[0], ref.Y, "Y fp32")
    grads = tj2.gated_ffn_bwd(dY, X, Wg, Wu, Wd, saved, activation=act)
    for g, n in zip(grads, ("dX", "dWg", "dWu", "dWd")):
        check(g, getattr(ref, n), n)
    if act == "silu":
        for g, n in zip(tj2.gated_ffn_bwd(dY, X, Wg, Wu, Wd, saved, activation=act, dx_dtype=torch.float32, dw_dtype=torch.float32),
                        ("dX", "dWg", "dWu", "dWd")):
            check(g, getattr(ref, n), n)


def test_many_tokens():
    """From 2048 tokens on the operands are copied into blocks first."""
    for T, D, F in ((2048, 144, 400), (3001, 400, 272), (5000, 64, 1040)):
        X, Wg, Wu, Wd = make(T, D, F)
        dY = normal((T, D), 9, 1e-2)
        ref = Exact(X, Wg, Wu, Wd, "silu", dY)
        Y, saved = tj2.gated_ffn_fwd(X, Wg, Wu, Wd, save=True)
        check(Y, ref.Y, "Y")
        for g, n in zip(tj2.gated_ffn_bwd(dY, X, Wg, Wu, Wd, saved), ("dX", "dWg", "dWu", "dWd")):
            check(g, getattr(ref, n), n)


@pytest.mark.parametrize("T", [3, 150])
def test_each_gradient_alone(T):
    X, Wg, Wu, Wd = make(T, 144, 208)
    dY = normal((T, 144), 9, 1e-2)
    _, saved = tj2.gated_ffn_fwd(X, Wg, Wu, Wd, save=True)
    ref = Exact(X, Wg, Wu, Wd, "silu", dY)
    for m in range(1, 16):
        need = [bool(m >> k & 1) for k in range(4)]
        got = tj2.gated_ffn_bwd(dY, X, Wg, Wu, Wd, saved, need=need)
        for g, n, name in zip(got, need, ("dX", "dWg", "dWu", "dWd")):
            assert (g is not None) == n
            if n:
                check(g, getattr(ref, name), name)


@pytest.mark.parametrize("T", [1, 20, 140, 2100])
def test_pitches(T):
    """Weights that are parts of one matrix, tokens that are part of a wider one, and results in given buffers."""
    D, F = 144, 208
    X, Wg, Wu, Wd = make(T, D, F)
    dY = normal((T, D), 9, 1e-2)
    both = torch.cat((Wg, Wu))
    wide = torch.cat((Wd, normal((D, 64), 11)), 1)
    xs = torch.cat((normal((T, 24), 12), X), 1)
    ds = torch.cat((dY, normal((T, 8), 13)), 1)
    Y, saved = tj2.gated_ffn_fwd(X, Wg, Wu, Wd, save=True)
    args = (xs[:, 24:], both[:F], both[F:], wide[:, :F])
    out = torch.empty_like(Y)
    Y2, saved2 = tj2.gated_ffn_fwd(*args, save=True, Y=out)
    assert Y2 is out and torch.equal(Y, Y2)
    into = [torch.empty(s, dtype=BF, device="cuda") for s in ((T, D), (F, D), (F, D), (D, F))]
    got = tj2.gated_ffn_bwd(ds[:, :D], *args, saved2, dX=into[0], dWg=into[1], dWu=into[2], dWd=into[3])
    for a, b, c in zip(tj2.gated_ffn_bwd(dY, X, Wg, Wu, Wd, saved), got, into):
        assert b is c and torch.equal(a, b)


@pytest.mark.parametrize("T", [40, 150, 2100])
def test_a_bad_token_stays_alone(T):
    D, F = 144, 208
    X, Wg, Wu, Wd = make(T, D, F)
    dY = normal((T, D), 9, 1e-2)
    Y, saved = tj2.gated_ffn_fwd(X, Wg, Wu, Wd, save=True)
    dX = tj2.gated_ffn_bwd(dY, X, Wg, Wu, Wd, saved, need=(True, False, False, False))[0]
    Xb = X.clone()
    Xb[7, 3], Xb[T - 1, 0] = float("nan"), float("inf")
    Yb, savedb = tj2.gated_ffn_fwd(Xb, Wg, Wu, Wd, save=True)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[7] = keep[T - 1] = False
    assert torch.equal(Yb[keep], Y[keep]) and torch.isnan(Yb[7].float()).all() and not torch.isfinite(Yb[T - 1].float()).any()
    dXb = tj2.gated_ffn_bwd(dY, Xb, Wg, Wu, Wd, savedb, need=(True, False, False, False))[0]
    assert torch.equal(dXb[keep], dX[keep]) and torch.isnan(dXb[7].float()).all()


def test_far_gates():
    """Gates far out on either side: activations and slopes are 0 or 1 there, never NaN."""
    T, D, F = 24, 16, 32
    X = torch.zeros(T, D, dtype=BF, device="cuda")
    Wg, Wu = torch.zeros(F, D, dtype=BF, device="cuda"), torch.zeros(F, D, dtype=BF, device="cuda")
    X[:, 0], X[:, 1] = torch.linspace(-1, 1, T, device="cuda").to(BF), 1.0
    Wg[:, 0] = torch.logspace(0, 30, F, device="cuda").to(BF)
    Wu[:, 1] = 1.0
    Wd, dY = normal((D, F), 3), normal((T, D), 4)
    for act in ACTS:
        ref = Exact(X, Wg, Wu, Wd, act, dY)
        Y, saved = tj2.gated_ffn_fwd(X, Wg, Wu, Wd, activation=act, save=True)
        assert torch.isfinite(Y.float()).all()
        grads = tj2.gated_ffn_bwd(dY, X, Wg, Wu, Wd, saved, activation=act, dx_dtype=torch.float32)
        assert all(torch.isfinite(g.float()).all() for g in grads)
        check(Y, ref.Y, act)
        # slopes: dWg's column 0 is sum_t dG x0, of which the far gates' slopes are 0 or 1
        dG = (dY.double() @ Wd.double()) * act64(act, (X.double() @ Wg.double().T))[1].nan_to_num()
        far = (X.double() @ Wg.double().T).abs() > 40
        sign = ((X.double() @ Wg.double().T) > 0).double()
        dG = torch.where(far, (dY.double() @ Wd.double()) * sign, dG)
        want = dG.T @ X.double()
        mag = (dY.double().abs() @ Wd.double().abs()).T @ X.double().abs()
        assert ((grads[1].double() - want).abs() <= 3 * H8 * 1.2 * mag + 1e-30).all(), act


@pytest.mark.parametrize("act", ACTS)
def test_differentiable(act):
    """Gradients of a scalar against torch's own of the formula in 64 bits, and against differences."""
    T, D, F = 33, 48, 80
    leaves = [t.requires_grad_() for t in make(T, D, F)]
    c = normal((T, D), 9, 1.0, torch.float32)
    loss = (tj2.gated_ffn(*leaves, activation=act).float() * c).sum()
    got = torch.autograd.grad(loss, leaves)

    def f(X, Wg, Wu, Wd):
        return ((act64(act, X @ Wg.T)[0] * (X @ Wu.T)) @ Wd.T * c.to(BF).double()).sum()
    d = [t.detach().double().requires_grad_() for t in leaves]
    want = torch.autograd.grad(f(*d), d)
    for i, (p, q) in enumerate(zip(got, want)):
        # dG, dU or H rounded to bf16, and the result: two half steps of the norm
        assert float((p.double() - q).norm() / q.norm()) <= 2 * H8, i
        e = normal(q.shape, 20 + i, 1.0, torch.float64)
        h = 1e-5
        up, down = ([t.detach() + (s * h * e if j == i else 0) for j, t in enumerate(d)] for s in (1, -1))
        diff = float((f(*up) - f(*down)) / (2 * h))
        assert abs(float((p.double() * e).sum()) - diff) <= 2 * H8 * float(q.norm() * e.norm())
    # a part of the leaves
    part = [leaves[0], leaves[1].detach(), leaves[2], leaves[3].detach()]
    a = torch.autograd.grad((tj2.gated_ffn(*part, activation=act).float() * c).sum(), [leaves[0], leaves[2]])
    assert torch.equal(a[0], got[0]) and torch.equal(a[1], got[2])
    with torch.no_grad():
        assert torch.equal(tj2.gated_ffn(*leaves, activation=act), tj2.gated_ffn_fwd(*[t.detach() for t in leaves], activation=act)[0])


def test_streams_graphs_and_shared_workspaces():
    T, D, F = 200, 144, 400
    xs = [make(T, D, F, s)[0] for s in (0, 50)]
    _, Wg, Wu, Wd = make(T, D, F)
    ds = [normal((T, D), s, 1e-2) for s in (9, 10)]
    want = []
    for x, d in zip(xs, ds):
        Y, saved = tj2.gated_ffn_fwd(x, Wg, Wu, Wd, save=True)
        want.append((Y, *tj2.gated_ffn_bwd(d, x, Wg, Wu, Wd, saved)))
    streams, got = [torch.cuda.Stream() for _ in xs], []
    torch.cuda.synchronize()
    for st, x, d in zip(streams, xs, ds):
        with torch.cuda.stream(st):
            Y, saved = tj2.gated_ffn_fwd(x, Wg, Wu, Wd, save=True)
            got.append((Y, *tj2.gated_ffn_bwd(d, x, Wg, Wu, Wd, saved)))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    L = tj2.lib()
    room = max(L.tj2_gated_ffn_fwd_workspace_size(T, D, F), L.tj2_gated_ffn_bwd_workspace_size(T, D, F))
    ws = torch.empty(room, dtype=torch.uint8, device="cuda")
    x, d = xs[0].clone(), ds[0].clone()
    gu = torch.empty(tj2.gated_ffn_saved_size(T, F), dtype=torch.uint8, device="cuda")
    outs = [torch.empty(s, dtype=BF, device="cuda") for s in ((T, D), (T, D), (F, D), (F, D), (D, F))]
    side, graphs = torch.cuda.Stream(), []
    with torch.cuda.stream(side):
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                _, saved = tj2.gated_ffn_fwd(x, Wg, Wu, Wd, gu=gu, Y=outs[0], workspace=ws)
                tj2.gated_ffn_bwd(d, x, Wg, Wu, Wd, saved, dX=outs[1], dWg=outs[2], dWu=outs[3], dWd=outs[4], workspace=ws)
            graphs.append(g)
    torch.cuda.synchronize()
    for i in range(6):
        x.copy_(xs[i % 2])
        d.copy_(ds[i % 2])
        ws.fill_(255)  # NaNs, were any of it read before it is written
        graphs[i // 2 % 2].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(want[i % 2], outs)), i
        tj2.gated_ffn_fwd(xs[1], Wg, Wu, Wd)


@pytest.mark.parametrize("T", range(1, 10))
@pytest.mark.parametrize("D,F", [(16, 16), (112, 336), (1024, 528)])
def test_up_to_eight_tokens_keep_both_parts_of_h(T, D, F):
    """H in two bf16 parts: what the first leaves is at most 2^-8 of H and rounded by 2^-8 of itself."""
    X, Wg, Wu, Wd = make(T, D, F)
    x, g, u, d = (t.double() for t in (X, Wg, Wu, Wd))
    G, U = x @ g.T, x @ u.T
    eG, eU = (D + 8) * H24 * (x.abs() @ g.abs().T), (D + 8) * H24 * (x.abs() @ u.abs().T)
    a = act64("silu", G)[0]
    ea = 1.2 * eG + 2.0 ** -20 * (a.abs() + G.abs())
    H = a * U
    eH = ea * U.abs() + a.abs() * eU + ea * eU + 2.0 ** -20 * H.abs()
    eH = eH + (2.0 ** -16 if T <= 8 else H8) * (H.abs() + eH)
    bound = (eH @ d.abs().T + (2 * F + 16) * H24 * (H.abs() @ d.abs().T)) * 1.01
    Y = tj2.gated_ffn_fwd(X, Wg, Wu, Wd, y_dtype=torch.float32)[0].double()
    assert ((Y - H @ d.T).abs() <= bound).all()
    alone = torch.cat([tj2.gated_ffn_fwd(X[t:t + 1], Wg, Wu, Wd, y_dtype=torch.float32)[0] for t in range(T)]).double()
    assert ((alone - H @ d.T).abs() <= bound).all()


@pytest.mark.parametrize("T", [1, 8, 9, 40])
def test_products_that_leave_the_range(T):
    """H beyond fp32 is infinite and so is Y (not a difference of infinities), for its own token."""
    X = torch.zeros(T, 32, device="cuda", dtype=BF)
    X[T - 1, :4] = 2.0 ** 60
    X[0, 4:8] = 1.0
    W = torch.full((48, 32), 2.0 ** 10, device="cuda", dtype=BF)
    Y = tj2.gated_ffn_fwd(X, W, W, torch.full((32, 48), 0.5, device="cuda", dtype=BF))[0]
    assert (Y[T - 1] == float("inf")).all() and torch.isfinite(Y[: T - 1]).all()
    # 24 2^24 of 48 features: exact
    assert T == 1 or (Y[0] == 24.0 * 2.0 ** 24).all()
