"""The head's losses on the GPU against plain fp64: values and gradients with bounds from their roundings,
ragged sizes, masks, pitches, special values, pieces and splits, streams, graphs and autograd."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

tj2 = pytest.importorskip("bit_fully_quantized_amd")

H24, H8 = 2.0 ** -24, 2.0 ** -8  # half a step of fp32 and of bf16, relative
NAN, INF = float("nan"), float("inf")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def ce_inputs(T, K, V, seed, learned=8.0, ignored=0.1):
    g = gen(seed)
    W = (torch.randn(V, K, generator=g, device="cuda") * 0.05).bfloat16()
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    X = torch.randn(T, K, generator=g, device="cuda")
    Wy = W[y].float()
    X += learned * torch.rand(T, 1, generator=g, device="cuda") * Wy / Wy.norm(dim=1, keepdim=True)
    y[torch.rand(T, generator=g, device="cuda") < ignored] = -100
    return X.bfloat16(), W, y, g


def ce_check(X, W, y, dloss, ignore=-100, dx_dtype=torch.bfloat16, dw_dtype=torch.bfloat16):
    loss, lse = tj2.linear_ce_fwd(X, W, y, ignore_index=ignore)
    dX, dW = tj2.linear_ce_bwd(X, W, y, lse, dloss, ignore_index=ignore, dx_dtype=dx_dtype, dw_dtype=dw_dtype)
    x, w, c, K = X.double(), W.double(), dloss.double(), X.shape[1]
    keep = y != ignore
    at = torch.where(keep, y, 0)
    z = x @ w.T
    rlse = torch.logsumexp(z, 1)
    rows = torch.arange(len(y), device="cuda")
    rloss = torch.where(keep, rlse - z[rows, at], 0.0)
    # a logit is an fp32 sum of K exact products: K + 16 half steps of the sum of magnitudes at most; exp2, log2 and
    # their fp32 arguments (of up to |z| log2 e + the row's maximum): 8 half steps of them; the join and the
    # subtraction: 8 of their operands
    ez = (K + 16) * H24 * (x.abs() @ w.abs().T)
    top = z.abs().amax(1)
    tol = 2 * ez.amax(1) + 16 * H24 * (2 * top + rlse.abs() + 1)
    assert ((lse.double() - rlse).abs() <= tol).all()
    assert ((loss.double() - rloss).abs() <= tol * 2).all()
    assert (loss[~keep] == 0).all()
    p = torch.exp(z - rlse[:, None])
    c = torch.where(keep, c, 0.0)
    dz = p * c[:, None]
    dz[rows, at] -= c
    # dz: p off by the exponent's error, then half a bf16 step; products exact, sums fp32 (half a step of the sum of
    # magnitudes a term); outputs half a step of their type
    # (the exponential's hardware result below the smallest normal, 2^-126, is 0: p is off by less than that)
    edz = (p * (ez + tol[:, None] + 16 * H24 * (1 + top[:, None])) + 2.0 ** -126) * c.abs()[:, None] + dz.abs() * H8
    # the fp32 sum of n terms in tiles, pieces and splits: (n + 64) half steps bound it
    for name, got, ref, bound, n in (("dX", dX, dz @ w, edz @ w.abs() + (len(w) + 64) * H24 * (dz.abs() @ w.abs()), len(w)),
                                     ("dW", dW, dz.T @ x, edz.T @ x.abs() + (len(x) + 64) * H24 * (dz.abs().T @ x.abs()), len(x))):
        half = H8 if got.dtype == torch.bfloat16 else H24
        err = (got.double() - ref).abs()
        lim = bound * (1 + half) + ref.abs() * half + 2.0 ** -130
        assert (err <= lim).all(), (name, float((err / lim).max()))
        # and taken together, where independent roundings (a third of a half step each) average out
        if ref.numel() > 4096 and float(ref.norm()) > 0:
            assert float(err.norm() / ref.norm()) <= 2 * H8, name
    return loss, lse, dX, dW


@pytest.mark.parametrize("T,K,V", [(1, 16, 1), (1, 32, 7), (5, 64, 300), (37, 528, 1003), (130, 256, 515), (513, 64, 2049),
                                   (64, 1024, 4999), (300, 144, 70000), (4, 48, 33)])
def test_cross_entropy_sizes(T, K, V):
    X, W, y, g = ce_inputs(T, K, V, T + K + V)
    ce_check(X, W, y, torch.rand(T, generator=g, device="cuda") - 0.3)


@pytest.mark.parametrize("T,K,V", [(16384, 64, 5000), (9000, 1024, 9001)])
def test_cross_entropy_in_pieces(T, K, V):
    X, W, y, g = ce_inputs(T, K, V, 1)
    ce_check(X, W, y, torch.full((T,), 1.0 / T, device="cuda"), dw_dtype=torch.float32, dx_dtype=torch.float32)


@pytest.mark.parametrize("dx,dw", [(torch.float32, torch.float32), (torch.bfloat16, torch.float32)])
def test_cross_entropy_fp32_gradients(dx, dw):
    X, W, y, g = ce_inputs(70, 96, 801, 3)
    ce_check(X, W, y, torch.randn(70, generator=g, device="cuda") * 1e-3, dx_dtype=dx, dw_dtype=dw)


def test_cross_entropy_gradient_against_differences():
    X, W, y, _ = ce_inputs(6, 32, 50, 4, ignored=0.0)
    d = torch.ones(6, device="cuda")
    _, lse = tj2.linear_ce_fwd(X, W, y)
    dX, dW = tj2.linear_ce_bwd(X, W, y, lse, d, dx_dtype=torch.float32, dw_dtype=torch.float32)

    def total(x, w):
        z = x @ w.T
        return (torch.logsumexp(z, 1) - z[torch.arange(6, device="cuda"), y]).sum()
    g, h = gen(5), 1e-6
    for got, which in ((dX, 0), (dW, 1)):
        v = torch.randn(got.shape, generator=g, device="cuda", dtype=torch.float64)
        x, w = X.double(), W.double()
        diff = (total(x + h * v, w) - total(x - h * v, w) if which == 0 else total(x, w + h * v) - total(x, w - h * v)) / (2 * h)
        # each dz entry is off by half a bf16 step of at most 1, times the other operand's magnitude
        other = W.double().abs().sum(0).max() if which == 0 else X.double().abs().sum(0).max()
        assert abs(float((got.double() * v).sum() - diff)) <= float(v.abs().sum() * other) * 2 * H8


def test_cross_entropy_all_ignored_and_other_ignore_index():
    X, W, y, _ = ce_inputs(33, 64, 90, 6, ignored=0.0)
    y[:] = 7
    loss, lse, dX, dW = ce_check(X, W, y, torch.ones(33, device="cuda"), ignore=7)
    assert (dX == 0).all() and (dW == 0).all() and (loss == 0).all()


def test_cross_entropy_ignored_rows_may_hold_anything():
    X, W, y, _ = ce_inputs(40, 64, 500, 7, ignored=0.0)
    y[3] = y[17] = -100
    d = torch.ones(40, device="cuda")
    loss, lse = tj2.linear_ce_fwd(X, W, y)
    dX, _ = tj2.linear_ce_bwd(X, W, y, lse, d)
    Xb = X.clone()
    Xb[3] = NAN
    Xb[17] = INF
    loss2, lse2 = tj2.linear_ce_fwd(Xb, W, y)
    dX2, _ = tj2.linear_ce_bwd(Xb, W, y, lse2, d)
    assert torch.equal(loss, loss2) and torch.equal(dX, dX2) and (loss2[[3, 17]] == 0).all()


def test_cross_entropy_target_outside_is_nan():
    X, W, y, _ = ce_inputs(20, 64, 100, 8, ignored=0.0)
    y[4], y[9] = 100, -3
    loss, lse = tj2.linear_ce_fwd(X, W, y)
    assert torch.isnan(loss[[4, 9]]).all() and int(torch.isnan(loss).sum()) == 2 and torch.isfinite(lse).all()
    dX, _ = tj2.linear_ce_bwd(X, W, y, lse, torch.ones(20, device="cuda"))
    assert torch.isnan(dX[[4, 9]]).all() and int(torch.isnan(dX).any(1).sum()) == 2


def test_cross_entropy_large_logits():
    X, W, y, _ = ce_inputs(50, 64, 300, 9)
    ce_check((X.float() * 100).bfloat16(), W, y, torch.ones(50, device="cuda"))


def test_cross_entropy_weights_of_many_sizes():
    X, W, y, g = ce_inputs(64, 64, 300, 10)
    d = torch.randn(64, generator=g, device="cuda") * torch.exp2(torch.randint(-30, 20, (64,), generator=g, device="cuda").float())
    d[5] = 0.0
    ce_check(X, W, y, d)
    ce_check(X, W, y, torch.zeros(64, device="cuda"))


def test_cross_entropy_pitched_inputs_and_one_gradient():
    X, W, y, _ = ce_inputs(45, 96, 333, 11)
    d = torch.rand(45, device="cuda")
    loss, lse = tj2.linear_ce_fwd(X, W, y)
    dX, dW = tj2.linear_ce_bwd(X, W, y, lse, d)
    Xp = torch.full((45, 120), NAN, device="cuda", dtype=torch.bfloat16)
    Wp = torch.full((333, 104), NAN, device="cuda", dtype=torch.bfloat16)
    Xp[:, 8:104] = X
    Wp[:, :96] = W
    xs, ws = Xp[:, 8:104], Wp[:, :96]
    l2, e2 = tj2.linear_ce_fwd(xs, ws, y)
    assert torch.equal(l2, loss) and torch.equal(e2, lse)
    for need in ((True, True), (True, False), (False, True)):
        a, b = tj2.linear_ce_bwd(xs, ws, y, e2, d, need_dx=need[0], need_dw=need[1])
        assert (a is None) != need[0] and (b is None) != need[1]
        assert a is None or torch.equal(a, dX)
        assert b is None or torch.equal(b, dW)


def test_cross_entropy_autograd_matches_calls():
    X, W, y, _ = ce_inputs(30, 64, 200, 12)
    x, w = X.clone().requires_grad_(), W.clone().requires_grad_()
    out = tj2.linear_cross_entropy(x, w, y)
    out.backward()
    loss, lse = tj2.linear_ce_fwd(X, W, y)
    n = (y != -100).sum()
    assert torch.equal(out.detach(), loss.sum() / n)
    dX, dW = tj2.linear_ce_bwd(X, W, y, lse, torch.full((30,), 1.0, device="cuda") / n)
    assert torch.equal(x.grad, dX) and torch.equal(w.grad, dW)
    x2 = X.clone().requires_grad_()
    tj2.linear_cross_entropy(x2, W, y, reduction="sum").backward()
    assert W.grad is None and x2.grad is not None


def test_cross_entropy_stream_graph_and_repeat():
    X, W, y, _ = ce_inputs(77, 128, 1111, 13)
    d = torch.rand(77, device="cuda")

    def both(x):
        loss, lse = tj2.linear_ce_fwd(x, W, y)
        return (loss, *tj2.linear_ce_bwd(x, W, y, lse, d))
    want = both(X)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = both(X)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    static, graph = X.clone(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both(static)
    for k in (1, 2, 3):
        static.copy_((X.float() * k).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, both(static.clone())))


def test_cross_entropy_ignored_rows_enter_no_gradient():
    for T in (40, 2100):  # rows read as they are, and copied into blocks first
        X, W, y, _ = ce_inputs(T, 64, 500, 7)
        y[3] = y[17] = -100
        d = torch.ones(T, device="cuda")
        d[3] = NAN
        _, lse = tj2.linear_ce_fwd(X, W, y)
        want = tj2.linear_ce_bwd(X, W, y, lse, torch.ones(T, device="cuda"))
        X[3], X[17] = NAN, INF
        _, lse = tj2.linear_ce_fwd(X, W, y)
        got = tj2.linear_ce_bwd(X, W, y, lse, d)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert (got[0][3] == 0).all() and torch.isfinite(got[1]).all()


@pytest.mark.parametrize("T", [15, 16, 17, 31, 33, 48, 63, 64, 65, 127])
@pytest.mark.parametrize("K", [16, 208, 1040])
def test_cross_entropy_few_tokens(T, K):
    X, W, y, g = ce_inputs(T, K, 515, T * K)
    ce_check(X, W, y, torch.randn(T, generator=g, device="cuda"))


@pytest.mark.parametrize("T,K,V", [(1, 1024, 5000), (15, 16, 270001), (16, 1040, 4099), (17, 208, 24001), (33, 528, 8001),
                                   (48, 80, 60000), (64, 1040, 4100), (64, 2064, 33003), (65, 1040, 4099), (96, 256, 17001),
                                   (127, 528, 9000), (128, 1024, 4097), (129, 1024, 4097)])
def test_cross_entropy_few_tokens_large_heads(T, K, V):
    """Few tokens and a head of 2^22 elements and more: dX from W as it lies, also with rows apart and by itself."""
    X, W, y, g = ce_inputs(T, K, V, T * K, ignored=0.2)
    Wp = torch.full((V, K + 8), NAN, device="cuda", dtype=torch.bfloat16)
    Wp[:, :K] = W
    d = torch.randn(T, generator=g, device="cuda")
    for w in (W, Wp[:, :K]):
        _, lse, dX, dW = ce_check(X, w, y, d)
        assert torch.equal(dX, tj2.linear_ce_bwd(X, w, y, lse, d, need_dw=False)[0])
    ce_check(X, W, y, d, dx_dtype=torch.float32, dw_dtype=torch.float32)


@pytest.mark.parametrize("T,K,V,ldx,ldw", [(2047, 80, 700, 88, 96), (2048, 80, 700, 80, 160), (2049, 144, 513, 152, 144),
                                           (30, 80, 700, 96, 88)])
def test_cross_entropy_pitched_with_and_without_blocks(T, K, V, ldx, ldw):
    X, W, y, _ = ce_inputs(T, K, V, 21)
    Xp = torch.full((T, ldx), NAN, device="cuda", dtype=torch.bfloat16)
    Wp = torch.full((V, ldw), NAN, device="cuda", dtype=torch.bfloat16)
    Xp[:, :K], Wp[:, :K] = X, W
    d = torch.full((T,), 1.0 / T, device="cuda")
    ce_check(Xp[:, :K], Wp[:, :K], y, d)


@pytest.mark.parametrize("T,K,V", [(16384, 32, 16400), (60000, 32, 4400), (2500, 608, 6000), (1024, 272, 20001)])
def test_cross_entropy_last_piece_and_large_tiles(T, K, V):
    X, W, y, g = ce_inputs(T, K, V, 22)
    ce_check(X, W, y, torch.rand(T, generator=g, device="cuda"))


@pytest.mark.parametrize("T,K,V", [(16384, 48, 20000), (200, 1024, 9000), (9000, 80, 33001)])
def test_cross_entropy_one_gradient_of_several_pieces(T, K, V):
    """Each gradient by itself is the one of both: the same dz, summed in an order of its own."""
    X, W, y, g = ce_inputs(T, K, V, 51)
    d = torch.rand(T, generator=g, device="cuda") / T
    _, lse = tj2.linear_ce_fwd(X, W, y)
    opt = dict(dx_dtype=torch.float32, dw_dtype=torch.float32)
    both = tj2.linear_ce_bwd(X, W, y, lse, d, **opt)
    dX, none = tj2.linear_ce_bwd(X, W, y, lse, d, need_dw=False, **opt)
    assert none is None
    none, dW = tj2.linear_ce_bwd(X, W, y, lse, d, need_dx=False, **opt)
    assert none is None
    # two fp32 sums of the same n products, each within n + 64 half steps of the sum of magnitudes; |dz| <= d (p + 1 at
    # the target), of which bf16 takes half a step
    z = X.double() @ W.double().T
    c = torch.where(y == -100, 0.0, d.double())
    dz = torch.exp(z - lse.double()[:, None]).mul_(c[:, None])
    dz[torch.arange(T, device="cuda"), y.clamp(min=0)] += c
    dz *= 1 + 2 * H8
    assert ((dX - both[0]).double().abs() <= 2 * (V + 64) * H24 * (dz @ W.double().abs()) + 2.0 ** -130).all()
    assert ((dW - both[1]).double().abs() <= 2 * (T + 64) * H24 * (dz.T @ X.double().abs()) + 2.0 ** -130).all()


def test_cross_entropy_graphs_share_a_workspace():
    """Two captured backward passes with one workspace, replayed in turns among eager calls that use it too."""
    cases = []
    ws = None
    for seed, (T, K, V) in ((31, (300, 96, 2000)), (32, (2100, 64, 900))):
        X, W, y, _ = ce_inputs(T, K, V, seed)
        d = torch.full((T,), 1.0 / T, device="cuda")
        n = int(tj2.lib().tj2_linear_ce_bwd_workspace_size(T, K, V))
        ws = torch.empty(n, dtype=torch.uint8, device="cuda") if ws is None or ws.numel() < n else ws
        cases.append((X, W, y, tj2.linear_ce_fwd(X, W, y)[1], d))
    want = [tj2.linear_ce_bwd(*c) for c in cases]
    graphs, held = [], []
    for c in cases:
        g = torch.cuda.CUDAGraph()
        dX, dW = torch.empty_like(c[0]), torch.empty_like(c[1])
        with torch.cuda.graph(g):
            tj2.linear_ce_bwd(*c, dX=dX, dW=dW, workspace=ws)
        graphs.append(g)
        held.append((dX, dW))
    for k in (0, 1, 0, 0, 1):
        for t in held[k]:
            t.fill_(NAN)
        graphs[k].replay()
        other = tj2.linear_ce_bwd(*cases[1 - k], workspace=ws)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held[k], want[k]))
        assert all(torch.equal(a, b) for a, b in zip(other, want[1 - k]))


def test_cross_entropy_on_two_streams_at_once():
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    data, want, got = [], [], [[], []]
    for seed, (T, K, V) in ((41, (700, 128, 3001)), (42, (60, 512, 9000))):
        X, W, y, _ = ce_inputs(T, K, V, seed)
        data.append((X, W, y, torch.full((T,), 0.5, device="cuda")))

    def both(X, W, y, d):
        loss, lse = tj2.linear_ce_fwd(X, W, y)
        return (loss, *tj2.linear_ce_bwd(X, W, y, lse, d))
    for c in data:
        want.append(both(*c))
    torch.cuda.synchronize()
    for _ in range(4):
        for i, s in enumerate(sides):
            with torch.cuda.stream(s):
                got[i].append(both(*data[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


# ---- distillation ----------------------------------------------------------------------------------------------
def distill_inputs(T, V, k, dtype, seed, pitch=None):
    g = gen(seed)
    z = torch.randn(T, pitch or V, generator=g, device="cuda") * 3
    ids = torch.stack([torch.randperm(V, generator=g, device="cuda")[:k] for _ in range(T)])
    if k > V:
        ids = torch.randint(0, V, (T, k), generator=g, device="cuda")
    u = torch.randn(T, k, generator=g, device="cuda") * 2 + 5
    drop = torch.rand(T, k, generator=g, device="cuda") < 0.2
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    y[torch.rand(T, generator=g, device="cuda") < 0.1] = -100
    w = torch.randn(T, generator=g, device="cuda")
    return z.to(dtype)[:, :V], torch.where(drop, -1, ids).int(), u.to(dtype), y, w


def distill_ref(z, ids, u, tau, alpha, y, w, ignore=-100):
    z, u, ids, w = z.double(), u.double(), ids.long(), w.double()
    T, V = z.shape
    on = torch.ones(T, dtype=torch.bool, device="cuda") if y is None else y != ignore
    valid = ids >= 0
    has = (valid & (u > -INF)).any(1)
    p = torch.softmax(torch.where(valid, u / tau, -INF), 1)
    p = torch.where(valid & has[:, None], p, 0.0)
    at = ids.clamp(min=0)
    lq = torch.log_softmax(z / tau, 1)
    kl = torch.where(p > 0, p * (torch.log(p.clamp(min=1e-300)) - lq.gather(1, at)), 0.0).sum(1)
    loss = alpha * tau * tau * kl
    dz = alpha * tau * (lq.exp() * has[:, None])
    mag = dz.clone().scatter_add_(1, at, alpha * tau * p)  # the magnitudes that are subtracted
    dz.scatter_add_(1, at, -alpha * tau * p)
    if alpha != 1.0:
        l1 = torch.log_softmax(z, 1)
        pick = torch.where(on, y, 0)
        loss = loss - (1 - alpha) * l1.gather(1, pick[:, None])[:, 0]
        h = l1.exp()
        mag = mag + (1 - alpha) * h
        mag.scatter_add_(1, pick[:, None], torch.full((T, 1), 1 - alpha, device="cuda", dtype=torch.float64))
        h.scatter_add_(1, pick[:, None], -torch.ones(T, 1, device="cuda", dtype=torch.float64))
        dz = dz + (1 - alpha) * h
    return torch.where(on, loss, 0.0), torch.where(on[:, None], dz * w[:, None], 0.0), on, \
        torch.where(on[:, None], mag * w.abs()[:, None], 0.0)


def distill_check(z, ids, u, tau, alpha, y, w, **kw):
    loss, dz = tj2.distill_topk(z, ids, u, temperature=tau, alpha=alpha, targets=y, weight=w, grad=True, **kw)
    rl, rd, on, mag = distill_ref(z, ids, u, tau, alpha, y, w)
    # fp32: logarithms and exponents of arguments up to A, their differences and V / 512-term sums in lanes
    # (a logit of -inf has probability 0 exactly)
    A = torch.where(on, z.double().abs().nan_to_num(posinf=0.0).amax(1), 0.0) + 40 + u.double().nan_to_num(neginf=0.0).abs().amax(1)
    lim = 64 * H24 * A * max(1.0, tau) * (1 + tau)
    assert ((loss.double() - rl).abs() <= lim).all(), float(((loss.double() - rl).abs() / lim).max())
    half = H8 if z.dtype == torch.bfloat16 else H24
    # each probability within 16 half steps of fp32 times its argument (at most A); the result is rounded once, and
    # what fp32 or bf16 exponentials lose below their range is far under 2^-100
    lim = mag * 16 * H24 * A[:, None] + rd.abs() * half + 2.0 ** -100 * (1 + w.double().abs()[:, None])
    err = (dz.double() - rd).abs()
    assert (err <= lim).all(), float((err / lim).max())
    return loss, dz


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,V,k", [(1, 1, 1), (3, 7, 5), (5, 33, 33), (9, 1001, 50), (4, 4096, 512), (7, 16384, 1), (6, 32003, 64),
                                   (3, 50304, 64), (2, 90001, 17)])
@pytest.mark.parametrize("tau,alpha", [(1.0, 1.0), (2.0, 0.5), (4.0, 0.0)])
def test_distill(dtype, T, V, k, tau, alpha):
    distill_check(*distill_inputs(T, V, k, dtype, T + V + k)[:3], tau, alpha, *distill_inputs(T, V, k, dtype, T + V + k)[3:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V,pitch", [(1000, 1001), (1001, 1003), (40000, 40001), (200000, 200003)])
def test_distill_pitches_in_place_and_misaligned_output(dtype, V, pitch):
    z, ids, u, y, w = distill_inputs(5, V, 20, dtype, V, pitch)
    loss, dz = distill_check(z, ids, u, 2.0, 0.3, y, w)
    out = torch.full((5, V + 7), 9.0, device="cuda", dtype=dtype)
    _, d2 = tj2.distill_topk(z, ids, u, temperature=2.0, alpha=0.3, targets=y, weight=w, dlogits=out[:, 5:5 + V])
    assert torch.equal(d2, dz) and (out[:, :5] == 9).all() and (out[:, 5 + V:] == 9).all()
    buf = z.clone() if pitch == V else torch.empty_strided(z.shape, z.stride(), dtype=dtype, device="cuda").copy_(z)
    l3, d3 = tj2.distill_topk(buf, ids, u, temperature=2.0, alpha=0.3, targets=y, weight=w, dlogits=buf)
    assert d3 is buf and torch.equal(d3, dz) and torch.equal(l3, loss)


def test_distill_special_rows():
    z, ids, u, y, w = distill_inputs(12, 300, 8, torch.float32, 1)
    y[:] = 5
    ids[0] = -1                              # the teacher kept nothing
    u[1] = -INF                              # and here gives nothing any weight
    ids[2] = ids[2, 0].abs()                 # one entry, listed again and again
    ids[3, 1] = ids[3, 0] = 17               # twice
    ids[4, 0] = 5                            # the hard target is among the teacher's
    z[5, 100:200] = -INF                     # masked logits that nobody names
    ids[5] = torch.arange(8, device="cuda", dtype=torch.int32)
    u[6, 3] = -INF                           # one kept entry without weight
    z[7] = NAN
    y[7] = -100                              # ignored, so whatever it holds
    z[8, 7] = 1e30                           # one logit takes everything
    ids[8] = torch.tensor([7, -1, -1, -1, -1, -1, -1, -1], device="cuda", dtype=torch.int32)
    w[9] = 0.0
    for alpha in (1.0, 0.5):
        keep = [0, 1, 2, 3, 4, 5, 6, 7, 9, 10, 11]
        loss, dz = distill_check(z[keep].contiguous(), ids[keep].contiguous(), u[keep].contiguous(), 2.0, alpha, y[keep], w[keep])
        assert (dz[7] == 0).all() and loss[7] == 0 and (dz[8] == 0).all()
        l8, d8 = tj2.distill_topk(z[8:9], ids[8:9], u[8:9], temperature=2.0, alpha=1.0, weight=w[8:9], grad=True)
        assert l8[0] == 0 and (d8 == 0).all()
    loss, dz = tj2.distill_topk(z[:2], ids[:2], u[:2], temperature=2.0, grad=True)
    assert (loss == 0).all() and (dz == 0).all()


def test_distill_what_gives_nan():
    z, ids, u, y, w = distill_inputs(6, 100, 4, torch.bfloat16, 2)
    ids[:] = torch.arange(4, device="cuda", dtype=torch.int32)
    y[:] = 3
    z[0, 50] = NAN
    ids[1, 2] = 100
    y[2] = 100
    u[3, 1] = NAN
    loss, dz = tj2.distill_topk(z, ids, u, alpha=0.5, targets=y, weight=w, grad=True)
    assert torch.isnan(loss[:4]).all() and torch.isnan(dz[:4]).any(1).all() and torch.isfinite(dz[4:]).all()
    loss = tj2.distill_topk(z, ids, u, targets=y)  # alpha 1: the hard target is not used
    assert torch.isfinite(loss[2])
    z[4, 1] = -INF                                 # the teacher believes in what the student has ruled out
    loss, dz = tj2.distill_topk(z, ids, u, grad=True)
    assert loss[4] == INF and torch.isfinite(dz[4]).all()


def test_distill_only_hard_target_is_cross_entropy():
    z, ids, u, y, w = distill_inputs(20, 777, 3, torch.float32, 3)
    ids[:] = -1
    loss = tj2.distill_topk(z, ids, u, alpha=0.0, targets=y)
    want = torch.nn.functional.cross_entropy(z.double(), y, reduction="none", ignore_index=-100)
    assert ((loss.double() - want).abs() <= 64 * H24 * 40).all()


def test_distill_gradient_against_differences():
    z, ids, u, y, w = distill_inputs(4, 60, 6, torch.float32, 4)
    _, dz = tj2.distill_topk(z, ids, u, temperature=1.5, alpha=0.6, targets=y, weight=w, grad=True)
    g, h = gen(5), 1e-6
    v = torch.randn(z.shape, generator=g, device="cuda", dtype=torch.float64)

    def total(zz):
        return (distill_ref(zz, ids, u, 1.5, 0.6, y, w)[0] * w.double()).sum()
    diff = (total(z.double() + h * v) - total(z.double() - h * v)) / (2 * h)
    assert abs(float((dz.double() * v).sum() - diff)) <= 1e-5 * float(v.abs().sum())


def test_distill_autograd_stream_and_graph():
    z, ids, u, y, w = distill_inputs(31, 2003, 10, torch.bfloat16, 6)
    a = z.clone().requires_grad_()
    out = tj2.distillation_loss(a, ids, u, temperature=2.0, alpha=0.7, targets=y)
    out.backward()
    n = (y != -100).sum()
    loss, dz = tj2.distill_topk(z, ids, u, temperature=2.0, alpha=0.7, targets=y, weight=torch.ones(31, device="cuda") / n, grad=True)
    assert torch.equal(out.detach(), loss.sum() / n) and torch.equal(a.grad, dz)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        l2 = tj2.distill_topk(z, ids, u, temperature=2.0, alpha=0.7, targets=y)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(l2, loss)
    static, graph = z.clone(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = tj2.distill_topk(static, ids, u, weight=w, grad=True)
    for k in (1, 2, 3):
        static.copy_(z * k)
        graph.replay()
        torch.cuda.synchronize()
        want = tj2.distill_topk(static.clone(), ids, u, weight=w, grad=True)
        assert all(torch.equal(p, q) for p, q in zip(held, want))
