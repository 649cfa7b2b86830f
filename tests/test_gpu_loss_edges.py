"""The head's losses on the GPU where a mask or a bad entry decides."""
import pytest
import torch

pytestmark = pytest.mark.gpu

tj2 = pytest.importorskip("bit_fully_quantized_amd")

from test_gpu_losses import H8, H24, INF, NAN, ce_check, ce_inputs, distill_inputs  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("T", [1, 5, 16, 33, 64, 65, 300])
def test_cross_entropy_masked_vocabulary(T):
    """Entries with logits of -inf (a mask's bias of -inf against a constant feature) have probability 0."""
    K, V = 128, 1100
    X, W, y, g = ce_inputs(T, K, V, T, ignored=0.0)
    masked = torch.zeros(V, dtype=torch.bool, device="cuda")
    masked[100:104] = masked[209] = masked[300:700] = masked[1030:] = True
    y %= 100
    X[:, 0] = 1.0
    W[masked, 0] = -INF
    loss, lse = tj2.linear_ce_fwd(X, W, y)
    x, w = X.double(), W[~masked].double()
    z = x @ w.T
    rlse = torch.logsumexp(z, 1)
    rows = torch.arange(T, device="cuda")
    place = (~masked).cumsum(0)[y] - 1
    # as for unmasked heads: K + 16 half steps of a logit's sum of magnitudes, 16 of the arguments of exp2 and log2
    ez = (K + 16) * H24 * (x.abs() @ w.abs().T).amax(1)
    tol = 2 * ez + 16 * H24 * (2 * z.abs().amax(1) + rlse.abs() + 1)
    assert ((lse.double() - rlse).abs() <= tol).all()
    assert ((loss.double() - (rlse - z[rows, place])).abs() <= 2 * tol).all()
    dX, dW = tj2.linear_ce_bwd(X, W, y, lse, torch.ones(T, device="cuda"), dw_dtype=torch.float32, dx_dtype=torch.float32)
    assert (dW[masked] == 0).all() and torch.isfinite(dW).all()
    p = torch.exp(z - rlse[:, None])
    dz = p.clone()
    dz[rows, place] -= 1
    # p off by its exponent's error, dz by half a bf16 step more; sums of fp32
    edz = p * (ez + tol + 16 * H24 * (1 + z.abs().amax(1)))[:, None] + dz.abs() * H8 + 2.0 ** -126
    n = T + 64
    assert ((dW[~masked].double() - dz.T @ x).abs() <= edz.T @ x.abs() + n * H24 * (dz.abs().T @ x.abs())).all()
    # (feature 0 is 0 times -inf there, as in a product with the logits kept)
    err = (dX.double() - dz @ w).abs()[:, 1:]
    assert (err <= (edz @ w.abs() + (V + 64) * H24 * (dz.abs() @ w.abs()))[:, 1:]).all()


@pytest.mark.parametrize("T", [5, 64, 65, 2100])
def test_cross_entropy_token_with_no_entry_left(T):
    """A token whose logits are all -inf: lse -inf, loss and gradients NaN, as of a softmax of them; others are as they were."""
    X, W, y, _ = ce_inputs(T, 64, 500, T, ignored=0.0)
    X[:, 0] = 0.0
    W[:, 0] = -3e38
    d = torch.ones(T, device="cuda")
    loss, lse = tj2.linear_ce_fwd(X, W, y)
    dX, _ = tj2.linear_ce_bwd(X, W, y, lse, d)
    Xm = X.clone()
    Xm[2] = 0.0
    Xm[2, 0] = 2.0  # 2 * -3e38: -inf in fp32
    loss2, lse2 = tj2.linear_ce_fwd(Xm, W, y)
    dX2, dW2 = tj2.linear_ce_bwd(Xm, W, y, lse2, d)
    keep = torch.arange(T, device="cuda") != 2
    assert lse2[2] == -INF and torch.isnan(loss2[2])
    assert torch.equal(loss[keep], loss2[keep]) and torch.equal(lse[keep], lse2[keep])
    assert torch.isnan(dX2[2]).all() and torch.equal(dX2[keep], dX[keep]) and torch.isnan(dW2).all()
    y[2] = -100  # left out, it enters nothing
    loss2, lse2 = tj2.linear_ce_fwd(Xm, W, y)
    dX2, dW2 = tj2.linear_ce_bwd(Xm, W, y, lse2, d)
    assert loss2[2] == 0 and (dX2[2] == 0).all() and torch.isfinite(dW2).all() and torch.equal(dX2[keep], dX[keep])


@pytest.mark.parametrize("T,K,V", [(65, 48, 800000), (130, 144, 400001), (1100, 272, 90001), (2047, 80, 60000), (2048, 80, 60001),
                                   (5000, 208, 30011), (4100, 1040, 24001)])
def test_cross_entropy_pieces_of_every_layout(T, K, V):
    """Vocabularies taken in several pieces with and without blocked copies, split and unsplit, W also with rows apart."""
    # dz twice and the copies of W, of all entries, are more than a piece's share of the workspace
    up = lambda n, m: -(-n // m) * m  # noqa: E731
    assert 2 * (up(T, 128) + up(T, 64) + up(K, 128) + (up(K, 64) if T >= 2048 else 0)) * V > max(3 << 27, T * V)
    X, W, y, g = ce_inputs(T, K, V, T + K, ignored=0.05)
    d = torch.rand(T, generator=g, device="cuda") - 0.3
    _, lse, dX, dW = ce_check(X, W, y, d)
    Wp = torch.full((V, K + 8), float("nan"), device="cuda", dtype=torch.bfloat16)
    Wp[:, :K] = W
    got = tj2.linear_ce_bwd(X, Wp[:, :K], y, lse, d)
    assert torch.equal(got[0], dX) and torch.equal(got[1], dW)


@pytest.mark.parametrize("T,K,V", [(1100, 272, 90001), (2300, 528, 50001)])
def test_cross_entropy_pieces_in_a_graph(T, K, V):
    """A captured backward of several pieces, replayed among eager calls that share its workspace."""
    X, W, y, g = ce_inputs(T, K, V, T, ignored=0.05)
    d = torch.rand(T, generator=g, device="cuda") / T
    _, lse = tj2.linear_ce_fwd(X, W, y)
    want = tj2.linear_ce_bwd(X, W, y, lse, d)
    ws = torch.empty(int(tj2.lib().tj2_linear_ce_bwd_workspace_size(T, K, V)), dtype=torch.uint8, device="cuda")
    dX, dW = torch.empty_like(X), torch.empty_like(W)
    graph, weights = torch.cuda.CUDAGraph(), d.clone()
    with torch.cuda.graph(graph):
        tj2.linear_ce_bwd(X, W, y, lse, weights, dX=dX, dW=dW, workspace=ws)
    for k in (1, 2, 3):
        dX.fill_(float("nan"))
        dW.fill_(float("nan"))
        weights.copy_(d * 2.0 ** k)  # dz is over the largest weight: a power of two scales the results exactly
        graph.replay()
        other = tj2.linear_ce_bwd(X, W, y, lse, d, workspace=ws, need_dw=False)[0]
        torch.cuda.synchronize()
        assert torch.equal(dX, want[0] * 2.0 ** k) and torch.equal(dW, want[1] * 2.0 ** k)
        # (dX by itself may be summed in an order of its own: two fp32 sums, each rounded once)
        assert float((other - want[0]).float().norm() / want[0].float().norm()) <= H8


# ---- distillation ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("alpha", [1.0, 0.5, 0.0])
def test_distill_id_outside_is_nan(alpha):
    """An id of V or more makes its token NaN, whatever the weight of the teacher's term; an ignored token stays 0."""
    z, ids, u, y, w = distill_inputs(6, 100, 4, F32, 2)
    ids[:] = torch.arange(4, device="cuda", dtype=torch.int32)
    y[:] = 3
    ids[1, 2] = 100
    ids[4, 0] = 2 ** 31 - 1
    ids[5, 1] = 100
    y[5] = -100
    loss, dz = tj2.distill_topk(z, ids, u, alpha=alpha, targets=y, weight=w, grad=True)
    bad = torch.tensor([False, True, False, False, True, False], device="cuda")
    assert torch.equal(torch.isnan(loss), bad) and torch.equal(torch.isnan(dz).any(1), bad)
    assert torch.isnan(dz[bad]).all() and loss[5] == 0 and (dz[5] == 0).all()


def test_distill_teacher_without_weight_enters_nothing():
    """alpha 0: whatever the teacher's logits are, infinities and NaN too."""
    z, ids, u, y, w = distill_inputs(9, 200, 5, F32, 12)
    opt = dict(alpha=0.0, targets=y, weight=w, grad=True)
    loss, dz = tj2.distill_topk(z, ids, u, **opt)
    u[0], u[1, 2], u[2, 0], u[3] = NAN, NAN, INF, -INF
    got = tj2.distill_topk(z, ids, u, **opt)
    assert torch.isfinite(loss).all() and torch.equal(got[0], loss) and torch.equal(got[1], dz)


def test_distillation_notices_targets_changed_before_the_backward():
    z, ids, u, y, _ = distill_inputs(8, 60, 4, F32, 11)
    a = z.clone().requires_grad_()
    out = tj2.distillation_loss(a, ids, u, alpha=0.5, targets=y)
    y.fill_(1)
    with pytest.raises(RuntimeError, match="inplace"):
        out.backward()
