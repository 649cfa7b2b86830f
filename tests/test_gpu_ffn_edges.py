"""Feed-forward block: what is not finite in the weights, gradients as autograd hands them over, and what is kept."""
import pytest
import torch

from test_gpu_ffn import ACTS, BF, make, normal

pytestmark = pytest.mark.gpu

tj2 = pytest.importorskip("bit_fully_quantized_amd")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T", [1, 20, 150, 2100])
def test_a_nan_gate_has_nan_gradients(T, act):
    """A NaN in a row of Wg makes its feature's gates NaN: so are the slopes there, dWg's, dWu's and dWd's parts of that
    feature, and no others."""
    D, F, f = 144, 208, 37
    X, Wg, Wu, Wd = make(T, D, F)
    dY = normal((T, D), 9, 1e-2)
    _, saved = tj2.gated_ffn_fwd(X, Wg, Wu, Wd, activation=act, save=True)
    clean = tj2.gated_ffn_bwd(dY, X, Wg, Wu, Wd, saved, activation=act)
    bad = Wg.clone()
    bad[f, 11] = float("nan")
    Y, saved = tj2.gated_ffn_fwd(X, bad, Wu, Wd, activation=act, save=True)
    assert torch.isnan(Y.float()).all()
    dX, dWg, dWu, dWd = tj2.gated_ffn_bwd(dY, X, bad, Wu, Wd, saved, activation=act)
    assert torch.isnan(dX.float()).all() and torch.isnan(dWg[f].float()).all() and torch.isnan(dWu[f].float()).all()
    assert torch.isnan(dWd[:, f].float()).all()
    keep = torch.arange(F, device="cuda") != f
    assert torch.equal(dWg[keep], clean[1][keep]) and torch.equal(dWu[keep], clean[2][keep]) and torch.equal(dWd[:, keep], clean[3][:, keep])


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 40])
def test_an_infinite_weight_makes_its_results_infinite(T):
    """Wd with an infinity: what it meets of H is neither 0 nor infinite, so Y there is an infinity of H's sign (also
    where H is kept in two parts, the second of which may be 0 or of the other sign)."""
    D, F = 64, 208
    X, Wg, Wu, Wd = make(T, D, F)
    Y = tj2.gated_ffn_fwd(X, Wg, Wu, Wd)[0]
    g, u = X.double() @ Wg.double().T, X.double() @ Wu.double().T
    h = g * torch.sigmoid(g) * u
    assert (h.abs() > 1e-6).all()
    bad = Wd.clone()
    for d in range(0, D, 2):
        bad[d, 3 * d + 1] = float("inf") if d % 4 else float("-inf")
    got = tj2.gated_ffn_fwd(X, Wg, Wu, bad)[0]
    for d in range(D):
        if d % 2:
            assert torch.equal(got[:, d], Y[:, d])
        else:
            assert (got[:, d].double() == bad[d, 3 * d + 1].double() * h[:, 3 * d + 1].sign()).all(), d


def test_gradients_at_any_address():
    """A gradient that autograd hands over as a view into a longer tensor starts at any of its elements."""
    leaves = [t.requires_grad_() for t in make(33, 48, 80)]
    c = normal((33 * 48,), 9, 1.0, torch.float32)
    want = torch.autograd.grad((tj2.gated_ffn(*leaves).flatten().float() * c).sum(), leaves)
    for before in (1, 3, 8):
        first = torch.zeros(before, dtype=BF, device="cuda")
        y = torch.cat((first, tj2.gated_ffn(*leaves).flatten()))
        got = torch.autograd.grad((y * torch.cat((first, c.to(BF)))).sum(), leaves)
        again = torch.autograd.grad((tj2.gated_ffn(*leaves).flatten() * c.to(BF)).sum(), leaves)
        assert all(torch.equal(a, b) for a, b in zip(got, again))
        assert all(a.shape == b.shape for a, b in zip(got, want))


def test_gates_are_kept_for_a_backward_pass_only(monkeypatch):
    """Where no gradients are recorded the forward writes no gates and factors, whatever the leaves ask for."""
    from bit_fully_quantized_amd import ffn
    kept, run = [], ffn.gated_ffn_fwd

    def look(*a, **kw):
        out = run(*a, **kw)
        kept.append(out[1] is not None)
        return out
    monkeypatch.setattr(ffn, "gated_ffn_fwd", look)
    leaves = [t.requires_grad_() for t in make(5, 48, 80)]
    Y = tj2.gated_ffn(*leaves)
    with torch.no_grad():
        assert torch.equal(tj2.gated_ffn(*leaves), Y)
    with torch.inference_mode():
        assert torch.equal(tj2.gated_ffn(*leaves), Y)
    assert torch.equal(tj2.gated_ffn(*(t.detach() for t in leaves)), Y)
    assert kept == [True, False, False, False]
    torch.autograd.grad(Y.float().sum(), leaves)
