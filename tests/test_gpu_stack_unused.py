"""The decoder stack's norm with the FP8 linears on it, where a loss uses some of the results."""
import pytest
import torch

import test_gpu_stack_fp8 as S

pytestmark = pytest.mark.gpu

tj2 = pytest.importorskip("bit_fully_quantized_amd")
from bit_fully_quantized_amd import decoder  # noqa: E402


@pytest.mark.parametrize("first", [False, True])
def test_results_that_no_loss_uses(first):
    """They count as zero: the other results' gradients are what they are with zeros for them, and a linear that was not
    used has a zero gradient, not the last step's."""
    cfg, stack = S.make(linear="fp8", norm="fused")
    blk, M, d = stack.blocks[0], 96, cfg.d_model
    lins = [blk["gate"], blk["up"]]
    g = torch.Generator(device="cuda")
    g.manual_seed(3)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)
    x, delta, w = normal(M, d).requires_grad_(), normal(M, d).requires_grad_(), blk["mlp_norm"]
    weights = [normal(M, d), normal(M, cfg.ffn), normal(M, cfg.ffn)]
    leaves = [x, w] if first else [x, delta, w]

    def run(used, zeros):
        for L in lins:
            L.grad.fill_(7.0)
        outs = decoder._NormLinearsFn.apply(x, None if first else delta, w, lins, cfg.norm_eps)
        loss = sum((o * c).float().sum() if k in used else (o * 0.0).float().sum()
                   for k, (o, c) in enumerate(zip(outs, weights)) if zeros or k in used)
        return [t if t is None else t.clone() for t in torch.autograd.grad(loss, leaves, allow_unused=True)], [L.grad.clone() for L in lins]
    for used in ((1,), (2,), (0, 1), (0, 2), (1, 2), (0,)):
        got, got_lins = run(used, False)
        want, want_lins = run(used, True)
        for a, b in zip(got, want):
            assert (torch.zeros_like(b) if a is None else a).equal(b), used
        for k, (a, b) in enumerate(zip(got_lins, want_lins)):
            assert torch.equal(a, b) and (k + 1 in used or not a.any()), used
