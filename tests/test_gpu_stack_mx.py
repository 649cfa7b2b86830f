"""The decoder stack on MXFP4 linears, with the head's cross entropy taken without the logits and with a teacher's
top logits: the operators together, as training calls them, each checked where it stands in the step."""
import numpy as np
import pytest
import torch
import torch.nn.functional as F

from oracle import mx

import _helpers as H

pytestmark = pytest.mark.gpu

tj2 = pytest.importorskip("bit_fully_quantized_amd")
from bit_fully_quantized_amd import decoder  # noqa: E402

H24, H8 = 2.0 ** -24, 2.0 ** -8
SMALL = dict(vocab=1008, d_model=128, layers=2, heads=2, ffn=320, seq=48, batch=2, lr_start=1e-3, total_steps=10)


def make(**kw):
    cfg = decoder.DecoderConfig(**{**SMALL, **kw})
    torch.manual_seed(0)
    stack = decoder.Decoder(cfg)
    stack.calibrate([decoder.random_tokens(cfg, 100)[0]])
    return cfg, stack


def teacher_of(cfg, k, seed=5):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    ids = torch.rand(cfg.batch, cfg.seq, cfg.vocab, generator=g, device="cuda").topk(k).indices.int()
    ids[0, 0, k // 2:] = -1  # a token whose teacher kept fewer
    return ids, torch.randn(cfg.batch, cfg.seq, k, generator=g, device="cuda").bfloat16()


def plain_loss(z, targets, teacher, cfg):
    """Mean loss of fp64 logits [T, V]."""
    y = targets.reshape(-1)
    on = y != -100
    ce = F.cross_entropy(z, y, reduction="none")
    if teacher is None:
        return ce[on].mean()
    tau, a = cfg.distill_temperature, cfg.distill_alpha
    ids, top = (t.reshape(len(y), -1) for t in teacher)
    lp = torch.log_softmax(top.double().masked_fill(ids < 0, float("-inf")) / tau, 1)
    lq = torch.log_softmax(z / tau, 1).gather(1, ids.clamp(min=0).long())
    kl = torch.where(ids >= 0, lp.exp() * (lp - lq), 0.0).sum(1)
    return (a * tau * tau * kl + (1 - a) * ce)[on].mean()


@pytest.mark.parametrize("linear,head,distil", [("mxfp4", "fused", False), ("mxfp4", "linear", True), ("mxfp4", "linear", False),
                                                ("mxfp4", "fused", True), ("nvfp4", "fused", False), ("nvfp4", "linear", True),
                                                ("bf16", "fused", False)])
def test_step_of_every_kind(linear, head, distil):
    cfg, stack = make(linear=linear, head=head, distill_temperature=2.0, distill_alpha=0.7)
    tokens, targets = decoder.random_tokens(cfg, 0)
    targets[1, -7:] = -100  # a padded sequence
    teacher = teacher_of(cfg, 9) if distil else None
    names = ("0.qkv", "0.up", "1.down") + (("head",) if head == "linear" else ()) if linear == "mxfp4" else ()
    lins = {L.name: L for L in stack.linears}
    for n in names:
        lins[n].capture = {}
    with torch.no_grad():
        h = stack.hidden(tokens)
        z = stack.head(h)
    for n in names:
        lins[n].capture = {}
    seen = {}

    def before(st):
        seen["W"] = st.head.W.clone()
        seen["head"] = st.head.grad.clone()

    loss = float(stack.train_step(tokens, targets, before_update=before, teacher=teacher))
    # the loss from its inputs: without logits from the hidden states and the bf16 weights, else from the logits
    without = head == "fused" and not distil
    W = seen["W"].bfloat16().double()
    ref = float(plain_loss(h.double() @ W.T if without else z.double(), targets, teacher, cfg))
    # a logit is an fp32 sum of d products (d half steps of the sum of magnitudes), the sums of the softmaxes and of
    # the tokens, exponents and logarithms of arguments below 2 log V: 64 half steps of them; tau^2 weighs the first
    mag = float((h.double().abs() @ W.abs().T).max())
    assert abs(loss - ref) <= H24 * (cfg.d_model * mag * 2 + 64 * 2 * np.log(cfg.vocab) * 4), (loss, ref)
    for L in stack.linears:
        assert torch.isfinite(L.grad).all() and float(L.grad.abs().max()) > 0, L.name
        assert torch.isfinite(L.W).all()
    for t in [stack.emb, stack.final_norm]:
        assert torch.isfinite(t).all()
    for n in names:
        c = lins[n].capture
        X, Wm, dY = (c[k].float().cpu().numpy() for k in ("X", "W", "dY"))
        rY, rX, rW = mx.linear(X, Wm, dY, seed=cfg.seed, offset=c["offset"])
        # fp32 sums, then half a bf16 step of each element (dW stays fp32)
        assert H.rel_fro(c["Y"].float().cpu().numpy(), rY) <= H8 + (X.shape[1] + 16) * H24 * 4, n
        assert H.rel_fro(c["dX"].float().cpu().numpy(), rX) <= H8 + (dY.shape[1] + 16) * H24 * 4, n
        assert H.rel_fro(c["dW"].cpu().numpy(), rW) <= (len(X) + 16) * H24 * 4, n
        assert torch.equal(lins[n].Wq.codes, tj2.mx_quantize(lins[n].W).codes)  # the updated master's codes
        assert not torch.equal(lins[n].W, c["W"])
    if head == "fused":
        assert torch.equal(stack.head.Wg, stack.head.W.bfloat16())
        x = h.double()
        z64 = (x @ W.T if without else z.double()).requires_grad_(True)
        dz, = torch.autograd.grad(plain_loss(z64, targets, teacher, cfg), z64)
        # dz rounded to bf16, the result too: one step of bf16 together, of the norm
        assert H.rel_fro(seen["head"].cpu().numpy(), (dz.T @ x).cpu().numpy()) <= 2 * H8


def test_fused_head_takes_the_same_step():
    """The bf16 stack's loss and every gradient, with and without logits, agree to the bf16 logits' rounding."""
    cfg, plain = make(linear="bf16")
    _, fused = make(linear="bf16", head="fused")
    tokens, targets = decoder.random_tokens(cfg, 0)
    grads = [[], []]
    a, b = (float(s.train_step(tokens, targets, before_update=lambda st, g=g: g.extend(L.grad.clone() for L in st.linears)))
            for s, g in zip((plain, fused), grads))
    # the plain path rounds a logit to bf16: half a step of logits below 4 at the most
    assert abs(a - b) <= 4 * H8
    for L, x, y in zip(plain.linears, *grads):
        # dlogits, the hidden gradient and dW are rounded in both, the logits in one: a handful of half steps each way
        assert float((x - y).norm() / x.norm()) <= 8 * H8, L.name


def test_single_tokens_and_scores():
    """One token at a time: the few-row products, and the score without logits."""
    cfg, stack = make(linear="mxfp4", head="fused")
    tokens, targets = decoder.random_tokens(cfg, 3)
    L = stack.linears[0]
    with torch.no_grad():
        for B, S in ((1, 1), (1, 5), (2, 8), (1, 17)):
            t, y = tokens[:B, :S].contiguous(), targets[:B, :S].contiguous()
            L.capture = {}
            h = stack.hidden(t)
            X, W = L.capture["X"].float().cpu().numpy(), L.W.cpu().numpy()
            Y = mx.dequantize(mx.quantize(X)) @ mx.dequantize(mx.quantize(W)).T
            assert H.rel_fro(L.capture["Y"].float().cpu().numpy(), Y) <= H8 + (X.shape[1] + 16) * H24 * 4
            z = h.double() @ stack.head.Wg.double().T
            mag = float((h.double().abs() @ stack.head.Wg.double().abs().T).max())
            got, ref = float(stack.loss(t, y)), float(F.cross_entropy(z, y.reshape(-1)))
            assert abs(got - ref) <= H24 * (cfg.d_model * mag * 2 + 64 * 2 * np.log(cfg.vocab)), (got, ref)


def test_steps_repeat_bit_for_bit():
    """Loss and the head's gradient of a first step (before torch's atomics in the embedding's) are the same each run."""
    runs = []
    for _ in range(2):
        cfg, stack = make(linear="mxfp4", head="fused")
        loss = stack.train_step(*decoder.random_tokens(cfg, 0))
        runs.append((loss, stack.head.grad, stack.linears[-2].grad))
    for a, b in zip(*runs):
        assert torch.equal(a, b)
