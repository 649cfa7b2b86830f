"""The decoder stack on FP8 linears, with the library's norms and feed-forward block: the operators together, as training
calls them, each checked where it stands in the step."""
import math

import numpy as np
import pytest
import torch
import torch.nn.functional as F

from oracle import formats

import _helpers as H
import test_gpu_fp8 as T8

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


def grid(x, tr, tc):
    codes, S = T8.ref_tiles(x, tr, tc)
    v = formats.e4m3_decode(codes).astype(np.float64)
    return v * np.repeat(np.repeat(S.astype(np.float64), tr, 0), tc, 1)[: v.shape[0], : v.shape[1]]


@pytest.mark.parametrize("linear,head,norm,mlp", [("fp8", "linear", "torch", "linear"), ("fp8", "linear", "fused", "linear"),
                                                  ("fp8", "fused", "fused", "fused"), ("fp8", "linear", "fused", "fused"),
                                                  ("nvfp4", "fused", "fused", "fused"), ("mxfp4", "linear", "fused", "linear"),
                                                  ("bf16", "fused", "fused", "fused"), ("bf16", "linear", "torch", "fused")])
def test_step_of_every_kind(linear, head, norm, mlp):
    cfg, stack = make(linear=linear, head=head, norm=norm, mlp=mlp)
    tokens, targets = decoder.random_tokens(cfg, 0)
    targets[1, -7:] = -100  # a padded sequence
    lins = {L.name: L for L in stack.linears}
    names = [n for n in ("0.qkv", "0.up", "1.o", "1.down", "head") if lins[n].kind == "fp8"]
    for n in names:
        lins[n].capture = {}
    before = {L.name: L.W.clone() for L in stack.linears}
    norms = [t for b in stack.blocks for t in (b["attn_norm"], b["mlp_norm"])] + [stack.final_norm]
    seen = {}

    def look(st):
        seen["norms"] = [t.grad.clone() for t in norms]
    loss = float(stack.train_step(tokens, targets, before_update=look))
    assert abs(loss - math.log(cfg.vocab)) < 0.2  # random weights
    for L in stack.linears:
        assert torch.isfinite(L.grad).all() and float(L.grad.abs().max()) > 0, L.name
        assert torch.isfinite(L.W).all() and not torch.equal(L.W, before[L.name]), L.name
        if L.kind == "fused":
            assert torch.equal(L.Wg, L.W.bfloat16())
        if L.kind == "fp8":
            q = tj2.fp8_quantize(L.W, block=True)
            assert torch.equal(L.Wq.codes, q.codes) and torch.equal(L.Wq.scale128, q.scale128)  # the updated master's
    for g in seen["norms"]:
        assert torch.isfinite(g).all() and float(g.abs().max()) > 0
    for n in names:
        c = lins[n].capture
        X, W, dY = c["X"].double().cpu().numpy(), grid(c["W"].cpu().numpy(), 128, 128), c["dY"].float().cpu().numpy()
        # fp32 sums, then half a bf16 step of each element (dW stays fp32)
        assert H.rel_fro(c["Y"].float().cpu().numpy(), X @ W.T) <= H8, n
        assert H.rel_fro(c["dX"].float().cpu().numpy(), grid(dY, 1, 128) @ W) <= H8, n
        ref = grid(dY.T.copy(), 1, 128) @ grid(c["X"].cpu().numpy().T.copy(), 1, 128).T
        assert H.rel_fro(c["dW"].cpu().numpy(), ref) <= (len(X) + 16) * H24 * 4, n


def losses_and_gradients(cfg_kw, seed=0):
    cfg, stack = make(**cfg_kw)
    grads = {}

    def look(st):
        for L in st.linears:
            grads[L.name] = L.grad.double().clone()
        for i, b in enumerate(st.blocks):
            grads[f"{i}.attn_norm"], grads[f"{i}.mlp_norm"] = b["attn_norm"].grad.double().clone(), b["mlp_norm"].grad.double().clone()
        grads["final_norm"], grads["emb"] = st.final_norm.grad.double().clone(), st.emb.grad.double().clone()
    tokens, targets = decoder.random_tokens(cfg, seed)
    return float(stack.train_step(tokens, targets, before_update=look)), grads


@pytest.mark.parametrize("kw", [dict(norm="fused"), dict(mlp="fused"), dict(norm="fused", mlp="fused")])
def test_the_bf16_stack_takes_the_same_step(kw):
    """Loss and every gradient of the bf16 stack, with torch's glue and with the library's: roundings to bf16 in other
    places (the feed-forward block's gates, factors and gradients, the norms' gradients), a handful of half steps each
    way per layer, of the norm."""
    a, ga = losses_and_gradients(dict(linear="bf16"))
    b, gb = losses_and_gradients(dict(linear="bf16", **kw))
    assert abs(a - b) <= 4 * H8
    for n in ga:
        assert float((ga[n] - gb[n]).norm() / ga[n].norm()) <= 12 * H8, n


def test_the_fp8_stack_with_either_norm():
    """The norm's own FP8 operand differs from the codes of its bf16 result by that rounding: where the two straddle a
    border of E4M3 an element moves by a step of it (2^-3), which of 2^-8 / 2^-3 of the elements it does."""
    a, ga = losses_and_gradients(dict(linear="fp8"))
    b, gb = losses_and_gradients(dict(linear="fp8", norm="fused"))
    assert abs(a - b) <= 2.0 ** -5
    for n in ga:
        assert float((ga[n] - gb[n]).norm() / ga[n].norm()) <= 2.0 ** -2, n


def test_single_tokens_and_repeats():
    cfg, stack = make(linear="fp8", head="fused", norm="fused", mlp="fused")
    tokens, targets = decoder.random_tokens(cfg, 3)
    with torch.no_grad():
        for B, S in ((1, 1), (1, 5), (2, 8), (1, 33)):
            h = stack.hidden(tokens[:B, :S].contiguous())
            z = h.double() @ stack.head.Wg.double().T
            got = float(stack.loss(tokens[:B, :S].contiguous(), targets[:B, :S].contiguous()))
            ref = float(F.cross_entropy(z, targets[:B, :S].reshape(-1)))
            mag = float((h.double().abs() @ stack.head.Wg.double().abs().T).max())
            assert abs(got - ref) <= H24 * (cfg.d_model * mag * 2 + 64 * 2 * np.log(cfg.vocab)), (got, ref)
    runs = []
    for _ in range(2):
        cfg, stack = make(linear="fp8", head="fused", norm="fused", mlp="fused")
        loss = stack.train_step(*decoder.random_tokens(cfg, 0))
        runs.append((loss, *(L.grad for L in stack.linears), *(b["mlp_norm"] for b in stack.blocks)))
    for a, b in zip(*runs):
        assert torch.equal(a, b)
