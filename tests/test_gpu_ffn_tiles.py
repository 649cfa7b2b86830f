"""The feed-forward block at sizes that take its larger tiles, with remainders on every side, all gradients."""
import pytest
import torch

from test_gpu_ffn import BF, Exact, check, make, normal

pytestmark = pytest.mark.gpu

tj2 = pytest.importorskip("bit_fully_quantized_amd")

# Tiles of the projections, of Y, of dH and of the four products after it (splits): 128 (of rows as they lie), 64, 64 and
# 128 (3, 1, 1, 1); 128, 64, 64 and 256 (3, 1, 1, 1); 128 (of blocked operands from here on), 128, 64 and 256; 128, 64 (3),
# 256 and 128 (2 each); 128, 64 (3), 256 and 128 (6, 1, 1, 1); 256 throughout
SIZES = [(1301, 272, 2064), (1301, 1040, 2064), (3001, 2064, 1040), (4099, 272, 2064), (2050, 528, 4112), (4099, 2064, 4112)]


@pytest.mark.parametrize("T,D,F,act", [(*s, "silu") for s in SIZES] + [(*SIZES[0], "gelu"), (*SIZES[3], "gelu"), (*SIZES[3], "gelu_tanh"),
                                                                        (*SIZES[5], "gelu")])
def test_forward_and_backward(T, D, F, act):
    X, Wg, Wu, Wd = make(T, D, F)
    dY = normal((T, D), 9, 1e-2)
    ref = Exact(X, Wg, Wu, Wd, act, dY)
    Y, saved = tj2.gated_ffn_fwd(X, Wg, Wu, Wd, activation=act, save=True)
    check(Y, ref.Y, "Y")
    check(tj2.gated_ffn_fwd(X, Wg, Wu, Wd, activation=act, y_dtype=torch.float32)[0], ref.Y, "Y fp32")
    names = ("dX", "dWg", "dWu", "dWd")
    grads = tj2.gated_ffn_bwd(dY, X, Wg, Wu, Wd, saved, activation=act)
    for g, n in zip(grads, names):
        check(g, getattr(ref, n), n)
    wide = tj2.gated_ffn_bwd(dY, X, Wg, Wu, Wd, saved, activation=act, dx_dtype=torch.float32, dw_dtype=torch.float32)
    for g, h, n in zip(wide, grads, names):
        check(g, getattr(ref, n), n)
        assert torch.equal(g.to(BF), h), n
    for a, b in zip(tj2.gated_ffn_bwd(dY, X, Wg, Wu, Wd, saved, activation=act), grads):
        assert torch.equal(a, b)
    # those of the weights without dX, whose plan is another
    for g, n in zip(tj2.gated_ffn_bwd(dY, X, Wg, Wu, Wd, saved, activation=act, need=(False, True, True, True))[1:], names[1:]):
        check(g, getattr(ref, n), n)
