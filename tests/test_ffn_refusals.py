"""The feed-forward block's entry points refuse bad arguments on the host, before any device work (CPU)."""
import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from bit_fully_quantized_amd import _lib
    return _lib


def test_entry_points(lib):
    L = lib.lib()
    ARG, SHAPE, ALIGN = lib.TJ2_ERR_ARG, lib.TJ2_ERR_SHAPE, lib.TJ2_ERR_ALIGN
    assert L.tj2_gated_ffn_fwd_workspace_size(0, 64, 64) == 0 and L.tj2_gated_ffn_bwd_workspace_size(5, -1, 64) == 0
    need = L.tj2_gated_ffn_fwd_workspace_size(5, 64, 96)
    assert need >= 5 * 96 * 2

    def fwd(X=0x1000, ldx=64, Wg=0x2000, Wu=0x3000, ldw=64, Wd=0x4000, ldd=96, T=5, D=64, F=96, act=0, gu=None, Y=0x5000, yd=lib.BF16,
            ws=0x10000, n=need):
        return L.tj2_gated_ffn_fwd(X, ldx, Wg, Wu, ldw, Wd, ldd, T, D, F, act, gu, Y, yd, ws, n, None)
    for k in ("X", "Wg", "Wu", "Wd", "Y", "ws"):
        assert fwd(**{k: None}) == ARG, k
    assert fwd(act=3) == ARG and fwd(act=-1) == ARG and fwd(yd=lib.FP8) == ARG and fwd(n=need - 1) == ARG
    assert fwd(T=0) == SHAPE and fwd(D=40) == SHAPE and fwd(F=40) == SHAPE and fwd(F=0) == SHAPE
    assert fwd(ldx=56) == SHAPE and fwd(ldx=68) == SHAPE and fwd(ldw=63) == SHAPE and fwd(ldd=90) == SHAPE
    assert fwd(T=(1 << 21) + 1) == SHAPE and fwd(ldd=1 << 22) == SHAPE and fwd(T=1 << 21, F=1 << 20, ldd=1 << 20) == SHAPE
    for k in ("X", "Wg", "Wu", "Wd", "Y", "ws"):
        assert fwd(**{k: 0x1008}) == ALIGN, k
    assert fwd(gu=0x6004) == ALIGN
    need = L.tj2_gated_ffn_bwd_workspace_size(5, 64, 96)

    def bwd(dY=0x1000, ldy=64, gu=0x6000, dX=0x7000, xd=lib.BF16, dWg=0x8000, dWu=0x9000, dWd=0xA000, wd=lib.F32, ws=0x10000, n=need, T=5):
        return L.tj2_gated_ffn_bwd(dY, ldy, 0x1000, 64, 0x2000, 0x3000, 64, 0x4000, 96, T, 64, 96, 0, gu, dX, xd, dWg, dWu, dWd, wd, ws,
                                   n, None)
    assert bwd(dY=None) == ARG and bwd(gu=None) == ARG and bwd(ws=None) == ARG and bwd(n=need - 1) == ARG
    assert bwd(dX=None, dWg=None, dWu=None, dWd=None) == ARG and bwd(xd=5) == ARG and bwd(wd=5) == ARG
    assert bwd(ldy=60) == SHAPE and bwd(ldy=68) == SHAPE and bwd(T=0) == SHAPE
    for k in ("dY", "gu", "dX", "dWg", "dWu", "dWd", "ws"):
        assert bwd(**{k: 0x1008}) == ALIGN, k


def test_binding():
    import bit_fully_quantized_amd as tj2
    x, w = torch.zeros(2, 16, dtype=torch.bfloat16), torch.zeros(32, 16, dtype=torch.bfloat16)
    for f in (tj2.gated_ffn, tj2.gated_ffn_fwd):
        with pytest.raises(ValueError):
            f(x, w, w, w.t().contiguous())


def test_gradients_are_apart(lib):
    L, need = lib.lib(), lib.lib().tj2_gated_ffn_bwd_workspace_size(5, 64, 64)

    def bwd(dX=0x7000, dWg=0x8000, dWu=0x9000, dWd=0xA000):
        return L.tj2_gated_ffn_bwd(0x1000, 64, 0x1000, 64, 0x2000, 0x3000, 64, 0x4000, 64, 5, 64, 64, 0, 0x6000, dX, lib.F32, dWg, dWu, dWd,
                                   lib.F32, 0x10000, need, None)
    assert bwd(dWu=0x8000) == bwd(dWd=0x8000) == bwd(dWd=0x9000) == bwd(dX=0x8000) == bwd(dX=0xA000) == lib.TJ2_ERR_ARG
