"""The losses' entry points refuse bad arguments on the host, before any device work (CPU)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from bit_fully_quantized_amd import _lib
    return _lib


def test_cross_entropy(lib):
    L = lib.lib()
    ARG, SHAPE, ALIGN = lib.TJ2_ERR_ARG, lib.TJ2_ERR_SHAPE, lib.TJ2_ERR_ALIGN
    need = L.tj2_linear_ce_fwd_workspace_size(5, 64, 300)
    assert need > 0 and L.tj2_linear_ce_fwd_workspace_size(0, 64, 300) == 0

    def fwd(X=0x1000, ldx=64, W=0x2000, ldw=64, y=0x3000, T=5, K=64, V=300, loss=0x4000, lse=0x5000, ws=0x10000, n=need):
        return L.tj2_linear_ce_fwd(X, ldx, W, ldw, y, T, K, V, -100, loss, lse, ws, n, None)
    assert fwd(X=None) == ARG and fwd(W=None) == ARG and fwd(y=None) == ARG and fwd(lse=None) == ARG and fwd(ws=None) == ARG
    assert fwd(n=need - 1) == ARG and b"needed" in L.tj2_last_error()
    assert fwd(T=0) == SHAPE and fwd(V=0) == SHAPE and fwd(K=40) == SHAPE and fwd(K=0) == SHAPE
    assert fwd(ldx=63) == SHAPE and fwd(ldx=68) == SHAPE and fwd(ldw=60) == SHAPE
    assert fwd(T=(1 << 21) + 1) == SHAPE and fwd(V=(1 << 21) + 1) == SHAPE and fwd(ldw=1 << 22) == SHAPE
    assert fwd(T=1 << 21, V=1 << 20) == SHAPE
    assert fwd(X=0x1002) == ALIGN and fwd(W=0x2008) == ALIGN and fwd(y=0x3004) == ALIGN and fwd(ws=0x10008) == ALIGN
    assert fwd(lse=0x5002) == ALIGN and fwd(loss=0x4001) == ALIGN

    need = L.tj2_linear_ce_bwd_workspace_size(5, 64, 300)

    def bwd(lse=0x5000, dl=0x6000, dX=0x7000, xd=lib.BF16, dW=0x8000, wd=lib.BF16, ws=0x10000, n=need, T=5):
        return L.tj2_linear_ce_bwd(0x1000, 64, 0x2000, 64, 0x3000, T, 64, 300, -100, lse, dl, dX, xd, dW, wd, ws, n, None)
    assert bwd(lse=None) == ARG and bwd(dl=None) == ARG and bwd(dX=None, dW=None) == ARG and bwd(ws=None) == ARG
    assert bwd(xd=7) == ARG and bwd(wd=lib.MXFP4) == ARG and bwd(n=need - 1) == ARG
    assert bwd(dX=0x7008) == ALIGN and bwd(dW=0x8004) == ALIGN and bwd(dl=0x6002) == ALIGN
    assert bwd(T=-1) == SHAPE


def test_distillation(lib):
    L = lib.lib()
    ARG, SHAPE, ALIGN = lib.TJ2_ERR_ARG, lib.TJ2_ERR_SHAPE, lib.TJ2_ERR_ALIGN

    def run(z=0x1000, dt=lib.F32, T=3, V=101, ldl=101, ids=0x2000, u=0x3000, k=4, tau=1.0, alpha=1.0, y=None, w=None,
            loss=0x4000, dz=0x5000, ldd=101):
        return L.tj2_distill_topk(z, dt, T, V, ldl, ids, u, k, ctypes.c_float(tau), ctypes.c_float(alpha), y, -100, w, loss, dz,
                                  ldd, None)
    assert run(z=None) == ARG and run(ids=None) == ARG and run(u=None) == ARG and run(loss=None, dz=None) == ARG
    assert run(dt=lib.NVFP4) == ARG
    assert run(T=0) == SHAPE and run(V=0) == SHAPE and run(k=0) == SHAPE and run(k=513) == SHAPE
    assert run(ldl=100) == SHAPE and run(ldd=100) == SHAPE and run(dz=0x1000, ldd=102) == SHAPE
    assert run(T=(1 << 22) + 1) == SHAPE
    for tau in (0.0, -1.0, float("inf"), float("nan")):
        assert run(tau=tau) == ARG
    for alpha in (-0.1, 1.1, float("nan")):
        assert run(alpha=alpha, y=0x6000) == ARG
    assert run(alpha=0.5) == ARG  # targets missing
    assert run(z=0x1002) == ALIGN and run(dt=lib.BF16, z=0x1001) == ALIGN and run(ids=0x2002) == ALIGN
    assert run(y=0x6004) == ALIGN and run(w=0x6002) == ALIGN and run(loss=0x4002) == ALIGN and run(dz=0x5002) == ALIGN


def test_binding_refuses_host_tensors():
    import bit_fully_quantized_amd as tj2
    X, W, y = torch.zeros(2, 16, dtype=torch.bfloat16), torch.zeros(5, 16, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError):
        tj2.linear_ce_fwd(X, W, y)
    with pytest.raises(ValueError):
        tj2.distill_topk(torch.zeros(2, 5), torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1))
    with pytest.raises(ValueError):
        tj2.linear_cross_entropy(X, W, y, reduction="median")
    with pytest.raises(ValueError):
        tj2.distillation_loss(X, y, X, reduction="median")
