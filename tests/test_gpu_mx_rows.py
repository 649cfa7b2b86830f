"""MXFP4 linears of few rows on both sides of the reduction's length that decides how they are done."""
import pytest
import torch

pytestmark = pytest.mark.gpu

tj2 = pytest.importorskip("bit_fully_quantized_amd")

from test_gpu_mx import near, values  # noqa: E402


@pytest.mark.parametrize("K", [1024, 2032, 2048, 2064, 4096, 7936, 7952, 16400])
@pytest.mark.parametrize("M,N", [(1, 4096), (7, 16), (16, 528), (17, 1040)])
def test_linear_of_few_rows_and_long_reductions(M, N, K):
    g = torch.Generator(device="cuda").manual_seed(M * N + K)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    w = torch.randn(N, K, generator=g, device="cuda") * 0.02
    Y, saved = tj2.mx_linear_fwd(x, w, N, y_dtype=torch.float32)
    qx, qw = tj2.mx_quantize(x), tj2.mx_quantize(w)
    assert torch.equal(saved["Xq"].codes, qx.codes) and torch.equal(saved["Xq"].scale16, qx.scale16)
    near(Y, values(qx), values(qw))
    near(tj2.mx_linear_fwd(x, None, N, Wq=qw)[0], values(qx), values(qw))
    near(tj2.mx_gemm(qx, qw), values(qx), values(qw))


@pytest.mark.parametrize("M,K,N", [(3, 64, 2048), (3, 64, 2064), (16, 48, 8000), (2048, 32, 16), (2064, 32, 16), (16, 4096, 4112)])
def test_backward_of_few_rows_and_long_reductions(M, K, N):
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    w = torch.randn(N, K, generator=g, device="cuda") * 0.02
    dy = (torch.randn(M, N, generator=g, device="cuda") * 1e-3).bfloat16()
    _, saved = tj2.mx_linear_fwd(x, w, N)
    dX, dW = tj2.mx_linear_bwd(dy, saved, K, seed=0, offset=0, rht=False, rounding=tj2.RTN, dx_dtype=torch.float32)
    col = dict(grouping=tj2.GROUP_COL)
    near(dX, values(tj2.mx_quantize(dy)), values(tj2.mx_quantize(saved["Wq"], **col)))
    near(dW, values(tj2.mx_quantize(dy, **col)), values(tj2.mx_quantize(saved["Xq"], **col)))
