"""The workspaces of the head's cross entropy: bounded however many logits there are (CPU)."""
import pytest


def up(n, m):
    return -(-n // m) * m


SIZES = [(16384, 1024, 50304), (5000, 1024, 50304), (4096, 1024, 50304), (2047, 1024, 50304), (9000, 512, 20000),
         (16000, 64, 50000), (16384, 1024, 131072), (65536, 4096, 131072), (1024, 4096, 131072), (65, 64, 1 << 21),
         (128, 1024, 1 << 21), (1 << 19, 64, 1 << 21), (1 << 21, 64, 50304), (1235, 528, 32003), (300, 2048, 150000),
         (70, 16, 100), (4097, 16, 1), (2048, 80, 257)]


@pytest.mark.parametrize("T,K,V", SIZES)
def test_backward(T, K, V):
    """Beside the copies of X and the sums of dX: half of bf16 logits, but for 384 MiB that may always be used, never
    above 1 GiB, and 1024 vocabulary entries in any case."""
    from bit_fully_quantized_amd import _lib
    got = _lib.lib().tj2_linear_ce_bwd_workspace_size(T, K, V)
    blocked = T >= 2048
    operands = 2 * (up(T, 128) * up(K, 64) * blocked + up(K, 128) * up(T, 64)) + 4 * T * K + 4 * T + 16 * 256
    least = 1024 * 2 * (up(T, 128) + up(T, 64) + up(K, 128) + up(K, 64) * blocked)
    # (that smallest piece may still have its products split; 32 slices of it and of dX at most)
    least += 32 * 4 * (1024 + T) * K if least > 3 << 27 else 0
    assert 0 < got <= operands + max(min(max(T * V, 3 << 27), 1 << 30), least)
    if T * V >= 1 << 29 and least < T * V:
        assert got - operands <= T * V * 2 / 2  # half of bf16 logits


@pytest.mark.parametrize("K,V", [(1024, 50304), (4096, 131072), (64, 1 << 21), (16, 100)])
def test_backward_of_few_tokens(K, V):
    """Up to 64 tokens take the vocabulary at once: 384 bytes an entry, dX in up to 32 slices, and a turned copy of W
    only where W has fewer than 2^22 elements."""
    from bit_fully_quantized_amd import _lib
    for T in (1, 16, 64):
        got = _lib.lib().tj2_linear_ce_bwd_workspace_size(T, K, V)
        turned = 2 * up(K, 128) * up(V, 256) if K * V < 1 << 22 else 0
        assert 0 < got <= 384 * up(V, 256) + 32 * 4 * T * K + turned + 128 * 2 * up(K, 128) + 4 * T * K + 4 * T + 16 * 256


@pytest.mark.parametrize("T,K,V", SIZES)
def test_forward(T, K, V):
    """One pair of numbers for 64 logits, and copies of X and W from 2048 tokens on."""
    from bit_fully_quantized_amd import _lib
    got = _lib.lib().tj2_linear_ce_fwd_workspace_size(T, K, V)
    copies = 2 * up(K, 64) * (up(T, 128) + up(V, 128)) if T >= 2048 else 0
    assert 0 < got <= max(up(V, 256) // 64, 2048) * T * 8 + copies + 4 * T + 16 * 256
