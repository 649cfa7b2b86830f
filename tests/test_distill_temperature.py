"""Temperatures whose square or reciprocal leaves fp32 are refused on the host (CPU)."""
import ctypes

import pytest


@pytest.mark.parametrize("tau,ok", [(2.0 ** -64, True), (1.0, True), (2.0 ** 63, True), (2.0 ** -65, False), (1e-39, False),
                                    (2.0 ** 64, False), (1e38, False), (0.0, False), (float("nan"), False)])
def test_range(tau, ok):
    from bit_fully_quantized_amd import _lib
    L = _lib.lib()
    # (a target array missing at alpha below 1 is what the call is refused for after its temperature is accepted)
    got = L.tj2_distill_topk(0x1000, _lib.F32, 3, 101, 101, 0x2000, 0x3000, 4, ctypes.c_float(tau), ctypes.c_float(0.5), None, -100,
                             None, 0x4000, 0x5000, 101, None)
    assert got == _lib.TJ2_ERR_ARG
    assert (b"targets" in L.tj2_last_error()) == ok and (b"temperature" in L.tj2_last_error()) != ok
