"""MXFP4 operands on the host: their arrays are views of one allocation, and one that a caller puts in their place is
what the entry points get (CPU)."""
import pytest
import torch

import bit_fully_quantized_amd as tj2


def fresh():
    return tj2.QTensor(tj2.MXFP4, 3, 200, device="cpu")


def pointers(q):
    c = q.c()
    return c.codes, c.scale16


def test_untouched():
    q = fresh()
    at = q.buffer.data_ptr()
    assert pointers(q) == (at, at + 3 * 2 * 64)
    assert pointers(q) == (q.codes.data_ptr(), q.scale16.data_ptr())  # also once they were looked at
    assert q.codes.shape == (3, 128) and q.scale16.shape == (3, 8) and q.storage() is q.codes


@pytest.mark.parametrize("name", ["codes", "scale16"])
def test_one_array_replaced(name):
    q, other = fresh(), fresh()
    new = torch.zeros(3, 128 if name == "codes" else 8, dtype=torch.uint8)
    setattr(q, name, new)
    codes, scale = pointers(q)
    assert codes == (new if name == "codes" else q.codes).data_ptr()
    assert scale == (new if name == "scale16" else q.scale16).data_ptr()
    assert getattr(q, "scale16" if name == "codes" else "codes").untyped_storage().data_ptr() == q.buffer.data_ptr()
    other.codes = torch.ones(3, 128, dtype=torch.uint8)
    other.scale16 = torch.ones(3, 8, dtype=torch.uint8)
    assert pointers(other) == (other.codes.data_ptr(), other.scale16.data_ptr())


def test_regrouping_into_its_own_arrays_is_refused():
    import ctypes
    from bit_fully_quantized_amd import _lib
    L = _lib.lib()

    def run(codes, scales):
        x, out = _lib.QTensorC(0x10000, 0x20000, 0, 64, 64, _lib.MXFP4, 0), _lib.QTensorC(codes, scales, 0, 64, 64, _lib.MXFP4, 0)
        return L.mxfp4_quantize(None, _lib.MXFP4, ctypes.byref(x), 64, 64, 1, 0, 0, 0, 0, 0, ctypes.byref(out), None)
    for codes, scales in ((0x10000, 0x20000), (0x10000, 0x30000), (0x30000, 0x20000)):
        assert run(codes, scales) == _lib.TJ2_ERR_ARG and b"x_q" in L.tj2_last_error()
