"""MXFP4 (microscaled 4-bit) quantizer, oracle; test infrastructure only.

Groups of 32 consecutive elements share one power of two 2^e, stored as the byte
e + 127; elements are E2M1.  The OCP microscaling formats fix the storage and
leave the choice of e to the implementation; the reading taken:

* round to nearest: e = floor(log2 amax) - 2 (their suggested rule: the group's
  largest binade is the element format's), elements above 6 saturate;
* stochastic rounding: the smallest e with amax <= 6 * 2^e, because a
  saturating element would bias the rounding;
* e is not below -127; a group of zeros has byte 0; a group with an infinity or
  NaN has byte 255 (the formats' NaN) and zero codes;
* a Hadamard transform, where asked for, acts on whole 16-element pieces; a
  shorter piece at the end of a row is left as it is.

All arithmetic is in Python's exact integers or fp64 powers of two, where every
step is exact.
"""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np

from . import formats, philox, rht
from .quant import pack_nibbles, unpack_nibbles


@dataclass
class MxTensor:
    codes: np.ndarray  # uint8 [rows, ceil(L / 2)]
    scale: np.ndarray  # uint8 [rows, ceil(L / 32)]
    rows: int
    L: int


def scale_byte(amax: float, rounding: str) -> int:
    """The scale byte of a group with this largest magnitude, by comparing powers of two."""
    if not np.isfinite(amax):
        return 255
    if amax == 0.0:
        return 0
    for e in range(-127, 128):
        if rounding == "rtn" and amax < 8.0 * 2.0 ** e:
            return e + 127
        if rounding == "sr" and amax <= 6.0 * 2.0 ** e:
            return e + 127
    raise AssertionError(amax)


def quantize_rows(y, rounding: str = "rtn", seed: int = 0, offset: int = 0, row_ids=None) -> MxTensor:
    """fp32 y [rows, L] in groups of 32 along its last axis; row_ids: the rows' numbers in the whole tensor (draws)."""
    y = np.asarray(y, dtype=np.float32)
    rows, L = y.shape
    ng = -(-L // 32)
    pad = np.zeros((rows, ng * 32), dtype=np.float32)
    pad[:, :L] = y
    g = pad.reshape(rows, ng, 32)
    amax = np.abs(g).max(axis=2).astype(np.float64)
    amax = np.where(np.isfinite(g).all(axis=2), amax, np.inf)
    uniq, inv = np.unique(amax, return_inverse=True)
    byte = np.array([scale_byte(float(a), rounding) for a in uniq], dtype=np.uint8)[inv].reshape(rows, ng)
    bad = byte == 255
    v = np.where(bad[:, :, None], 0.0, g).astype(np.float64) * np.ldexp(1.0, 127 - np.where(bad, 127, byte).astype(int))[:, :, None]
    v = np.clip(v, -6.0, 6.0).astype(np.float32).reshape(rows, ng * 32)
    if rounding == "rtn":
        q = formats.e2m1_rtn(v)
    else:
        ids = np.arange(rows, dtype=np.uint64) if row_ids is None else np.asarray(row_ids, dtype=np.uint64)
        e = ids[:, None] * np.uint64(ng * 32) + np.arange(ng * 32, dtype=np.uint64)[None, :]
        q = formats.e2m1_sr(v, philox.sr_draws_u16(e, seed, offset))
    q = np.where(np.repeat(bad, 32, axis=1), 0, q).astype(np.uint8)
    keep = (L + 1) // 2 * 2
    q[:, L:] = 0
    return MxTensor(pack_nibbles(q[:, :keep]), byte, rows, L)


def transform(y, mask):
    """The Hadamard transform of whole 16-element pieces along the last axis."""
    y = np.asarray(y, dtype=np.float32)
    n = y.shape[1] // 16 * 16
    out = y.copy()
    if n:
        out[:, :n] = rht.rht_along_last(y[:, :n], mask)
    return out


def quantize(x, *, grouping: str = "row", rounding: str = "rtn", rht_mask=None, seed: int = 0, offset: int = 0) -> MxTensor:
    y = np.asarray(x, dtype=np.float32)
    if grouping == "col":
        y = np.ascontiguousarray(y.T)
    if rht_mask is not None:
        y = transform(y, rht_mask)
    return quantize_rows(y, rounding, seed, offset)


def dequantize(q: MxTensor) -> np.ndarray:
    """fp64 values [rows, L]; a group with the NaN scale is NaN."""
    v = formats.e2m1_decode(unpack_nibbles(q.codes))[:, : q.L].astype(np.float64)
    s = np.where(q.scale == 255, np.nan, np.ldexp(1.0, q.scale.astype(int) - 127))
    return v * np.repeat(s, 32, axis=1)[:, : q.L]


def linear(X, W, dY, *, rounding: str = "sr", rht: bool = True, seed: int = 0, offset: int = 0):
    """Forward and backward of the linear layer in fp64 on the quantized operands: (Y, dX, dW)."""
    xq, wq = quantize(X), quantize(W)
    xh, wh = dequantize(xq), dequantize(wq)
    sx = philox.rht_signs(seed, offset) if rht else None
    sw = philox.rht_signs(seed, offset + 2) if rht else None
    opt = dict(rounding=rounding, seed=seed)
    dyq = dequantize(quantize(dY, rht_mask=sx, offset=offset, **opt))
    wt = dequantize(quantize(wh, grouping="col", rht_mask=sx, offset=offset + 1, **opt))
    dyt = dequantize(quantize(dY, grouping="col", rht_mask=sw, offset=offset + 2, **opt))
    xt = dequantize(quantize(xh, grouping="col", rht_mask=sw, offset=offset + 3, **opt))
    return xh @ wh.T, dyq @ wt.T, dyt @ xt.T
