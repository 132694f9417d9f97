"""Oracle of the 4-bit pool format: E2M1 codes with an E4M3 scale for every
block of 16 dims.

TEST INFRASTRUCTURE ONLY (see the package docstring).

E2M1 (OCP microscaling formats): s ee m, bias 1: the non-negative values are
0, 0.5, 1, 1.5, 2, 3, 4, 6.  Quantising a block of 16 consecutive dims of an
fp16 row under the pool's scale S, every step rounded to fp32:
    y     = x * fp32(1 / S)
    scale = E4M3(max|y| * fp32(1 / 6))       (oracle.fp8's encoder)
    code  = E2M1(y * fp32(1 / scale)), nearest, ties to the even code,
            beyond 6 it is 6; 0 where scale is 0
and a code reads back as code * scale * S.
"""
from __future__ import annotations

import numpy as np

from . import fp8

BLOCK = 16
VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def nearest_e2m1(y) -> np.ndarray:
    """The E2M1 value of each float64 ``y`` (signed, zeros lose their sign)."""
    y = np.asarray(y, dtype=np.float64)
    a = np.abs(y)[..., None]
    d = np.abs(a - VALUES)
    best = d.min(-1, keepdims=True)
    # of two equally near values the one with the even code
    near = (d == best)
    idx = np.where(near, np.arange(8) + 8 * (np.arange(8) % 2), 99).min(-1) % 8
    return np.sign(y) * VALUES[idx]


def quantize(x, S: float) -> tuple[np.ndarray, np.ndarray]:
    """(code values [..., D], block scales [..., D / 16]) of fp16 rows."""
    x32 = np.asarray(x, dtype=np.float16).astype(np.float32)
    y = (x32 * fp8.inverse_scale(S)).reshape(*x32.shape[:-1], x32.shape[-1] // BLOCK, BLOCK)
    top = np.abs(y).max(-1)
    scale = fp8.decode(fp8.encode(top * (np.float32(1) / np.float32(6))))
    with np.errstate(divide="ignore"):
        inv = np.where(scale > 0, np.float32(1) / scale.astype(np.float32), np.float32(0)).astype(np.float32)
    z = y * inv[..., None]
    assert z.dtype == np.float32
    return nearest_e2m1(z).reshape(x32.shape), scale


def dequantize(codes, scale, S: float) -> np.ndarray:
    """The elements attention sees, float64."""
    return stored(codes, scale) * float(np.float32(S))


def stored(codes, scale) -> np.ndarray:
    """The same in units of S (exact in fp16)."""
    return codes * np.repeat(scale, BLOCK, axis=-1)


def roundtrip(x, S: float) -> np.ndarray:
    return dequantize(*quantize(x, S), S)
