"""Plain NumPy oracle of the MXFP4 weight format (OCP microscaling, 4-bit).

TEST INFRASTRUCTURE ONLY, like the rest of this package.

A row of K values is cut into groups of 32.  Each group has one E8M0 byte s
(scale 2^(s-127), s = 255 NaN), each value one E2M1 code: sign, two exponent
bits (bias 1), one mantissa bit, so 0, 0.5, 1, 1.5, 2, 3, 4, 6.  Two codes share
a byte, the even value in the low four bits.
"""
from __future__ import annotations

import numpy as np

GROUP = 32
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def unpack(codes: np.ndarray) -> np.ndarray:
    """[.., K/2] bytes -> [.., K] 4-bit codes."""
    c = np.asarray(codes, np.uint8)
    return np.stack((c & 15, c >> 4), axis=-1).reshape(*c.shape[:-1], -1)


def decode_e2m1(nibbles: np.ndarray) -> np.ndarray:
    """E2M1 codes (one per element) -> fp64; exponent 0 is subnormal (m/2)."""
    n = np.asarray(nibbles).astype(np.int64)
    ex, man = (n >> 1) & 3, n & 1
    mag = np.where(ex == 0, man * 0.5, (1 + 0.5 * man) * np.exp2(ex - 1.0))
    return np.where(n >> 3, -mag, mag)


def dequant(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """codes [.., K/2], scales [.., K/32] -> values [.., K] fp64."""
    s = np.asarray(scales, np.uint8).astype(np.float64)
    scale = np.where(s == 255, np.nan, np.exp2(s - 127.0))
    return decode_e2m1(unpack(codes)) * np.repeat(scale, GROUP, axis=-1)


def quantize(w: np.ndarray):
    """Values [.., K] (exact in fp64) -> (codes [.., K/2], scales [.., K/32]).

    scale exponent max(floor(log2 amax) - 2, -127); each value to the nearest
    grid point, halfway to the one with an even code, beyond 6 to 6; zeros keep
    their sign.  A group with a non-finite value: s = 255, codes 0."""
    w = np.asarray(w, np.float64)
    g = w.reshape(*w.shape[:-1], -1, GROUP)
    amax = np.abs(g).max(axis=-1)
    bad = ~np.isfinite(amax)
    am = np.where(bad | (amax == 0), 1.0, amax)
    e = np.maximum(np.frexp(am)[1] - 1 - 2, -127)
    e = np.where(amax == 0, -127, e)
    with np.errstate(invalid="ignore"):
        a = np.abs(g) * np.exp2(-e.astype(np.float64))[..., None]
    a = np.where(bad[..., None], 0.0, a)
    d = np.abs(a[..., None] - GRID)  # distance to every grid point
    near = d.min(axis=-1, keepdims=True)
    hit = d == near
    code = hit.argmax(axis=-1)  # the lower of two equally near points
    other = 7 - hit[..., ::-1].argmax(axis=-1)  # the upper one
    code = np.where(code % 2 == 0, code, other)
    code = np.where(a > 6, 7, code)
    code = code | np.where(np.signbit(g) & ~bad[..., None], 8, 0)
    code = code.reshape(w.shape).astype(np.uint8)
    packed = code[..., 0::2] | (code[..., 1::2] << 4)
    return packed.astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)
