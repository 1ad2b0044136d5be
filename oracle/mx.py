"""Caches of 4-bit numbers (oracle).  TEST INFRASTRUCTURE ONLY.

Each 32 elements of a row share a power of two, and an element is the code of
the value nearest to it among the eight magnitudes of E2M1; plain definitions
in float64, by trying all magnitudes.
"""
from __future__ import annotations

import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = 32


def scale_exponents(x) -> np.ndarray:
    """x [..., D] -> e [..., D / 32] with scale 2^e; a block that is not finite
    as float32 gives 128 (byte 255)."""
    x = np.asarray(x, np.float64)
    blocks = x.reshape(x.shape[:-1] + (-1, BLOCK))
    out = np.zeros(blocks.shape[:-1], np.int64)
    with np.errstate(over="ignore"):
        finite = np.isfinite(blocks.astype(np.float32)).all(-1)
    for at in np.ndindex(out.shape):
        a = float(np.abs(blocks[at]).max()) if finite[at] else 0.0
        e = -125
        while e < 125 and a >= 7.0 * 2.0 ** e:     # from 7 units on the next power holds the largest as 4
            e += 1
        out[at] = e if finite[at] else 128
    return out


def pack(x):
    """x [..., D] -> codes [..., D / 2] and scale bytes [..., D / 32], uint8."""
    x = np.asarray(x, np.float64)
    e = scale_exponents(x)
    bad = np.repeat(e == 128, BLOCK, axis=-1)
    y = np.where(bad, 0.0, x) / 2.0 ** np.repeat(np.where(e == 128, 0, e), BLOCK, axis=-1)
    far = np.abs(np.abs(y)[..., None] - MAGNITUDES)
    least = far.min(-1, keepdims=True)
    near = far == least                            # two of them for a tie
    even = np.arange(8) % 2 == 0
    code = np.where(near.sum(-1) == 2, np.argmax(near & even, axis=-1), np.argmax(near, axis=-1))
    code = np.where(bad, 0, code + 8 * np.signbit(np.where(bad, 0.0, x))).astype(np.uint8)
    return (code[..., 0::2] | code[..., 1::2] << 4).astype(np.uint8), (e + 127).astype(np.uint8)


def unpack(codes, scales) -> np.ndarray:
    """The values in float64, NaN where the scale byte is above 252."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    out = np.empty(codes.shape[:-1] + (2 * codes.shape[-1],))
    for half, c in ((0, codes & 15), (1, codes >> 4)):
        out[..., half::2] = np.where(c & 8, -1.0, 1.0) * MAGNITUDES[c & 7]
    s = np.where(scales > 252, np.nan, 2.0 ** (np.maximum(scales, 1).astype(np.float64) - 127))
    return out * np.repeat(s, BLOCK, axis=-1)


def border_distance(x) -> np.ndarray:
    """How far each element is, relative to it, from where its code or its
    block's scale would change (infinite for zeros)."""
    x = np.asarray(x, np.float64)
    e = np.repeat(scale_exponents(x), BLOCK, axis=-1)
    size = np.abs(x) / 2.0 ** np.where(e == 128, 0, e)
    middles = (MAGNITUDES[1:] + MAGNITUDES[:-1]) / 2
    with np.errstate(divide="ignore", invalid="ignore"):
        own = (np.abs(size[..., None] - middles) / size[..., None]).min(-1)
        top = size.reshape(size.shape[:-1] + (-1, BLOCK)).max(-1)
        both = np.minimum(np.abs(top - 3.5), np.abs(top - 7.0)) / top
    own = np.where(size == 0, np.inf, own)
    both = np.where(top == 0, np.inf, both)
    return np.minimum(own, np.repeat(both, BLOCK, axis=-1))
