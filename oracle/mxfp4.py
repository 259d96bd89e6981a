"""MXFP4 blocks (OCP microscaling: 32 E2M1 codes and one E8M0 scale byte), from the definition, and
the pool tiles that hold them.  NumPy, fp64; shares nothing with the CUDA path.

A scale byte e stands for 2^(e - 127), 255 for NaN.  An E2M1 code is a sign bit, two exponent bits
(bias 1) and one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6.
"""

from __future__ import annotations

import numpy as np


def e2m1_value(code: int) -> float:
    exp, man = (code >> 1) & 3, code & 1
    v = 0.5 * man if exp == 0 else (1 + 0.5 * man) * 2.0 ** (exp - 1)
    return -v if code & 8 else v


VALUES = np.array([e2m1_value(c) for c in range(16)])


def encode(x: np.ndarray):
    """x [..., D] (values of bf16 numbers) -> (codes uint8 [..., D], scale bytes [..., D / 32])."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(x.shape[:-1] + (x.shape[-1] // 32, 32))
    amax = np.abs(b).max(-1)
    nan = np.isnan(amax)
    # floor(log2 amax): frexp's exponent less one; infinity counts as 2^128, zero as the smallest
    e = np.frexp(np.where(np.isfinite(amax), amax, 0.0))[1] - 1
    e = np.where(np.isinf(amax), 128, np.where(amax == 0, -1000, e)) - 2
    byte = np.clip(e, -127, None) + 127
    with np.errstate(invalid="ignore", over="ignore"):
        y = np.abs(b) * np.exp2(127.0 - byte)[..., None]
    # nearest magnitude; a tie goes to the even code
    mags = VALUES[:8]
    mid = (mags[1:] + mags[:-1]) / 2
    y = np.where(np.isnan(y), 0.0, y)
    code = np.zeros(y.shape, dtype=np.int64)
    for i, m in enumerate(mid):
        code += (y > m) | ((y == m) & (i % 2 == 1))
    code |= np.where(np.signbit(b), 8, 0)
    code = np.where(nan[..., None], 0, code)
    byte = np.where(nan, 255, byte)
    return code.reshape(x.shape).astype(np.uint8), byte.astype(np.uint8)


def decode(codes: np.ndarray, byte: np.ndarray) -> np.ndarray:
    scale = np.where(byte == 255, np.nan, np.exp2(byte.astype(np.float64) - 127))
    return VALUES[codes] * np.repeat(scale, 32, axis=-1)


def pack_tiles(codes: np.ndarray, byte: np.ndarray) -> np.ndarray:
    """codes [NB, H, 16, D], byte [NB, H, 16, D / 32] -> the pool's bytes [NB, H, 17 D / 2]."""
    nb, h, rows, d = codes.shape
    n = d // 32
    out = np.zeros((nb, h, rows, d // 2), dtype=np.uint8)
    for dim in range(d):
        b, g, i = dim // 32, dim % 32 // 4, dim % 4
        at = 2 * (g * n + b) + i // 2
        out[..., at] |= codes[..., dim] << (4 * (i % 2))
    return np.concatenate([out.reshape(nb, h, -1), byte.reshape(nb, h, -1)], axis=-1)


def unpack_tiles(pool: np.ndarray):
    nb, h, tile = pool.shape
    d = tile * 2 // 17
    n = d // 32
    rows = pool[..., :8 * d].reshape(nb, h, 16, d // 2)
    codes = np.zeros((nb, h, 16, d), dtype=np.uint8)
    for dim in range(d):
        b, g, i = dim // 32, dim % 32 // 4, dim % 4
        codes[..., dim] = (rows[..., 2 * (g * n + b) + i // 2] >> (4 * (i % 2))) & 15
    return codes, pool[..., 8 * d:].reshape(nb, h, 16, n)
