"""fp64 oracle for the microscaled 4-bit operators: block quantisation, the packed layout, and
the products and gated block on quantised operands.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Source: the vampireachao.github.io page lists FP4 among Megatron Core's mixed precisions and gives
no recipe. Readings:
  * elements e2m1, +-{0, 0.5, 1, 1.5, 2, 3, 4, 6}, nearest with ties to even, saturating;
  * "mxfp4" (OCP Microscaling Formats 1.0): blocks of 32, scale 2^e, e = floor(log2 amax) - 2,
    at least -127; "nvfp4": blocks of 16, scale e4m3(amax / (6 f)), factor f of the tensor;
  * a block that holds an infinity or a NaN has the scale NaN and zero codes.
Blocks run along the last axis. x is taken as given (fp32 or bf16 values, exact in float64).
"""
from __future__ import annotations

import numpy as np

from .fp8 import e4m3_round

BLOCK = {"mxfp4": 32, "nvfp4": 16}
LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _up(n, m):
    return -(-n // m) * m


def e2m1_round(v):
    """(code 0..7 of the magnitude) nearest level by distance; a tie goes to the even code."""
    # (beyond 8 the distances may round alike; all of it saturates)
    a = np.minimum(np.abs(np.asarray(v, np.float64)), 8.0)[..., None]
    d = np.abs(a - LEVELS)
    best = d.min(-1, keepdims=True)
    near = d == best
    even = near & (np.arange(8) % 2 == 0)
    pick = np.where(even.any(-1, keepdims=True), even, near)
    return np.argmax(pick, -1)


def tensor_factor(x):
    """f = 2^ceil(log2(amax / 2688)) over the finite entries, at least 2^-126; 1 for zeros."""
    x = np.asarray(x, np.float64)
    amax = float(np.max(np.abs(x[np.isfinite(x)]), initial=0.0))
    if amax == 0:
        return amax, 1.0
    e = -126
    while 2688.0 * 2.0 ** e < amax:
        e += 1
    return amax, 2.0 ** e


def quantize(x, fmt, f=1.0):
    """x [rows, cols] -> (codes [rows, ld] 0..15, scale bytes [rows, ld / block], values
    [rows, cols] in float64), ld = cols rounded up to 128."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    n, ld = BLOCK[fmt], _up(cols, 128)
    b = np.zeros((rows, ld))
    b[:, :cols] = x
    b = b.reshape(rows, ld // n, n)
    bad = ~np.isfinite(b).all(-1)
    z = np.where(bad[..., None], 0.0, b)
    amax = np.abs(z).max(-1)
    if fmt == "mxfp4":
        e = np.where(amax > 0, np.frexp(amax)[1] - 1 - 2, -127)
        e = np.maximum(e, -127)
        scale, byte = np.ldexp(1.0, e), e + 127
        byte = np.where(bad, 255, byte)
    else:
        s = e4m3_round(np.minimum(amax / (6 * f), 448.0))
        fr, ex = np.frexp(np.where(s > 0, s, 1.0))  # s = fr 2^ex, 0.5 <= fr < 1
        normal = s >= 2.0 ** -6
        byte = np.where(normal, (ex - 1 + 7) * 8 + np.round((2 * fr - 1) * 8), np.round(s * 512))
        byte = np.where(bad, 0x7F, byte)
        scale = s * f
    q = np.where(scale[..., None] > 0, z / np.where(scale > 0, scale, 1.0)[..., None], 0.0)
    level = np.where(bad[..., None], 0, e2m1_round(q))
    neg = np.signbit(z) & ~bad[..., None] & (scale[..., None] > 0)
    codes = level + 8 * neg
    value = np.where(neg, -LEVELS[level], LEVELS[level]) * scale[..., None]
    value = np.where(bad[..., None], np.nan, value)
    return (codes.reshape(rows, ld).astype(np.uint8), byte.astype(np.uint8),
            value.reshape(rows, ld)[:, :cols])


def values(x, fmt, f=1.0):
    return quantize(x, fmt, f)[2]


def pack(codes, byte):
    """(packed codes [rows, ld / 2], scale tiles as [tiles of rows * 128, blocks] row-major bytes
    in the order of the layout, int16 with -1 where nothing is written)."""
    rows, nb = byte.shape
    packed = codes[:, 0::2] | (codes[:, 1::2] << 4)
    tiles = np.full((_up(rows, 128) // 128, nb // 4, 512), -1, np.int16)
    for r in range(rows):
        for b in range(nb):
            tiles[r // 128, b // 4, 16 * (r % 32) + 4 * (r % 128 // 32) + b % 4] = byte[r, b]
    return packed, tiles.reshape(-1)


def act(z, name):
    """Activation and derivative."""
    from scipy.special import erfc
    z = np.asarray(z, np.float64)
    if name == "silu":
        s = 1 / (1 + np.exp(-z))
        return z * s, s * (1 + z * (1 - s))
    if name == "gelu":
        c = 0.5 * erfc(-z / np.sqrt(2))
        return z * c, c + z * np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
    # (1 + tanh y) / 2 = 1 / (1 + e^-2y): 1 + tanh y is zero in 64 bits from y = -19 on, the value is not
    w = 2 * np.sqrt(2 / np.pi)
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-w * (z + 0.044715 * z ** 3)))
    return z * s, s * (1 + z * (1 - s) * w * (1 + 3 * 0.044715 * z * z))


def gated_bwd(da, g, u, name):
    h, dh = act(g, name)
    da, u = np.asarray(da, np.float64), np.asarray(u, np.float64)
    return da * u * dh, da * h, h * u
