"""The block operators from their definitions, in numpy and 64 bits.

Shares nothing with the library.  Beside each result the functions return the
magnitude that its rounding errors are relative to, from which the tests derive
their bounds.  Codes of 8 bits are defined by fp32 operations that round once
each, so they are computed in fp32 here too and must be equal bit for bit.
"""
from __future__ import annotations

import numpy as np

TOPS = {"int8": 127.0, "e4m3": 448.0}


def e4m3_numbers():
    """The 256 numbers of e4m3 by their codes (0x7f and 0xff: NaN)."""
    out = np.empty(256)
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        v = np.nan if (e, m) == (15, 7) else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        out[code] = -v if code & 128 else v
    return out


def to_e4m3(x):
    """Codes of the nearest e4m3 numbers (ties to the even code), |x| <= 448."""
    table = e4m3_numbers()[:127]  # the non-negative ones, ascending
    a = np.abs(x)
    up = np.clip(np.searchsorted(table, a), 0, 126)
    down = np.maximum(up - 1, 0)
    near = np.where(table[up] - a < a - table[down], up, down)
    tie = table[up] - a == a - table[down]
    near = np.where(tie, np.where(up % 2 == 0, up, down), near)
    return (near | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def pack(x, fmt, group):
    """(codes as uint8, scales) of an fp32 matrix; one rounding an operation."""
    x = np.asarray(x, dtype=np.float32)
    rows, cols = x.shape
    width = group or max(cols, 1)
    groups = -(-cols // width) if group else 1
    codes, scales = np.zeros((rows, cols), np.uint8), np.zeros((rows, groups), np.float32)
    top = np.float32(TOPS[fmt])
    for g in range(groups):
        part = x[:, g * width:(g + 1) * width]
        if part.shape[1] == 0:
            continue
        bad = ~np.isfinite(part).all(1)
        a = np.abs(np.where(bad[:, None], np.float32(1), part)).max(1)
        none = a < np.float32(2.0 ** -100)
        with np.errstate(divide="ignore", over="ignore"):
            inv = np.where(none, np.float32(0), top / np.where(none, np.float32(1), a)).astype(np.float32)
        scale = np.where(none, np.float32(0), a * (np.float32(1) / top)).astype(np.float32)
        y = (np.where(bad[:, None], np.float32(0), part) * inv[:, None]).astype(np.float32)
        c = np.rint(y).astype(np.int8).view(np.uint8) if fmt == "int8" else to_e4m3(y.astype(np.float64))
        codes[:, g * width:(g + 1) * width] = np.where(bad[:, None], 0, c)
        scales[:, g] = np.where(bad, np.float32(np.nan), scale)
    return codes, scales


def unpack(codes, scales, fmt, group):
    """fp32: RN(code * scale)."""
    v = codes.view(np.int8).astype(np.float32) if fmt == "int8" else e4m3_numbers()[codes].astype(np.float32)
    cols = codes.shape[1]
    return v * np.repeat(scales, group or max(cols, 1), axis=1)[:, :cols]


def norm(x, residual, weight, eps):
    """(h, rstd, out) of float64 arrays."""
    h = x if residual is None else x + residual
    r = 1 / np.sqrt((h * h).mean(1) + eps)
    y = h * r[:, None]
    return h, r, y if weight is None else y * weight


def norm_gradient(dout, h, r, weight, residual_grad, base):
    """((dx, magnitude), (weight gradient, magnitude), again)."""
    n = h * r[:, None]
    g = dout if weight is None else dout * weight
    D = dout.shape[1]
    dx = r[:, None] * (g - n * ((g * n).sum(1, keepdims=True) / D))
    mag = r[:, None] * (np.abs(g) + np.abs(n) * (np.abs(g * n).sum(1, keepdims=True) / D))
    if residual_grad is not None:
        dx, mag = dx + residual_grad, mag + np.abs(residual_grad)
    dw, wmag = (dout * n).sum(0), np.abs(dout * n).sum(0)
    if base is not None:
        dw, wmag = dw + base, wmag + np.abs(base)
    return (dx, mag), (dw, wmag), n if weight is None else n * weight


def value_and_slope(x, kind):
    """(f, its magnitude, f', its magnitude)."""
    if kind == "silu":
        z, dz = x, np.ones_like(x)
    else:
        k = 2 * np.sqrt(2 / np.pi)
        z, dz = k * (x + 0.044715 * x ** 3), k * (1 + 3 * 0.044715 * x ** 2)
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-z))
        rest = 1 / (1 + np.exp(z))  # 1 - s
    along = 1 + rest * np.minimum(np.abs(z), 1e4)  # what an error of z does to s
    # A fast quotient gives 0 where 1 + exp(-z) is above 2^126, so an s of up to 2^-126 may be lost,
    # which takes |x| 2^-126 from f and (1 + |x z'|) 2^-126 from f'; both stand here over the 16 and
    # 32 units of 2^-24 that the tests allow of a magnitude.
    lost = np.where(z < 0, 2.0 ** -126 / 2.0 ** -24, 0.0)
    f, slope = x * s, s + x * s * rest * dz
    return (f, np.abs(f) * along + np.abs(x) * lost / 16,
            slope, s * along + np.abs(f * dz) * (rest + s) * along + (1 + np.abs(x * dz)) * lost / 32)


def rotate(x, positions, frequencies, magnitude, interleaved, inverse):
    """(rotated, magnitude) of x (places, heads, head_dim)."""
    R = 2 * len(frequencies)
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    angle = np.asarray(positions, np.float64)[:, None, None] * np.asarray(frequencies, np.float64)
    c, s = magnitude * np.cos(angle), magnitude * np.sin(angle) * (-1 if inverse else 1)
    out, mag = x.copy(), np.zeros_like(x)
    out[..., a], out[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    mag[..., a] = mag[..., b] = abs(magnitude) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return out, mag
