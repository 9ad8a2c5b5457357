"""The input-layer operators from their definitions, in numpy and 64 bits.

Shares nothing with the library: the generator is written with numpy's
unsigned arithmetic, the sums are plain float64 sums per row.  Alongside each
result the functions return the sum of the magnitudes that went into every
element, from which the tests derive their error bounds.
"""
from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24  # unit roundoff of fp32


def splitmix64(start: int, k: np.ndarray) -> np.ndarray:
    with np.errstate(over="ignore"):
        z = np.uint64(start) + (k.astype(np.uint64) + np.uint64(1)) * np.uint64(0x9E3779B97F4A7C15)
        z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
        z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
        return z ^ (z >> np.uint64(31))


def threshold(p: float) -> int:
    return int(np.floor(float(np.float32(p)) * 65536.0 + 0.5))


def keep_mask(rows: int, cols: int, drop) -> np.ndarray:
    if drop is None or threshold(drop[0]) == 0:
        return np.ones((rows, cols), dtype=bool)
    p, seed, stream = drop
    n = rows * cols
    key = int(splitmix64(seed, np.array([stream], dtype=np.uint64))[0])
    z = splitmix64(key, np.arange((n + 3) // 4, dtype=np.uint64))
    fields = (z[:, None] >> np.array([0, 16, 32, 48], dtype=np.uint64)) & np.uint64(0xFFFF)
    return (fields.reshape(-1)[:n] >= np.uint64(threshold(p))).reshape(rows, cols)


def rescale(drop) -> float:
    """1 / (share kept) in 64 bits; 0 when nothing is kept."""
    if drop is None:
        return 1.0
    t = threshold(drop[0])
    return 0.0 if t == 65536 else 65536.0 / (65536.0 - t)


def place_positions(n, positions, seq_len, first):
    return np.arange(n) % seq_len + first if positions is None else np.asarray(positions).reshape(-1)


def lookup(tokens, table, pos_table, scale, drop, positions=None, seq_len=1, first=0):
    """(out, magnitude), float64."""
    tokens = np.asarray(tokens).reshape(-1)
    n, (V, D) = tokens.size, table.shape
    out, mag = np.zeros((n, D)), np.zeros((n, D))
    q = place_positions(n, positions, seq_len, first)
    for i, t in enumerate(tokens):
        if 0 <= t < V:
            row = scale * table[t].astype(np.float64)
            out[i], mag[i] = row, np.abs(row)
            if pos_table is not None and 0 <= q[i] < pos_table.shape[0]:
                out[i] += pos_table[q[i]]
                mag[i] += np.abs(pos_table[q[i]])
    keep, r = keep_mask(n, D, drop), rescale(drop)
    return np.where(keep, out * r, 0.0), np.where(keep, mag * r, 0.0)


def key_sums(keys, nkeys, dout, keep, factor, base):
    """(sums, magnitudes, counts) of keep * dout over the places of each key
    (keys outside [0, nkeys) are left out)."""
    D = dout.shape[1]
    out, mag = np.zeros((nkeys, D)), np.zeros((nkeys, D))
    count = np.zeros((nkeys, 1))
    for i, k in enumerate(keys):
        if 0 <= k < nkeys:
            x = np.where(keep[i], dout[i], 0.0)
            out[k] += x
            mag[k] += np.abs(x)
            count[k] += 1
    out, mag = out * factor, mag * abs(factor)
    if base is not None:
        out, mag = out + base, mag + np.abs(base)
    return out, mag, count


def gradients(tokens, vocab, npos, dout, scale, drop, base=None, pos_base=None, positions=None, seq_len=1, first=0):
    """((grad, mag, count), (pos_grad, mag, count) or None)."""
    tokens = np.asarray(tokens).reshape(-1)
    keep, r = keep_mask(*dout.shape, drop), rescale(drop)
    token = key_sums(tokens, vocab, dout, keep, scale * r, base)
    if not npos:
        return token, None
    q = np.where((tokens >= 0) & (tokens < vocab), place_positions(tokens.size, positions, seq_len, first), -1)
    return token, key_sums(q, npos, dout, keep, r, pos_base)


def limits(exact, magnitude, terms):
    """Range of the results of an fp32 evaluation with `terms` roundings, each
    at most U32 of the magnitude (to first order; 1 % covers the rest); 1e-37
    covers results below the normal range.  Rounding is monotonic, so a result
    that is rounded once more lies between the limits rounded alike."""
    err = 1.01 * U32 * terms * magnitude + 1e-37
    return exact - err, exact + err
