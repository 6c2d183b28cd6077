"""Float64 definitions of the fp8 head: E4M3 codes, hidden states under a scale per
128, and the product of such operands.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Written from the formulas
of include/flashhead.h in numpy.
"""

from __future__ import annotations

import numpy as np


def e4m3_values():
    """The value of each of the 256 codes: sign, 4 bits of exponent with bias 7,
    3 of fraction; no infinities, NaN at 0x7F and 0xFF."""
    c = np.arange(256)
    e, f = (c >> 3) & 15, c & 7
    v = np.where(e == 0, f / 8.0 * 2.0 ** -6, (1 + f / 8.0) * 2.0 ** (e - 7.0))
    v = np.where(c & 0x7F == 0x7F, np.nan, v)
    return np.where(c >= 128, -v, v)


def e4m3_encode(t):
    """Codes of t, |t| <= 448, to the nearest, ties to the even code."""
    t = np.asarray(t, np.float64)
    grid = e4m3_values()[:127]  # 0 .. 448, ascending
    a = np.minimum(np.abs(t), 448.0)
    hi = np.clip(np.searchsorted(grid, a), 1, 126)
    lo = hi - 1
    down, up = a - grid[lo], grid[hi] - a
    code = np.where(down < up, lo, np.where(up < down, hi, np.where(lo % 2 == 0, lo, hi)))
    return (code + 128 * np.signbit(t)).astype(np.uint8)


def groups(y):
    """Columns of each 128, as slices."""
    return [slice(lo, min(lo + 128, y)) for lo in range(0, y, 128)]


def quant(y):
    """(codes, scales) of float32 rows y [B x d]: the scale and the quotient each
    rounded to float32 as the definition has it, then E4M3."""
    y = np.asarray(y, np.float32)
    scales = np.stack([np.abs(y[:, g]).max(1) / np.float32(448) for g in groups(y.shape[1])], 1)
    codes = np.zeros(y.shape, np.uint8)
    for i, g in enumerate(groups(y.shape[1])):
        s = scales[:, i:i + 1]
        with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
            codes[:, g] = np.where(s > 0, e4m3_encode(np.where(s > 0, y[:, g] / s, 0)), 0)
    return codes, scales


def quant_weight(W):
    """(codes, scales) of W [n x k] by blocks of 128 x 128."""
    W = np.asarray(W, np.float32)
    rows, cols = groups(W.shape[0]), groups(W.shape[1])
    scales = np.array([[np.abs(W[r, c]).max() / np.float32(448) for c in cols] for r in rows], np.float32)
    codes = np.zeros(W.shape, np.uint8)
    for i, r in enumerate(rows):
        for j, c in enumerate(cols):
            if scales[i, j] > 0:
                codes[r, c] = e4m3_encode(W[r, c] / scales[i, j])
    return codes, scales


def product(q, q_scale, codes, scales):
    """(out, size): [B x n] in float64, and the sum of magnitudes behind each."""
    v = e4m3_values()
    a, w = v[np.asarray(q, np.uint8)], v[np.asarray(codes, np.uint8)]
    out = np.zeros((a.shape[0], w.shape[0]))
    size = np.zeros_like(out)
    per = np.repeat(np.asarray(scales, np.float64), 128, 0)[:w.shape[0]]
    for i, g in enumerate(groups(a.shape[1])):
        s = np.asarray(q_scale, np.float64)[:, i:i + 1] * per[None, :, i]
        out += (a[:, g] @ w[:, g].T) * s
        size += (np.abs(a[:, g]) @ np.abs(w[:, g]).T) * np.abs(s)
    return out, size
