"""Float64 definitions of the operators around the dense head: the norm with the
residual's addition and its int8 output, the int8 product, the rules on logits
and the choice of the token.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Written from the
formulas of include/flashhead.h, one row and one rule at a time, in numpy.
"""

from __future__ import annotations

import numpy as np

from .philox import gumbel


def rmsnorm(x, residual, weight, eps, offset):
    """(y, s) of rows x [B x d]: y = s / sqrt(mean(s^2) + eps) (offset + weight)."""
    s = np.asarray(x, np.float64)
    if residual is not None:
        s = s + np.asarray(residual, np.float64)
    y = s / np.sqrt(np.mean(s * s, axis=1, keepdims=True) + np.float64(np.float32(eps)))
    if weight is not None:
        y = y * (offset + np.asarray(weight, np.float64))
    return y, s


def product(q, q_scale, codes, scales):
    """[B x n]: exact sums (whole numbers below 2^53 in float64), scaled in float64."""
    acc = np.asarray(q, np.float64) @ np.asarray(codes, np.float64).T
    return acc * np.asarray(q_scale, np.float64)[:, None] * np.asarray(scales, np.float64)[None, :]


def apply_rules(z, ids, v, *, history=None, n_prompt=None, n_history=None, repetition=None, frequency=None,
                presence=None, bias_ids=None, bias=None, n_bias=None, mask=None, mask_row=None):
    """(logits, size): the rules on z [B x n] of tokens ids [B x n] (None: all v
    tokens), and the sum of magnitudes that each result was rounded from."""
    z = np.asarray(z, np.float64).copy()
    B, n = z.shape
    size = np.abs(z)
    for b in range(B):
        t = np.arange(n) if ids is None else np.asarray(ids[b], np.int64)
        known = (t >= 0) & (t < v)
        tt = np.where(known, t, 0)
        if history is not None:
            L = history.shape[1]
            nh = int(np.clip(L if n_history is None else n_history[b], 0, L))
            np_ = int(np.clip(0 if n_prompt is None else n_prompt[b], 0, nh))
            text = np.asarray(history[b, :nh], np.int64)
            valid = (text >= 0) & (text < v)
            seen = np.zeros(v, bool)
            seen[text[valid]] = True
            count = np.bincount(text[np_:][valid[np_:]], minlength=v)
            rep = 1.0 if repetition is None else float(repetition[b])
            hit = seen[tt] & known
            with np.errstate(invalid="ignore"):
                z[b] = np.where(hit, np.where(z[b] > 0, z[b] / rep, z[b] * rep), z[b])
            c = np.where(known, count[tt], 0)
            often = c * (0.0 if frequency is None else float(frequency[b]))
            once = (c > 0) * (0.0 if presence is None else float(presence[b]))
            # each step's own magnitude: z - often is rounded at up to |z| + |often|, also
            # where presence then takes it back (f = 0.1807, p = -0.1743, z = -0.0055:
            # 2^-24 * 0.186 = 1.1e-8, where 8 * 2^-24 (|z| + |often + once|) is 5.6e-9)
            size[b] = np.abs(z[b]) + np.abs(often) + np.abs(once)
            z[b] -= often + once
        if bias_ids is not None:
            N = bias_ids.shape[1]
            nb = int(np.clip(N if n_bias is None else n_bias[b], 0, N))
            add, mag = np.zeros(v), np.zeros(v)
            for i in range(nb):
                if 0 <= bias_ids[b, i] < v:
                    add[bias_ids[b, i]] += float(bias[b, i])
                    mag[bias_ids[b, i]] += 4 * abs(float(bias[b, i]))
            z[b] += np.where(known, add[tt], 0.0)
            size[b] += np.where(known, mag[tt], 0.0)
        shut = ~known
        if mask is not None:
            r = b if mask_row is None else int(mask_row[b])
            if 0 <= r < mask.shape[0]:
                words = np.asarray(mask[r]).astype(np.int64) & 0xFFFFFFFF
                shut |= ((words[tt >> 5] >> (tt & 31)) & 1) == 0
        z[b, shut] = -np.inf
        size[b, shut] = 0.0
    return z, size


def keys(z, ids, mode, temperature, seed):
    """The selection keys [B x n] of logits z: z, or z / T + G(seed, row, token, 1)."""
    z = np.asarray(z, np.float64)
    if not mode & 2:
        return z
    B, n = z.shape
    t = np.broadcast_to(np.arange(n), (B, n)) if ids is None else np.asarray(ids, np.int64)
    rows = np.broadcast_to(np.arange(B)[:, None], (B, n))
    return z / np.float64(np.float32(temperature)) + gumbel(seed, rows, np.maximum(t, 0), 1)


def lse(z, tprime):
    """log sum exp(z / T') of rows; -inf where nothing is left."""
    x = np.asarray(z, np.float64) / tprime
    m = x.max(axis=1)
    with np.errstate(invalid="ignore", divide="ignore"):
        s = np.exp(x - np.where(np.isneginf(m), 0.0, m)[:, None]).sum(axis=1)
        return np.where(np.isneginf(m), -np.inf, m + np.log(s))


def check_choice(z, z_tol, ids, mode, temperature, seed, out):
    """Failures of a choice: out["token"], ["token_logit"], ["lse"] against
    logits z [B x n] known to z_tol (absolute, per element).

    Rounding of what the kernel computes from a logit, in float32 (u = 2^-24):
    x = z / T' one division (|x| u).  A Gumbel draw -ln(-ln u'): both logarithms
    within 2 u of themselves, the inner one's relative error an absolute one of
    the outer, |G| <= 16.7: 36 u, and the key's sum one rounding more; 4 u of
    (|x| + 24) covers them.  LSE: each exponential within (2 + |x - m|) 2 u of
    itself, whose mean over the row is at most 2 + ln n (the entropy), sums of
    positive terms of depth <= n / 8192 + 160, one logarithm.
    """
    u = 2.0 ** -24
    fails = []
    T = float(np.float32(temperature)) if mode & 2 else 1.0
    key = keys(z, ids, mode, temperature, seed)
    with np.errstate(invalid="ignore"):
        ktol = z_tol / T + 4 * u * (np.abs(np.where(np.isfinite(z), z, 0.0)) / T + (24.0 if mode & 2 else 0.0))
    want_lse = lse(z, T)
    B, n = z.shape
    for b in range(B):
        live = key[b] > -np.inf
        tok = int(out["token"][b])
        if not live.any():
            if tok != -1 or out["token_logit"][b] != -np.inf or out["lse"][b] != -np.inf:
                fails.append(f"row {b}: nothing is left, got token {tok}, lse {out['lse'][b]}")
            continue
        at = np.flatnonzero((np.arange(n) if ids is None else np.asarray(ids[b])) == tok)
        at = at[live[at]]
        if not at.size:
            fails.append(f"row {b}: token {tok} is not one of those left")
            continue
        i = at[key[b, at].argmax()]  # a token listed several times is taken at its best place
        best = np.where(live, key[b], -np.inf)
        j = int(best.argmax())
        if not best[i] >= best[j] - ktol[b, i] - ktol[b, j]:
            fails.append(f"row {b}: token {tok} has key {best[i]}, the best is {best[j]}")
        if abs(out["token_logit"][b] - z[b, i]) > z_tol[b, i] + u * abs(z[b, i]):
            fails.append(f"row {b}: token logit {out['token_logit'][b]}, expected {z[b, i]}")
        fin = np.isfinite(z[b])
        xmax = np.abs(z[b, fin] / T).max() if fin.any() else 0.0
        tol = (z_tol[b].max() / T + 2 * u * xmax + 4 * u * (2 + np.log(n)) + u * (n / 8192 + 160)
               + 2 * u * (abs(want_lse[b]) + 16.0))
        if not abs(out["lse"][b] - want_lse[b]) <= tol:
            fails.append(f"row {b}: lse {out['lse'][b]}, expected {want_lse[b]} within {tol:.3g}")
    return fails
