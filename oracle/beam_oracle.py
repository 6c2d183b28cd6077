"""Float64 definitions of decoding by beams: the best continuations of each sequence
and the reordering of states.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Written from the formulas
of include/flashhead.h in numpy, one sequence and one beam at a time.
"""

from __future__ import annotations

import numpy as np

U = 2.0 ** -24  # half a step of float32


def log_sum_exp(z):
    """Of one row; NaN where it holds NaN or +inf."""
    m = z.max() if z.size else -np.inf
    if np.isnan(z).any() or m == np.inf:
        return np.nan
    if m == -np.inf:
        return -np.inf
    return m + np.log(np.exp(z - m).sum())


def totals(z, scores, ids=None, v=None, lse=None, finished=None, eos=-1):
    """Per sequence the continuations (total, beam, place, token) that it has, in
    the order of beam and place, as arrays."""
    z, scores = np.asarray(z, np.float64), np.asarray(scores, np.float64)
    S, W = scores.shape
    out = []
    for s in range(S):
        t, beam, place, token = [], [], [], []
        for w in range(W):
            r, score = s * W + w, scores[s, w]
            if not score > -np.inf:
                continue
            if finished is not None and finished[s, w]:
                t.append(np.array([score]))
                beam.append(np.array([w]))
                place.append(np.array([0]))
                token.append(np.array([eos]))
                continue
            row = z[r].copy()
            tok = np.arange(row.size) if ids is None else np.asarray(ids[r], np.int64)
            if ids is not None:
                row[(tok < 0) | (tok >= v)] = -np.inf
            l = log_sum_exp(row) if lse is None else np.float64(lse[r])
            with np.errstate(invalid="ignore"):
                x = score + (row - l)
            at = np.flatnonzero(x > -np.inf)
            t.append(x[at])
            beam.append(np.full(at.size, w))
            place.append(at)
            token.append(tok[at])
        empty = np.zeros(0)
        out.append(tuple(np.concatenate(a) if a else empty for a in (t, beam, place, token)))
    return out


def select(z, scores, keep, **kw):
    """(score, token, parent) [S x keep]: the largest totals, ties to the smaller
    beam, then the earlier place."""
    found = totals(z, scores, **kw)
    S = len(found)
    score, token, parent = np.full((S, keep), -np.inf), np.full((S, keep), -1), np.full((S, keep), -1)
    for s, (t, beam, place, tok) in enumerate(found):
        best = np.lexsort((place, beam, -t))[:keep]
        score[s, :best.size], token[s, :best.size], parent[s, :best.size] = t[best], tok[best], beam[best]
    return score, token, parent


def check_select(z, scores, keep, out, exact=False, **kw):
    """Failures of out["score"], ["token"], ["parent"] (and ["finished"]).

    exact: logits and log-sum-exps that leave nothing to round, every token as the
    definition's.  Else a total is known to its lse's error: each exponential within
    (2 + |x - m|) 2 u of itself, twice (a part's and the parts'), whose mean over
    the row is at most 2 + ln n (the entropy); 24 roundings of the sum of a part,
    one of its product with its exponential; float64 from there, and the result
    rounded to float32.
    """
    fails = []
    score, token, parent = select(z, scores, keep, **kw)
    n = np.asarray(z).shape[1]
    known = kw.get("lse") is not None
    err = 0.0 if exact or known else 2 * 4 * U * (2 + np.log(n)) + 26 * U
    found = totals(z, scores, **kw)
    for s in range(score.shape[0]):
        got = list(zip(out["parent"][s].tolist(), out["token"][s].tolist()))
        live = int((score[s] > -np.inf).sum())
        if any(p != -1 or t != -1 for p, t in got[live:]) or not np.all(np.isneginf(out["score"][s, live:])):
            fails.append(f"sequence {s}: {live} continuations, got {got[live:]} behind them")
            continue
        t, beam, place, tok = found[s]
        value = {}
        for a, b, c in zip(t, beam, tok):  # a token listed twice is two
            value.setdefault((int(b), int(c)), []).append(a)
        used = {}
        for r in range(live):
            want, have = score[s, r], value.get(got[r])
            k = used.get(got[r], 0)
            used[got[r]] = k + 1
            if have is None or k >= len(have):
                fails.append(f"sequence {s}, rank {r}: {got[r]} is no continuation, or twice")
                continue
            mine = sorted(have, reverse=True)[k]
            if exact or known:
                if got[r] != (parent[s, r], token[s, r]):
                    fails.append(f"sequence {s}, rank {r}: {got[r]}, expected {(parent[s, r], token[s, r])}")
            elif abs(mine - want) > 2 * err:
                fails.append(f"sequence {s}, rank {r}: {got[r]} has total {mine}, expected {want}")
            if abs(out["score"][s, r] - mine) > err + U * abs(mine) * (1 + U):
                fails.append(f"sequence {s}, rank {r}: score {out['score'][s, r]}, expected {mine}")
        if "finished" in out:
            want = [int(i < live and p[1] == kw["eos"]) for i, p in enumerate(got)]
            if out["finished"][s].tolist() != want:
                fails.append(f"sequence {s}: finished {out['finished'][s].tolist()}, expected {want}")
    return fails


def reorder(state, parent, lengths=None, dim=0, length_dim=None):
    """The state after every row s W + w took row s W + parent[s, w]."""
    parent = np.asarray(parent)
    S, W = parent.shape
    old = np.moveaxis(np.asarray(state), dim, 0)
    new = old.copy()
    for s in range(S):
        for w in range(W):
            p = int(parent[s, w])
            if not 0 <= p < W:
                continue
            at = [slice(None)] * (old.ndim - 1)
            if lengths is not None:
                # the row is gone from the front: what was behind dim stays one place on
                axis = length_dim % np.asarray(state).ndim - 1
                at[axis] = slice(0, int(np.clip(lengths[s * W + p], 0, old.shape[axis + 1])))
            new[(s * W + w, *at)] = old[(s * W + p, *at)]
    return np.moveaxis(new, 0, dim)
