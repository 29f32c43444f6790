"""The definition of moe_beam_select in 64 bits (numpy), for its tests."""
from __future__ import annotations

import math

import numpy as np


def lse64(x: np.ndarray) -> float:
    """log of the sum of exponentials of one row; NaN where it has a NaN or +infinity."""
    x = np.asarray(x, np.float64)
    if np.isnan(x).any() or np.isposinf(x).any():
        return math.nan
    top = x.max()
    if top == -math.inf:
        return -math.inf
    return float(top + math.log(math.fsum(np.exp(x - top))))


def select64(logits, scores, n_out, done=None, end_token=-1):
    """parent, token [requests][n_out], score (float64), done_out and lse [requests][beams] of logits [requests * beams][vocab]
    (float64 of the values as stored) and scores [requests][beams]."""
    R, B = scores.shape
    parent, token = np.full((R, n_out), -1, np.int64), np.full((R, n_out), -1, np.int64)
    score, ended = np.full((R, n_out), -np.inf), np.ones((R, n_out), bool)
    lse = np.array([[lse64(logits[r * B + b]) for b in range(B)] for r in range(R)])
    for r in range(R):
        found = []  # (-sum, row, -logit, token)
        for b in range(B):
            row, base = r * B + b, np.float64(scores[r, b])
            if done is not None and done[r, b]:
                if np.isfinite(base):
                    found.append((-base, row, 0.0, end_token))
                continue
            with np.errstate(invalid="ignore"):
                base = base - lse[r, b]
            if not np.isfinite(base):
                continue
            x = logits[row]
            v = np.nonzero(x > -np.inf)[0]
            v = v[np.lexsort((v, -x[v]))][:n_out]
            found += [(-(base + x[t]), row, -x[t], int(t)) for t in v]
        found.sort()
        for i, (c, row, _, t) in enumerate(found[:n_out]):
            parent[r, i], token[r, i], score[r, i] = row, t, -c
            ended[r, i] = t == end_token or (done is not None and bool(done[r, row - r * B]))
    return parent, token, score, ended, lse
