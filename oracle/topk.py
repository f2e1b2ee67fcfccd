"""Top-k expert choice from router scores in fp64 — oracle, test infrastructure only.

Scores are the softmax or the sigmoid of the logits; a logit of -inf or NaN masks its expert
(score 0).  The choice goes by the logits, or with a bias by score + bias; groups are ranked
by the sum of their topn best keys (scores without a bias); ties go to the lower index and
masked experts come last.  The weights are the chosen scores, divided by their sum if
renormalised, times a factor; a sum of 0 gives weights of 0.
"""
from __future__ import annotations

import math

import numpy as np


def scores(l: np.ndarray, score: str) -> np.ndarray:
    """fp64 scores of one token's fp64 logits."""
    off = np.isnan(l) | np.isneginf(l)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            s = 1.0 / (1.0 + np.exp(-np.where(off, 0.0, l)))
        return np.where(off, 0.0, s)
    if off.all():
        return np.zeros_like(l)
    m = l[~off].max()
    d = np.where(off | (l == m), 0.0, l - m)
    e = np.where(off, 0.0, np.exp(d))
    return e / e.sum()


def choose(logits, k, score="softmax", bias=None, num_groups=1, topk_groups=1, topn=2):
    """int32 [T][k]."""
    L = np.asarray(logits, dtype=np.float64)
    T, E = L.shape
    out = np.zeros((T, k), dtype=np.int32)
    gs = E // num_groups
    for t in range(T):
        l = L[t]
        s = scores(l, score)
        off = np.isnan(l) | np.isneginf(l)
        key = l.copy() if bias is None else s + np.asarray(bias, dtype=np.float64)
        off = off | np.isnan(key) | np.isneginf(key)
        kept = range(num_groups)
        if topk_groups < num_groups:
            by = s if bias is None and topn == 2 else key
            g = []
            for j in range(num_groups):
                best = sorted((by[e] for e in range(j * gs, (j + 1) * gs) if not off[e]), reverse=True)[:topn]
                g.append(sum(best) if best else -math.inf)
            kept = sorted(range(num_groups), key=lambda j: (-g[j], j))[:topk_groups]
        pool = [e for j in kept for e in range(j * gs, (j + 1) * gs)]
        out[t] = sorted(pool, key=lambda e: (off[e], 0.0 if off[e] else -key[e], e))[:k]
    return out


def weights(logits, idx, score="softmax", renorm=True, scale=1.0):
    """fp64 [T][k]; sigmoid ratios are taken from logarithms so that they survive underflow."""
    L = np.asarray(logits, dtype=np.float64)
    T, k = idx.shape
    w = np.zeros((T, k))
    for t in range(T):
        s = scores(L[t], score)[idx[t]]
        if renorm:
            l = L[t][idx[t]]
            on = ~(np.isnan(l) | np.isneginf(l))
            if not on.any():
                s = np.zeros(k)
            else:
                if score == "sigmoid":
                    lg = np.where(on, -np.logaddexp(0.0, -np.where(on, l, 0.0)), -np.inf)
                else:
                    lg = np.where(on, l, -np.inf)
                m = lg.max()
                s = np.where(on, np.exp(np.where(lg == m, 0.0, lg - m)), 0.0)
                s = s / s.sum()
        w[t] = s * scale
    return w


def bwd(logits, idx, d_prob, score="softmax", renorm=True, scale=1.0):
    """fp64 [T][E]: the Jacobian of the weights, written out slot by slot."""
    L = np.asarray(logits, dtype=np.float64)
    d = np.asarray(d_prob, dtype=np.float64) * scale
    T, E = L.shape
    k = idx.shape[1]
    out = np.zeros((T, E))
    for t in range(T):
        s = scores(L[t], score)
        use = [i for i in range(k) if 0 <= idx[t, i] < E]
        w = weights(L[t:t + 1], idx[t:t + 1, use], score, True, 1.0)[0] if use else np.zeros(0)
        if renorm:
            dot = sum(w[j] * d[t, i] for j, i in enumerate(use))
            for j, i in enumerate(use):
                e = idx[t, i]
                f = (1.0 - s[e]) if score == "sigmoid" else 1.0
                out[t, e] += w[j] * (d[t, i] - dot) * f
        elif score == "sigmoid":
            for i in use:
                e = idx[t, i]
                out[t, e] += d[t, i] * s[e] * (1.0 - s[e])
        else:
            dot = sum(s[idx[t, i]] * d[t, i] for i in use)
            out[t] -= s * dot
            for i in use:
                out[t, idx[t, i]] += s[idx[t, i]] * d[t, i]
    return out
