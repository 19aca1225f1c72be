"""The choice of experts from router logits and the experts' mean scores, float64.

PagedWeight, "Dynamic Paging": the router decides which experts a pass needs;
"Quality-Aware Quantization" takes an importance p_e per expert, its mean
routing probability over a calibration set. For a token's logits l:

    s_e = e^{l_e} / sum_i e^{l_i}   or   s_e = 1 / (1 + e^{-l_e}),
    key_e = s_e + bias_e.

Experts form n_groups groups of consecutive indices; the keep_groups groups of
highest score (their largest key, or the sum of their two largest) stay, and
the k experts of largest key in them are chosen. w_e = scale s_e, divided by
the sum of the chosen scores when renormalised. p_e is the mean of s_e over
the tokens.

Readings taken: ties go to the lower index, without a bias the order (of groups
by their largest key too) is the logits' own, a logit of -inf scores 0 (so does a softmax over nothing but
-inf), weights whose sum is 0 are 0, NaN keys rank lowest, and a token with a
NaN logit (or +inf under the softmax) gets NaN weights.
"""
from __future__ import annotations

import math

import numpy as np


def scores(logits: np.ndarray, score: str) -> np.ndarray:
    """s [T, E] for logits [T, E]."""
    l = np.asarray(logits, dtype=np.float64)
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-l))
        m = l.max(axis=1, keepdims=True)
        e = np.where(np.isneginf(l) & ~np.isnan(m), 0.0, np.exp(l - m))
        total = e.sum(axis=1, keepdims=True)
        return np.where(total == 0.0, 0.0, e / np.where(total == 0.0, 1.0, total))


def _rank(values, indices):
    """indices by descending value, NaN last, ties by index."""
    return sorted(indices, key=lambda i: (math.isnan(values[i]), 0.0 if math.isnan(values[i]) else -values[i], i))


def select_experts(logits, k: int, bias=None, score: str = "softmax", n_groups: int = 1,
                   keep_groups: int | None = None, group_score: str = "top2",
                   renormalize: bool = True, scale: float = 1.0):
    """(ids int32 [T, k], w float64 [T, k])."""
    l = np.asarray(logits, dtype=np.float64)
    T, E = l.shape
    keep_groups = n_groups if keep_groups is None else keep_groups
    s = scores(l, score)
    ids = np.zeros((T, k), dtype=np.int32)
    w = np.zeros((T, k), dtype=np.float64)
    size = E // n_groups
    for t in range(T):
        key = s[t] if bias is None else s[t] + np.asarray(bias, dtype=np.float64)
        pool = range(E)
        if keep_groups < n_groups:
            value = []
            for g in range(n_groups):
                members = range(g * size, (g + 1) * size)
                if group_score == "max":
                    by = l[t] if bias is None else key
                    value.append(float(by[_rank(by, members)[0]]))
                else:
                    value.append(sum(float(key[i]) for i in _rank(key, members)[:2]))
            kept = _rank(value, range(n_groups))[:keep_groups]
            pool = [e for g in sorted(kept) for e in range(g * size, (g + 1) * size)]
        chosen = _rank(l[t] if bias is None else key, pool)[:k]
        got = s[t][chosen]
        if renormalize:
            if score == "softmax":  # the softmax over the chosen ones alone
                got = scores(l[t][chosen][None], score)[0]
            elif max(l[t][chosen]) < 0.0:  # e^l / (1 + e^l), over e^(the largest l): float64 has no score this small
                lc = l[t][chosen]
                got = np.where(np.isneginf(lc), 0.0, np.exp(lc - max(lc.max(), -1e300)) / (1.0 + np.exp(lc)))
            total = got.sum()
            got = np.zeros(k) if total == 0.0 else got / total
        broken = np.isnan(l[t]).any() or (score == "softmax" and np.isposinf(l[t]).any())
        ids[t] = chosen
        w[t] = np.nan if broken else scale * got
    return ids, w


def expert_importance(logits, score: str = "softmax") -> np.ndarray:
    """p [E]: the mean of s over the tokens."""
    s = scores(logits, score)
    return np.array([math.fsum(s[:, e]) if np.isfinite(s[:, e]).all() else math.nan
                     for e in range(s.shape[1])]) / s.shape[0]
