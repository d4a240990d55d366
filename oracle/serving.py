"""Float64 single-token serving operators: attention of one new token over
the cache, eviction by accumulated attention weight, and token sampling with
temperature, top-k, top-p and min-p.

TEST INFRASTRUCTURE: part of the CPU oracle (see oracle/__init__.py).

What the pages fix: decoding with a KV cache, GQA and paged KV ("LLM
inference acceleration", section two), the sampler's temperature (section
3.2).  Readings: rows outside the attended set never take part, whatever
they hold; an empty set gives o = 0 and lse = -inf; eviction keeps the first
`sinks` and the last `recent` rows and of the others the largest
accumulated weights (equal ones: the lowest row), per layer and KV head, in
row order; the filters of a sample apply in the order top-k, top-p, min-p to
the ids in the order of falling logits (equal ones: the lowest id), and the
token is drawn by inverse CDF over ids in increasing order.
"""
from __future__ import annotations

import numpy as np


def decode_attention(q, k, v, k_new=None, v_new=None, window: int = 0):
    """One request, one layer.  q [n_q, hd]; k, v [L, n_kv, hd]; new rows [n_kv, hd] or None.

    Returns out [n_q, hd], lse [n_q], weights [n_kv, n] summed over each KV head's query heads (0 outside the set)."""
    if k_new is not None:
        k = np.concatenate([k, k_new[None]])
        v = np.concatenate([v, v_new[None]])
    n, n_kv, hd = k.shape
    n_q = q.shape[0]
    g = n_q // n_kv
    lo = max(0, n - window) if window else 0
    out, lse, weights = np.zeros((n_q, hd)), np.full(n_q, -np.inf), np.zeros((n_kv, n))
    if n == 0:
        return out, lse, weights
    for hq in range(n_q):
        h = hq // g
        s = k[lo:, h] @ q[hq] / np.sqrt(hd)
        m = s.max()
        e = np.exp(s - m)
        p = e / e.sum()
        out[hq] = p @ v[lo:, h]
        lse[hq] = m + np.log(e.sum())
        weights[h, lo:] += p
    return out, lse, weights


def evict_rows(score, L: int, budget: int, sinks: int = 0, recent: int = 0) -> np.ndarray:
    """Rows kept by one (layer, request, KV head), ascending; score [>= L]."""
    if L <= budget:
        return np.arange(L)
    lo, hi = sinks, L - recent
    mid = np.asarray(score[lo:hi], np.float64)
    order = sorted(range(lo, hi), key=lambda i: (np.isnan(mid[i - lo]), -mid[i - lo] if mid[i - lo] == mid[i - lo] else 0.0, i))
    chosen = order[: budget - sinks - recent]
    return np.array(sorted(list(range(lo)) + chosen + list(range(hi, L))), np.int64)


def filtered(x, T: float, top_k: int = 0, top_p: float = 1.0, min_p: float = 0.0) -> np.ndarray:
    """Weights of the kept tokens (0 elsewhere), relative to the largest."""
    x = np.asarray(x, np.float64)
    live = ~(np.isnan(x) | (x == -np.inf))
    w = np.zeros(len(x))
    if not live.any():
        return w
    m = x[live].max()
    with np.errstate(invalid="ignore"):
        w[live] = np.where(x[live] == m, 1.0, np.exp((x[live] - m) / T))
    ids = np.nonzero(live)[0]
    ids = ids[np.lexsort((ids, -x[ids]))]
    if 0 < top_k < len(x):
        ids = ids[:top_k]
    if top_p < 1.0:
        c = np.cumsum(w[ids])
        ids = ids[: max(1, int(np.searchsorted(c, top_p * c[-1], side="left")) + 1)]
    if min_p > 0.0:
        ids = ids[w[ids] >= min(min_p, 1.0)]
    kept = np.zeros(len(x))
    kept[ids] = w[ids]
    return kept


def sample_logits(x, u: float, T: float = 1.0, top_k: int = 0, top_p: float = 1.0, min_p: float = 0.0):
    """(token, logprob, distance of u * total to the nearest cumulative boundary relative to the total)."""
    x = np.asarray(x, np.float64)
    live = ~(np.isnan(x) | (x == -np.inf))
    if not live.any():
        return -1, -np.inf, np.inf
    if not T > 0:
        return int(np.argmax(np.where(live, x, -np.inf))), 0.0, np.inf
    w = filtered(x, T, top_k, top_p, min_p)
    c = np.cumsum(w)
    t = min(max(u, 0.0), 1.0) * c[-1]
    tok = int(np.searchsorted(c, t, side="left")) if t > 0 else int(np.nonzero(w)[0][0])
    lo = c[tok - 1] if tok else 0.0
    return tok, float(np.log(w[tok] / c[-1])), float(min(t - lo, c[tok] - t) / c[-1])
