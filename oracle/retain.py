"""fp64 CPU oracle of accumulated attention weights and of the eviction by them.

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle/``: plain definitions, a
loop per sequence and head, sharing nothing with the CUDA path.
"""
from __future__ import annotations

from typing import List, Tuple

import numpy as np

from .attention import scores
from .paged import paged_rows

__all__ = ["weights_paged", "keep_positions", "evict_paged"]


def weights_paged(q: np.ndarray, k_pages: np.ndarray, lse: np.ndarray, weights: np.ndarray, table: np.ndarray,
                  cu: np.ndarray, kv_lens: np.ndarray, causal: bool, scale: float) -> Tuple[np.ndarray, np.ndarray]:
    """weights [n_pages, Hkv, page] after the packed rows q [H, total, d] with
    their lse [H, total]; and what they added to each."""
    q, lse = np.asarray(q, np.float64), np.asarray(lse, np.float64)
    out, new = np.array(weights, np.float64), np.zeros(weights.shape)
    Hkv, page = weights.shape[1], weights.shape[2]
    group = q.shape[0] // Hkv
    for b in range(len(kv_lens)):
        s0, s1, nk = int(cu[b]), int(cu[b + 1]), int(kv_lens[b])
        n = s1 - s0
        if n == 0 or nk == 0:
            continue
        k = paged_rows(k_pages, table[b], nk)
        seen = np.arange(nk)[None] <= np.arange(n)[:, None] + nk - n if causal else np.ones((n, nk), bool)
        for h in range(Hkv):
            got = np.zeros(nk)
            for i in range(h * group, (h + 1) * group):
                with np.errstate(invalid="ignore", over="ignore"):
                    p = np.exp(scores(q[i, s0:s1], k[h], scale) - lse[i, s0:s1, None])
                got += np.where(seen, p, 0.0).sum(0)
            for j in range(nk):
                at = table[b][j // page], h, j % page
                out[at] = got[j] + (out[at] if j < nk - n else 0.0)
                new[at] = got[j]
    return out, new


def keep_positions(weights: np.ndarray, budget: int, sinks: int, recent: int) -> List[int]:
    """Positions of a sequence's head that stay, by its weights."""
    n = len(weights)
    if n <= budget:
        return list(range(n))
    middle = list(range(sinks, n - recent))
    heavy = [np.inf if np.isnan(w) else w for w in weights]
    nan = [np.isnan(w) for w in weights]
    middle.sort(key=lambda j: (not nan[j], -heavy[j], j))
    return list(range(sinks)) + sorted(middle[:budget - sinks - recent]) + list(range(n - recent, n))


def evict_paged(pages: List[np.ndarray], weights: np.ndarray, table: np.ndarray, kv_lens: np.ndarray, budget: int,
                sinks: int, recent: int) -> Tuple[List[np.ndarray], np.ndarray, np.ndarray]:
    """Each of pages [n_pages, Hkv, page, ...] with the rows that stay moved to the
    front; kept [n_seq, Hkv, budget]; new lengths."""
    page = weights.shape[2]
    out = [np.array(p) for p in pages]
    kept = np.full((len(kv_lens), weights.shape[1], budget), -1, np.int32)
    for b, n in enumerate(kv_lens):
        at = np.arange(n)
        where = np.asarray(table[b])[at // page], at % page
        for h in range(weights.shape[1]):
            keep = keep_positions(weights[where[0], h, where[1]], budget, sinks, recent)
            kept[b, h, :len(keep)] = keep
            for o, p in zip(out, pages):
                o[where[0][:len(keep)], h, where[1][:len(keep)]] = p[where[0][keep], h, where[1][keep]]
    return out, kept, np.minimum(kv_lens, budget)
