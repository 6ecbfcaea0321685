"""fp64 CPU oracle of rotary positions, the append to a paged key/value cache
and attention over it.

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle/``: plain definitions, a
loop per sequence, head and page, sharing nothing with the CUDA path.
"""
from __future__ import annotations

from typing import Optional, Tuple

import numpy as np

from .attention import masked_softmax, scores

__all__ = ["rotary", "paged_rows", "append_paged", "attention_paged"]


def rotary(x: np.ndarray, positions: np.ndarray, inv_freq: np.ndarray, axis: np.ndarray,
           interleaved: bool, inverse: bool = False) -> np.ndarray:
    """x [..., N, d] turned: channel pair p of row n by positions[axis[p], n]
    * inv_freq[p], as the complex product (x_a + i x_b) e^{i angle}."""
    x = np.asarray(x, np.float64)
    half = len(inv_freq)
    ang = np.asarray(positions, np.float64)[np.asarray(axis)].T * np.asarray(inv_freq, np.float64)
    a = np.arange(half) * 2 if interleaved else np.arange(half)
    b = a + 1 if interleaved else a + half
    z = (x[..., a] + 1j * x[..., b]) * np.exp((-1j if inverse else 1j) * ang)
    y = x.copy()
    y[..., a], y[..., b] = z.real, z.imag
    return y


def paged_rows(pages: np.ndarray, table_row: np.ndarray, n: int) -> np.ndarray:
    """Rows 0..n-1 of one sequence: [Hkv, n, d] from [n_pages, Hkv, page, d]."""
    page = pages.shape[2]
    out = np.zeros((pages.shape[1], n, pages.shape[3]))
    for p in range(n):
        out[:, p] = pages[table_row[p // page], :, p % page]
    return out


def append_paged(new: np.ndarray, pages: np.ndarray, table: np.ndarray, cu: np.ndarray,
                 kv_lens: np.ndarray) -> np.ndarray:
    """pages with new [Hkv, total, d] written at the end of every sequence."""
    pages = np.array(pages)
    page = pages.shape[2]
    for b in range(len(kv_lens)):
        n = int(cu[b + 1] - cu[b])
        for i in range(n):
            p = int(kv_lens[b]) - n + i
            pages[table[b, p // page], :, p % page] = new[:, cu[b] + i]
    return pages


def attention_paged(q: np.ndarray, k_pages: np.ndarray, v_pages: np.ndarray, table: np.ndarray,
                    cu: np.ndarray, kv_lens: np.ndarray, causal: bool, scale: float,
                    ) -> Tuple[np.ndarray, np.ndarray, np.ndarray, Optional[float]]:
    """O, LSE, A = sum_j P_ij |v_j| (what bounds the rounding of P) and the
    largest |score| of packed new tokens q [H, total, d].  Rows outside every
    sequence are NaN; a row that sees no key has O = 0, LSE = -inf."""
    q = np.asarray(q, np.float64)
    H, total, d = q.shape
    group = H // k_pages.shape[1]
    O, A = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    L = np.full((H, total), np.nan)
    big = 0.0
    for b in range(len(kv_lens)):
        s0, s1, nk = int(cu[b]), int(cu[b + 1]), int(kv_lens[b])
        n = s1 - s0
        if n == 0:
            continue
        k, v = paged_rows(k_pages, table[b], nk), paged_rows(v_pages, table[b], nk)
        j = np.arange(nk)[None, :]
        allowed = j <= np.arange(n)[:, None] + nk - n if causal else np.ones((n, nk), bool)
        some = allowed.any(axis=1)
        for h in range(H):
            O[h, s0:s1], A[h, s0:s1], L[h, s0:s1] = 0.0, 0.0, -np.inf
            if not some.any():
                continue
            S = scores(q[h, s0:s1][some], k[h // group], scale)
            big = max(big, float(np.max(np.abs(S))))
            P, lse = masked_softmax(S, allowed[some])
            rows = np.arange(s0, s1)[some]
            O[h, rows], A[h, rows], L[h, rows] = P @ v[h // group], P @ np.abs(v[h // group]), lse
    return O, L, A, big
