"""Attention weights and eviction without a GPU: what the library refuses on the
host, and the oracle pinned."""
import ctypes
import math

import numpy as np
import pytest
import torch

import exact_attention_75_gb300 as attn
import oracle
from test_paged_args import BAD, INVALID, L, P, P1, P2, P3, P4, UNSUPPORTED  # noqa: F401

P5 = ctypes.c_void_p(6 << 20)
WEIGHTS = dict(q=P, kp=P1, lse=P2, w=P3, table=P4, cu=P4, kv=P4, n_seq=2, max_q=4, total=9, n_pages=8, page=16,
               max_pages=4, Hq=4, Hkv=2, d=64, bits=16, causal=1, scale=0.1, dtype=1, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(q=BAD), INVALID), (dict(kp=None), INVALID), (dict(lse=BAD), INVALID), (dict(w=None), INVALID),
    (dict(w=P2), INVALID), (dict(w=P), INVALID), (dict(w=P1), INVALID), (dict(table=None), INVALID),
    (dict(cu=None), INVALID), (dict(kv=None), INVALID), (dict(max_q=0), INVALID), (dict(max_q=10), INVALID),
    (dict(n_seq=0), INVALID), (dict(n_pages=0), INVALID), (dict(page=48), UNSUPPORTED), (dict(Hq=5), INVALID),
    (dict(Hq=258), UNSUPPORTED), (dict(d=192), UNSUPPORTED), (dict(d=80), UNSUPPORTED), (dict(bits=8), INVALID),
    (dict(causal=2), INVALID), (dict(scale=0.0), INVALID), (dict(scale=math.nan), INVALID),
    (dict(scale=math.inf), INVALID), (dict(dtype=3), INVALID), (dict(max_pages=1 << 26), INVALID)])
def test_weights_refusals(L, change, want):  # noqa: F811
    for bits in (4, 16):
        assert L.attn_kv_weights(*dict(dict(WEIGHTS, bits=bits), **change).values()) == want


EVICT = dict(kp=P, vp=P1, w=P2, table=P3, kv=P4, kept=P5, lens=ctypes.c_void_p(7 << 20), n_seq=2, n_pages=8, page=16,
             max_pages=4, Hkv=2, d=64, bits=16, budget=20, sinks=4, recent=10, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(kp=BAD), INVALID), (dict(vp=None), INVALID), (dict(vp=P), INVALID), (dict(w=None), INVALID),
    (dict(w=P), INVALID), (dict(w=P1), INVALID), (dict(table=None), INVALID), (dict(kv=None), INVALID),
    (dict(kept=None), INVALID), (dict(lens=None), INVALID), (dict(lens=P4), INVALID), (dict(kept=P4), INVALID),
    (dict(lens=P5), INVALID), (dict(kept=P3), INVALID), (dict(lens=P3), INVALID), (dict(n_seq=0), INVALID),
    (dict(n_pages=0), INVALID), (dict(max_pages=0), INVALID), (dict(Hkv=0), INVALID), (dict(page=20), UNSUPPORTED),
    (dict(d=80), UNSUPPORTED), (dict(d=192, bits=4), UNSUPPORTED), (dict(bits=2), INVALID), (dict(budget=0), INVALID),
    (dict(sinks=-1), INVALID), (dict(recent=-1), INVALID), (dict(sinks=11), INVALID), (dict(budget=13), INVALID),
    (dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1, budget=2 ** 31 - 1), INVALID), (dict(n_seq=1 << 28), INVALID),
    (dict(budget=(1 << 30) + 1), INVALID), (dict(budget=2 ** 31 - 1), INVALID), (dict(kept=P2), INVALID),
    (dict(kept=P), INVALID), (dict(lens=P1), INVALID), (dict(lens=P2), INVALID)])
def test_evict_refusals(L, change, want):  # noqa: F811
    assert L.attn_evict_kv(*dict(EVICT, **change).values()) == want


def test_binding_refuses_cpu_tensors():
    q = torch.zeros(2, 5, 64, dtype=torch.bfloat16)
    pages = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    w, lse = torch.zeros(3, 2, 16), torch.zeros(2, 5)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        attn.kv_weights(q, pages, i(1, 2), i(2), i(1), lse, w, 1)
    with pytest.raises(ValueError):
        attn.evict_kv(pages, pages.clone(), w, i(1, 2), i(1), 5)


# ------------------------------------------------------------------ oracle ---

def test_oracle_weights_are_the_columns_of_the_probabilities():
    """A scalar loop over rows, keys and heads; full attention's weights sum to
    the rows."""
    g = np.random.default_rng(0)
    Hq, Hkv, page, d = 4, 2, 4, 8
    lens = [(3, 7), (0, 5), (2, 2), (1, 9)]
    cu = np.concatenate([[0], np.cumsum([n for n, _ in lens])])
    kv = [k for _, k in lens]
    table = g.permutation(12).reshape(4, 3)
    k = g.standard_normal((12, Hkv, page, d))
    q = g.standard_normal((Hq, cu[-1], d))
    w = g.random((12, Hkv, page))
    for causal in (False, True):
        _, lse, _, _ = oracle.attention_paged(q, k, k, table, cu, kv, causal, 0.3)
        got, new = oracle.weights_paged(q, k, lse, w, table, cu, kv, causal, 0.3)
        want = w.copy()
        for b, (n, nk) in enumerate(lens):
            for h in range(Hkv):
                for j in range(nk):
                    total = 0.0
                    for i in range(n):
                        if causal and j > i + nk - n:
                            continue
                        for hq in range(h * 2, h * 2 + 2):
                            s = 0.3 * float(q[hq, cu[b] + i] @ k[table[b, j // page], h, j % page])
                            total += math.exp(s - lse[hq, cu[b] + i])
                    at = table[b, j // page], h, j % page
                    if n:
                        want[at] = total + (w[at] if j < nk - n else 0.0)
        assert np.allclose(got, want, rtol=1e-12)
        assert abs(new.sum() - Hq * cu[-1]) < 1e-9


def test_oracle_eviction_by_hand():
    nan = math.nan
    w = np.array([9.0, 1, 5, 5, nan, 0, 5, 2, 7, 1])
    assert oracle.keep_positions(w, 10, 0, 0) == list(range(10))
    assert oracle.keep_positions(w, 3, 0, 0) == [0, 4, 8]  # the NaN counts most, then 9, 7
    assert oracle.keep_positions(w, 5, 0, 0) == [0, 2, 3, 4, 8]  # of three fives the first two
    assert oracle.keep_positions(w, 4, 2, 1) == [0, 1, 4, 9]
    assert oracle.keep_positions(w, 4, 2, 2) == [0, 1, 8, 9]
    pages = np.arange(40).reshape(5, 1, 2, 4)
    weights = np.zeros((5, 1, 2))
    table = np.array([[4, 0, 2]])
    for j, x in enumerate([0.0, 3, 1, 2, 5]):
        weights[table[0, j // 2], 0, j % 2] = x
    out, kept, lens = oracle.evict_paged([pages], weights, table, np.array([5]), 3, 0, 1)
    assert kept.tolist() == [[[1, 3, 4]]] and lens.tolist() == [3]
    rows = oracle.paged_rows(out[0], table[0], 5)[0]
    old = oracle.paged_rows(pages, table[0], 5)[0]
    assert np.array_equal(rows[:3], old[[1, 3, 4]]) and np.array_equal(rows[3:], old[3:])
    assert np.array_equal(out[0][[1, 3]], pages[[1, 3]])
