"""The oracle of rotary positions and the paged cache, pinned by identities
and brute force (CPU)."""
import math

import numpy as np
import pytest

import oracle


def _freq(rot, axes=1):
    half = rot // 2
    return 10000.0 ** (-np.arange(half) / half), np.arange(half) * axes // half


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_by_hand(interleaved):
    inv, axis = _freq(4, 2)
    x = np.array([[1.0, 2.0, 3.0, 4.0, 5.0]])
    pos = np.array([[2], [700]])
    y = oracle.rotary(x, pos, inv, axis, interleaved)
    for p, ang in enumerate([2 * 1.0, 700 * 0.01]):
        a, b = (2 * p, 2 * p + 1) if interleaved else (p, p + 2)
        assert math.isclose(y[0, a], x[0, a] * math.cos(ang) - x[0, b] * math.sin(ang))
        assert math.isclose(y[0, b], x[0, b] * math.cos(ang) + x[0, a] * math.sin(ang))
    assert y[0, 4] == 5.0


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_scores_depend_on_differences_and_the_inverse_undoes_it(interleaved):
    g = np.random.default_rng(0)
    inv, axis = _freq(16, 3)
    q, k = g.standard_normal((2, 6, 24))
    pos = g.integers(-50, 50, (3, 6))
    turn = lambda x, p: oracle.rotary(x, p, inv, axis, interleaved)  # noqa: E731
    s0 = turn(q, pos) @ turn(k, pos).T
    s1 = turn(q, pos + 37) @ turn(k, pos + 37).T
    assert np.allclose(s0, s1, atol=1e-11)
    assert np.allclose(oracle.rotary(turn(q, pos), pos, inv, axis, interleaved, inverse=True), q)


def test_rotary_backward_is_the_inverse_turn():
    """dL/dx of L = <dy, turn(x)> by central differences."""
    g = np.random.default_rng(1)
    inv, axis = _freq(16, 2)
    x, dy = g.standard_normal((2, 3, 16))
    pos = g.integers(0, 100, (2, 3))
    want = oracle.rotary(dy, pos, inv, axis, False, inverse=True)
    for n, c in [(0, 0), (1, 7), (2, 8), (2, 15)]:
        e = np.zeros_like(x)
        e[n, c] = 1e-6
        diff = np.sum(dy * (oracle.rotary(x + e, pos, inv, axis, False)
                            - oracle.rotary(x - e, pos, inv, axis, False))) / 2e-6
        assert abs(diff - want[n, c]) < 1e-8


@pytest.mark.parametrize("causal", [False, True])
def test_paged_attention_is_dense_attention_over_the_gathered_rows(causal):
    g = np.random.default_rng(2)
    Hq, Hkv, d, page = 4, 2, 8, 4
    lens = [(3, 9), (0, 5), (1, 1), (5, 5)]  # new, keys
    cu = np.concatenate([[0], np.cumsum([n for n, _ in lens])])
    kv = np.array([k for _, k in lens])
    table = g.permutation(16)[:12].reshape(4, 3)
    kp, vp = g.standard_normal((2, 16, Hkv, page, d))
    new_k = g.standard_normal((Hkv, cu[-1] + 2, d))
    kp2 = oracle.append_paged(new_k, kp, table, cu, kv)
    q = g.standard_normal((Hq, cu[-1] + 2, d))
    O, L, A, _ = oracle.attention_paged(q, kp2, vp, table, cu, kv, causal, 0.3)
    assert np.isnan(O[:, cu[-1]:]).all()
    for b, (n, nk) in enumerate(lens):
        if n == 0:
            continue
        rows = slice(cu[b], cu[b + 1])
        k = np.concatenate([kp2[t] for t in table[b]], axis=1)[:, :nk]
        v = np.concatenate([vp[t] for t in table[b]], axis=1)[:, :nk]
        assert np.array_equal(k[:, nk - n:], new_k[:, rows])
        O_ref, L_ref = oracle.attention_kv(q[None, :, rows], k[None], v[None], causal, 0.3, 1)
        assert np.allclose(O[:, rows], O_ref[0, 0]) and np.allclose(L[:, rows], L_ref[0, 0])
    assert (A[:, :cu[-1]] >= np.abs(O[:, :cu[-1]]) - 1e-12).all()


def test_rows_without_a_key():
    q = np.ones((1, 3, 4))
    pages = np.ones((1, 1, 4, 4))
    O, L, _, _ = oracle.attention_paged(q, pages, pages, np.array([[0]]), np.array([0, 3]),
                                        np.array([2]), True, 1.0)
    assert (O[0, 0] == 0).all() and L[0, 0] == -np.inf and np.isfinite(L[0, 1:]).all()
    O, L, _, _ = oracle.attention_paged(q, pages, pages, np.array([[0]]), np.array([0, 3]),
                                        np.array([0]), False, 1.0)
    assert (O == 0).all() and (L == -np.inf).all()
