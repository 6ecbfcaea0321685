"""The 4-bit cache without a GPU: what the library refuses on the host, and the
oracle of its format pinned."""
import ctypes

import numpy as np
import pytest
import torch

import exact_attention_75_gb300 as attn
import oracle
from test_paged_args import (APPEND, APPEND_APART, INVALID, P, P1, P2, P3, P4, PAGED, UNSUPPORTED, L,  # noqa: F401
                             test_append_refusals, test_append_refuses_turned_queries_over_inputs,
                             test_paged_refusals)

WIDE = [(dict(d=192), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(d=32, rot=16), UNSUPPORTED)]


@pytest.mark.parametrize("change,want", test_append_refusals.pytestmark[0].args[1] + WIDE)
def test_append4_refusals(L, change, want):  # noqa: F811
    for base in (APPEND, APPEND_APART):
        assert L.attn_append_kv4(*dict(base, **change).values()) == want


@pytest.mark.parametrize("change", test_append_refuses_turned_queries_over_inputs.pytestmark[0].args[1])
def test_append4_refuses_turned_queries_over_inputs(L, change):  # noqa: F811
    assert L.attn_append_kv4(*dict(APPEND_APART, **change).values()) == INVALID


@pytest.mark.parametrize("change,want", test_paged_refusals.pytestmark[0].args[1])
def test_paged4_refusals(L, change, want):  # noqa: F811
    assert L.attn_fwd_paged4(*dict(PAGED, **change).values()) == want


READ = dict(kp=P, vp=P1, k=P2, v=P3, table=P4, cu=P4, kv=P4, n_seq=2, total=9, n_pages=8, page=16, max_pages=4,
            Hkv=2, d=64, dtype=0, stream=None)
BAD = ctypes.c_void_p(0x10008)


@pytest.mark.parametrize("change,want", [
    (dict(kp=BAD), INVALID), (dict(vp=None), INVALID), (dict(k=None), INVALID), (dict(v=BAD), INVALID),
    (dict(k=P3), INVALID), (dict(k=P), INVALID), (dict(v=P1), INVALID), (dict(v=P), INVALID),
    (dict(k=P1), INVALID), (dict(table=None), INVALID), (dict(cu=None), INVALID), (dict(kv=None), INVALID),
    (dict(n_seq=0), INVALID), (dict(total=0), INVALID), (dict(n_pages=0), INVALID), (dict(max_pages=0), INVALID),
    (dict(page=48), UNSUPPORTED), (dict(Hkv=0), INVALID), (dict(d=192), UNSUPPORTED), (dict(d=80), UNSUPPORTED),
    (dict(dtype=2), INVALID), (dict(total=1 << 30), INVALID), (dict(max_pages=1 << 26), INVALID)])
def test_read4_refusals(L, change, want):  # noqa: F811
    assert L.attn_read_kv4(*dict(READ, **change).values()) == want


def test_binding_refuses_cpu_tensors():
    q = torch.zeros(2, 5, 64, dtype=torch.bfloat16)
    pages = torch.zeros(3, 2, 16, 40, dtype=torch.uint8)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        attn.append_kv4(q, q, pages, pages, i(1, 2), i(2), i(1))
    with pytest.raises(ValueError):
        attn.read_kv4(pages, pages, i(1, 2), i(2), i(1), 5)
    with pytest.raises(ValueError):
        attn.fwd_paged4(q, pages, pages, i(1, 2), i(2), i(1), 1)


# ------------------------------------------------------------------ oracle ---

def test_oracle_of_16_bit_numbers():
    """Against torch: every finite number both ways, halves to even, overflow."""
    for bf16, dt in ((True, torch.bfloat16), (False, torch.float16)):
        bits = np.arange(65536, dtype=np.uint16)
        t = torch.from_numpy(bits.view(np.int16)).view(dt)
        want = t.double().numpy()
        got = oracle.from16(bits, bf16)
        assert np.array_equal(got, want, equal_nan=True)
        g = np.random.default_rng(0)
        x = np.concatenate([g.standard_normal(4000), g.standard_normal(4000) * 10.0 ** g.integers(-9, 9, 4000),
                            (want[:-1] + want[1:])[np.isfinite(want[:-1] + want[1:])] / 2]).astype(np.float32)
        want = torch.from_numpy(x).to(dt).view(torch.int16).numpy().view(np.uint16)
        assert np.array_equal(oracle.to16(x, bf16), want)


@pytest.mark.parametrize("bf16", [False, True])
def test_oracle_of_the_format(bf16):
    """Hand-made rows, the error bound of half a step, one-valued groups."""
    d = 64
    row = np.zeros(40, np.uint8)
    row[0], row[31] = 0x3A, 0xF0  # channels 0, 1: 10, 3; channels 62, 63: 0, 15
    row[32:] = oracle.to16(np.array([0.5, -2.0, 0.25, 1.0]), bf16).view(np.uint8)
    got = oracle.values4(row, bf16)
    assert got[0] == 3.0 and got[1] == -0.5 and got[2] == -2.0 and got[62] == 1.0 and got[63] == 4.75
    g = np.random.default_rng(1)
    x = oracle.from16(oracle.to16(g.standard_normal((50, d)) * 3 + g.standard_normal(d), bf16), bf16)
    x[0], x[1, :32] = 1.5, -0.75
    rows = oracle.quantize4(x, bf16)
    back = oracle.values4(rows, bf16)
    assert np.array_equal(back[0], x[0]) and np.array_equal(back[1, :32], x[1, :32])
    s = oracle.from16(np.ascontiguousarray(rows[:, d // 2:]).view("<u2")[:, ::2], bf16).repeat(32, 1)
    u = 2.0 ** (-9 if bf16 else -12)
    assert (np.abs(back - x) <= s / 2 * (1 + 2 ** -15) + 15 * s * 2 * u).all()
    # brute force: no other code is nearer (but where the top is cut)
    for r in range(10):
        for ch in range(d):
            near = min(abs(x[r, ch] - (back[r, ch] + j * s[r, ch])) for j in range(-15, 16))
            assert abs(x[r, ch] - back[r, ch]) <= near + 15 * s[r, ch] * 2 * u + 1e-12


def test_oracle_of_groups_that_are_not_finite():
    for bf16 in (False, True):
        for bad in (np.inf, -np.inf, np.nan):
            x = np.ones((1, 64))
            x[0, 3] = bad
            back = oracle.values4(oracle.quantize4(x, bf16), bf16)
            assert np.isnan(back[0, :32]).all() and (back[0, 32:] == 1.0).all()
