"""The 4-bit cache at the ends of its types' ranges: CUDA path vs the fp64 oracle.

Tolerances are those of test_kv4_gpu.py and test_retain_gpu.py, with what a test
adds to them derived beside it.
"""
import numpy as np
import pytest
import torch

import oracle
import test_paged_gpu as paged
from helpers import to64
from test_kv4_gpu import check4, exact4, four, largest, pack4, parts4  # noqa: F401
from test_paged_gpu import widen

pytestmark = pytest.mark.gpu


FEW = [([(1, 3), (2, 2), (1, 1), (1, 5)], 16, 4, 2), ([(1, 3), (1, 5), (2, 4)] * 12, 5000, 4, 2),
       ([(1, 5)], 16, 12, 1)]
CHUNK = [([(20, 20), (1, 4)], 16, 4, 2)]


@pytest.mark.parametrize("amp,lens,reach,Hq,Hkv", [
    (2.0 ** e, *case) for e in (123, 119, -116, -122) for case in FEW + (CHUNK if e < 120 else [])])
@pytest.mark.parametrize("d", [64, 96, 128])
def test_far_values_of_bf16(four, amp, lens, reach, Hq, Hkv, d):
    """Values up to a fifth of bf16's largest number, whose scales pass 2^121, and
    least ones: finite, and as precise as others.  Scores are all but equal, so that sums
    of 5 values (20 of the smaller ones) stay in the range of fp32."""
    x = widen(paged.make(lens, Hq, Hkv, d, 32, "bf16", seed=d, amp=2.0 ** -6), reach)
    x["v4"] = pack4(x["v"] * amp)
    s = parts4(x["v4"], torch.bfloat16)[0]
    if amp == 2.0 ** 123:
        assert float(s[torch.isfinite(s)].max()) > 2.0 ** 121
    o, lse = paged.run(four, x, True)
    assert four.poll_status() == (0, 0)
    check4(x, o, lse, True)


def weights_with(attn, x, causal, scale, n_bits=4):
    """kv_weights over the keys k4 of x (or its 16-bit keys k) at a scale, from weights of
    1, against the oracle.  The tolerance is that of test_retain_gpu.py, with
    * the exponential of a score's error (scores reach 10^4 here);
    * n 2^-126: a term below 2^-126 is a subnormal number, which fp32 holds to 2^-149 and
      the exponential may take for 0;
    * 2^-24 of the weight for each of the passes of 64 rows that add to it."""
    dt, args = x["q"].dtype, (x["table"].cpu().numpy(), x["cu"].cpu().numpy(), x["kv"].cpu().numpy(), causal, scale)
    pages = x["k4"] if n_bits == 4 else x["k"]
    k = to64(exact4(pages, dt)) if n_bits == 4 else to64(pages)
    _, L, _, big = oracle.attention_paged(to64(x["q"]), k, np.nan_to_num(to64(x["v"])), *args)
    lse = torch.tensor(L, dtype=torch.float32).cuda()
    one = torch.ones(pages.shape[:3], device="cuda")
    ref, new = oracle.weights_paged(to64(x["q"]), k, to64(lse), to64(one), *args)
    got = to64(attn.kv_weights(x["q"], pages, x["table"], x["cu"], x["kv"], lse, one, x["max_q"], causal=causal,
                               scale=scale))
    if n_bits == 4:
        s, m, _ = parts4(pages, dt)
        err = 48 * 2.0 ** -24 * largest(x, causal, scale, m.abs() + 15 * s)
    else:
        err = k.shape[3] * 2.0 ** -24 * largest(x, causal, scale, pages.double().abs())
    L = np.max(np.abs(L), where=np.isfinite(L), initial=0.0) + big
    n = x["max_q"] * (x["q"].shape[0] // k.shape[1])
    tol = (np.expm1(err + 2 * L * 2.0 ** -24) + 2.0 ** -21 + n * 2.0 ** -24) * new
    tol += -(-n // 64) * 2.0 ** -24 * np.abs(ref) + n * 2.0 ** -126
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= tol).all(), float(np.max(np.abs(got - ref) - tol))


@pytest.mark.parametrize("lens,reach", [([(1, 1), (2, 64)], 16), ([(1, 70), (1, 1)] * 12, 5000),
                                        ([(40, 70), (33, 33)], 16)])
@pytest.mark.parametrize("q_amp,scale", [(2.0 ** -60, 2.0 ** -100), (1.0, 2.0 ** -125), (2.0 ** -110, 0.0625),
                                         (2.0 ** -60, 2.0 ** -30)])
def test_small_scales_and_large_keys(four, lens, reach, q_amp, scale):
    """Scales and queries so small that their product is a subnormal number, or none,
    beside keys near the largest that are allowed (2^100): the scores are all but 0."""
    x = widen(paged.make(lens, 4, 2, 128, 32, "bf16", seed=113), reach)
    x["k4"], x["q"] = pack4(x["k"].abs() * 2.0 ** 97), x["q"].abs() * q_amp
    o, lse = paged.run(four, x, True, scale=scale)
    check4(x, o, lse, True, scale)
    weights_with(four, x, True, scale)
    assert four.poll_status() == (0, 0)


def one_channel(dtype, top, least, amp, n_new, keys, Hq=2):
    """Queries of one large channel, which no key has, and a small odd one at 33; keys of
    that channel alone, up to amp."""
    x = paged.make([(n_new, keys)], Hq, 1, 64, 16, dtype, seed=1)
    q, k = torch.zeros_like(x["q"]), torch.where(torch.isnan(x["k"]), x["k"], x["k"].new_zeros(()))
    q[:, :, 0], q[:, :, 33] = top, least
    for j in range(keys):
        k[int(x["table"][0, j // 16]), :, j % 16, 33] = amp * (j % 3) / 2
    x["q"], x["k4"] = q, pack4(k)
    x["v4"] = pack4(x["v"])
    return x


def lse_error(x, lse, scale):
    args = x["table"].cpu().numpy(), x["cu"].cpu().numpy(), x["kv"].cpu().numpy(), False, scale
    k = to64(exact4(x["k4"], x["q"].dtype))
    _, L, _, big = oracle.attention_paged(to64(x["q"]), k, np.nan_to_num(to64(x["v"])), *args)
    rounding = 2.0 ** -20 + int(x["kv"].max()) * 2.0 ** -24 + 64 * 2.0 ** -24 * big + 2.0 ** -23 * np.abs(L)
    return np.max(np.abs(to64(lse) - L) - rounding), L


@pytest.mark.parametrize("reach", [16, 5000])
@pytest.mark.parametrize("dtype,top,least,amp,share", [
    ("bf16", 1.0, 1.5 * 2.0 ** -29, 2.0 ** 30, 2.0 ** -34), ("bf16", 2.0 ** -40, 1.5 * 2.0 ** -74, 2.0 ** 74, 2.0 ** -34),
    ("fp16", 2.0 ** 15, 1.5 * 2.0 ** -14, 2.0 ** 14, 2.0 ** -30)])
def test_queries_of_a_wide_range_in_few_rows(four, reach, dtype, top, least, amp, share):
    """A channel of a query is off by at most the share of its row's largest that the
    header states, whatever the keys."""
    x = widen(one_channel(dtype, top, least, amp, 1, 3), reach)
    _, lse = paged.run(four, x, False, scale=1.0)
    error, L = lse_error(x, lse, 1.0)
    assert error <= share * top * amp, error
    # the weights: each exp(s - lse) by that in the score
    one = torch.zeros(x["k4"].shape[:3], device="cuda")
    exact = torch.tensor(L, dtype=torch.float32).cuda()
    four.kv_weights(x["q"], x["k4"], x["table"], x["cu"], x["kv"], exact, one, 1, scale=1.0)
    got = torch.stack([one[int(x["table"][0, 0]), 0, j] for j in range(3)]).double().cpu().numpy()
    ref = 2 * np.exp(least * amp * np.arange(3) / 2 - L[0, 0])
    assert (np.abs(got - ref) <= np.expm1(share * top * amp + 2.0 ** -18) * ref).all(), (got, ref)
    assert four.poll_status() == (0, 0)


@pytest.mark.parametrize("dtype,big,small", [("bf16", 2.0 ** 27, 1.5 * 2.0 ** -4), ("bf16", 2.0 ** 27, 1.5 * 2.0 ** -5),
                                             ("fp16", 2.0 ** 12, 1.5 * 2.0 ** -19)])
def test_keys_of_a_wide_range_in_chunks(four, dtype, big, small):
    """Among 32 cached positions one of a scale of `big`, in channels that the queries do not
    have, and others of `small`: their channels are off by at most 2^-30 of the
    largest.  (s / 16, or in fp16 its upper bits and what they leave over 16, is rounded
    to 2^-25 at worst, times 16 |c - 8|: 2^-18, twice, where the largest of 8 s and
    |m + 8 s|, at most 16/15 of the largest value, is brought to 2^14.)"""
    x = one_channel(dtype, 0.0, 1.0 if dtype == "bf16" else 2.0 ** 15, 15 * small, 40, 40, Hq=1)
    rows = exact4(x["k4"], x["q"].dtype)
    rows[int(x["table"][0, 0]), :, 1, :32] = 15 * big * (torch.arange(32, device="cuda") % 2)
    x["k4"] = pack4(rows.to(x["q"].dtype))
    scale = 1.0 if dtype == "bf16" else 2.0 ** -2
    _, lse = paged.run(four, x, False, scale=scale)
    assert four.poll_status() == (0, 0)
    error, _ = lse_error(x, lse, scale)
    assert error <= 2.0 ** -30 * 15 * big * float(x["q"].max()) * scale + 2.0 ** -20, error


@pytest.mark.parametrize("lens,reach", [([(1, 700), (2, 64)], 16), ([(40, 700), (33, 64)], 16), ([(1, 70)] * 40, 16)])
@pytest.mark.parametrize("k_amp,q_amp", [(2.0 ** 40, 2.0 ** -40), (2.0 ** -60, 2.0 ** 60), (2.0 ** -70, 2.0 ** -40),
                                         (2.0 ** 17, 2.0 ** -17)])
def test_weights_of_far_exponents(four, lens, reach, k_amp, q_amp):
    x = widen(paged.make(lens, 4, 2, 128, 32, "bf16", seed=107), reach)
    x["k4"], x["q"] = pack4(x["k"] * k_amp), x["q"] * q_amp
    weights_with(four, x, True, 128 ** -0.5)
    assert four.poll_status() == (0, 0)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp16", 64), ("bf16", 96)])
@pytest.mark.parametrize("lens", [[(1, 700), (2, 64)], [(40, 700), (33, 64)]])
@pytest.mark.parametrize("scale", [0.01, 0.3, 1.0])
@pytest.mark.parametrize("n_bits", [4, 16])
def test_weights_at_other_scales(four, dtype, d, lens, scale, n_bits):
    """The scale is the caller's, in either cache."""
    x = paged.make(lens, 4, 2, d, 32, dtype, seed=5)
    x["k4"] = pack4(x["k"])
    weights_with(four, x, True, scale, n_bits)
    assert four.poll_status() == (0, 0)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp16", 64), ("bf16", 96)])
def test_weights_of_a_key_that_stands_for_nan(four, dtype, d):
    """A group of NaN makes the weight of its own position NaN, and no other's; in a
    position that no row sees it reaches nothing."""
    lens = [(3, 90), (1, 40), (20, 70)]
    x = paged.make(lens, 4, 2, d, 16, dtype, seed=31)
    x["k4"] = pack4(x["k"])
    args = x["table"].cpu().numpy(), x["cu"].cpu().numpy(), x["kv"].cpu().numpy(), True, d ** -0.5
    L = oracle.attention_paged(to64(x["q"]), to64(exact4(x["k4"], x["q"].dtype)), np.nan_to_num(to64(x["v"])),
                               *args)[1]
    lse = torch.tensor(L, dtype=torch.float32).cuda()

    def weights(k):
        w = torch.ones(k.shape[:3], device="cuda")
        four.kv_weights(x["q"], k, x["table"], x["cu"], x["kv"], lse, w, x["max_q"], causal=True)
        return w

    clean = weights(x["k4"])
    k, table, hit = x["k4"].clone(), x["table"].tolist(), torch.zeros_like(clean, dtype=torch.bool)
    for b, at, head in ((0, 17, 0), (1, 39, 1), (2, 3, 1), (2, 69, 0)):
        k[table[b][at // 16], head, at % 16, d // 2:d // 2 + 4] = 0xFF
        hit[table[b][at // 16], head, at % 16] = True
    got = weights(k)
    assert four.poll_status() == (0, 0)
    assert torch.isnan(got[hit]).all()
    assert torch.equal(got[~hit], clean[~hit])


@pytest.mark.parametrize("n_bits", [4, 16])
@pytest.mark.parametrize("lens,Hq,Hkv", [([(700, 700)], 4, 1), ([(513, 900), (1, 40)], 2, 2), ([(1100, 1100)], 1, 1)])
def test_weights_of_whole_prompts(four, n_bits, lens, Hq, Hkv):
    """Many passes over the keys: every further 64 rows of a head add to the same weights."""
    x = paged.make(lens, Hq, Hkv, 64, 32, "bf16", seed=41)
    x["k4"] = pack4(x["k"])
    weights_with(four, x, True, 0.125, n_bits)
    assert four.poll_status() == (0, 0)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("lens,reach,Hq,Hkv", [([(1, 1)] * 3, 16, 4, 2), ([(1, 1)] * 30, 5000, 2, 1),
                                               ([(1, 1)] * 3, 16, 12, 1)])
@pytest.mark.parametrize("shift", [0.0, 30.0])
def test_values_of_one_key(four, dtype, d, lens, reach, Hq, Hkv, shift):
    """O of a sequence of one key is its value: P is 1 but for 2^-20, so that what is left
    is a rounding of m + c s, u |O|, and none of c s or m by themselves, which are both
    far larger than a value in the middle of its group."""
    x = widen(paged.make(lens, Hq, Hkv, d, 16, dtype, seed=d), reach)
    x["v4"] = pack4(x["v"] + shift)
    o, lse = paged.run(four, x, True)
    assert four.poll_status() == (0, 0)
    s, m, c = (t.cpu().numpy() for t in parts4(x["v4"], x["q"].dtype))
    u = torch.finfo(x["q"].dtype).eps / 2
    for b, page in enumerate(x["table"][:, 0].tolist()):
        for h in range(Hq):
            at = page, h // (Hq // Hkv), 0
            want, got = (m + c * s)[at], to64(o)[h, b]
            assert (np.abs(got - want) <= (u + 2.0 ** -20) * (1 + u) * np.abs(want)).all()
