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
    least ones: finite, and as precise as others.  (In few rows c s / 16 is rounded to a
    bf16 number, which may be subnormal: half a step of those times 16, 2^-130, a
    value.)  Scores are all but equal, so that sums of 5 values (20 of the smaller ones)
    stay in the range of fp32."""
    x = widen(paged.make(lens, Hq, Hkv, d, 32, "bf16", seed=d, amp=2.0 ** -6), reach)
    x["v4"] = pack4(x["v"] * amp)
    s = parts4(x["v4"], torch.bfloat16)[0]
    if amp == 2.0 ** 123:
        assert float(s[torch.isfinite(s)].max()) > 2.0 ** 121
    o, lse = paged.run(four, x, True)
    assert four.poll_status() == (0, 0)
    check4(x, o, lse, True)


def weights_with(attn, x, causal, scale):
    """kv_weights over the 4-bit keys k4 of x at a scale, from weights of 1, against the
    oracle.  The tolerance is that of test_retain_gpu.py, with the exponential of a
    score's error (scores reach 10^4 here), and n 2^-126: a term below 2^-126 is a
    subnormal number, which fp32 holds to 2^-149 and the exponential may take for 0."""
    dt, args = x["q"].dtype, (x["table"].cpu().numpy(), x["cu"].cpu().numpy(), x["kv"].cpu().numpy(), causal, scale)
    k = to64(exact4(x["k4"], dt))
    _, L, _, big = oracle.attention_paged(to64(x["q"]), k, np.nan_to_num(to64(x["v"])), *args)
    lse = torch.tensor(L, dtype=torch.float32).cuda()
    one = torch.ones(x["k4"].shape[:3], device="cuda")
    ref, new = oracle.weights_paged(to64(x["q"]), k, to64(lse), to64(one), *args)
    got = to64(attn.kv_weights(x["q"], x["k4"], x["table"], x["cu"], x["kv"], lse, one, x["max_q"], causal=causal,
                               scale=scale))
    s, m, _ = parts4(x["k4"], dt)
    err = 48 * 2.0 ** -24 * largest(x, causal, scale, m.abs() + 15 * s)
    L = np.max(np.abs(L), where=np.isfinite(L), initial=0.0) + big
    n = x["max_q"] * (x["q"].shape[0] // k.shape[1])
    tol = (np.expm1(err + 2 * L * 2.0 ** -24) + 2.0 ** -21 + n * 2.0 ** -24) * new
    tol += 2.0 ** -24 * np.abs(ref) + n * 2.0 ** -126
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
