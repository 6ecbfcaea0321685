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
