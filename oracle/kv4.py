"""CPU oracle of the rows of a key/value cache held in 4 bits.

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle/``: the format from its
definition, a loop per group, sharing nothing with the CUDA path.  16-bit
numbers are handled by their bits, since numpy has no bfloat16.
"""
from __future__ import annotations

import numpy as np

__all__ = ["to16", "from16", "quantize4", "values4"]

GROUP = 32


def to16(x: np.ndarray, bf16: bool) -> np.ndarray:
    """Bits of the nearest 16-bit numbers (ties to even) of float32 x."""
    x = np.asarray(x, np.float32)
    if not bf16:
        with np.errstate(over="ignore"):
            return x.astype(np.float16).view(np.uint16)
    b = x.view(np.uint32)
    up = (b + 0x7FFF + (b >> 16 & 1)) >> 16
    return np.where(np.isnan(x), 0x7FFF, up).astype(np.uint16)


def from16(bits: np.ndarray, bf16: bool) -> np.ndarray:
    """float64 values of 16-bit numbers given by their bits."""
    bits = np.asarray(bits, np.uint16)
    if not bf16:
        return bits.view(np.float16).astype(np.float64)
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def quantize4(x: np.ndarray, bf16: bool) -> np.ndarray:
    """Rows uint8 [..., 5 d / 8] for 16-bit values x [..., d] (as float64)."""
    x = np.asarray(x, np.float32)
    rows = x.reshape(-1, x.shape[-1])
    d = rows.shape[1]
    out = np.zeros((len(rows), d // 2 + d // 8), np.uint8)
    for r, row in enumerate(rows):
        code = np.zeros(d, np.uint8)
        par = []
        for at in range(0, d, GROUP):
            g = row[at:at + GROUP]
            with np.errstate(all="ignore"):
                m = g.min()  # NaN if one is
                s = to16((g.max() - m) / np.float32(15), bf16)
                if not np.isfinite(from16(s, bf16)):
                    par += [0x7FFF, 0x7FFF]
                    continue
                # the largest code must not pass the type's range
                if np.isinf(from16(to16(np.float32(15 * from16(s, bf16) + np.float64(m)), bf16), bf16)):
                    s = np.uint16(s - 1)
                step = np.float32(from16(s, bf16))
                if step > 0:
                    code[at:at + GROUP] = np.minimum(np.rint((g - m) / step), 15)
            par += [int(s), int(to16(m, bf16))]
        out[r, :d // 2] = code[0::2] | code[1::2] << 4
        out[r, d // 2:] = np.array(par, "<u2").view(np.uint8)
    return out.reshape(x.shape[:-1] + (out.shape[1],))


def values4(rows: np.ndarray, bf16: bool) -> np.ndarray:
    """What rows uint8 [..., 5 d / 8] stand for: m + c s, float64 [..., d]."""
    rows = np.asarray(rows, np.uint8)
    d = rows.shape[-1] // 5 * 8
    out = np.zeros(rows.shape[:-1] + (d,))
    par = np.ascontiguousarray(rows[..., d // 2:]).view("<u2")
    for ch in range(d):
        code = rows[..., ch // 2] >> (4 * (ch % 2)) & 15
        s, m = (from16(np.ascontiguousarray(par[..., ch // GROUP * 2 + i]), bf16) for i in (0, 1))
        out[..., ch] = m + code * s
    return out
