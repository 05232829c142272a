"""The largest |bf16(act(z))| of many bf16 z is that of one of four of them: the largest
z, the two negative ones on either side of the point where |act| peaks, and a NaN of
negative sign.  Holds for any act whose fp32 value is within the stated error; here
from act in 64 bits at every finite bf16 z."""
import math

import numpy as np
import pytest
from scipy.special import erfc, log_ndtr

PEAK = {"silu": 0x3FA4, "gelu_tanh": 0x3F41, "gelu": 0x3F40}


def act64(act, z):
    """(act(z), by how much a relative error of 1 of the exponential's argument moves it
    relatively: |v| (1 - s(v)); gelu: the share of the tail z^2 / 2 P(-|z|) / P(z))"""
    if act == "gelu":
        return z * np.exp(log_ndtr(z)), z * z / 2 * np.exp(log_ndtr(-np.abs(z)) - log_ndtr(z))
    v = z if act == "silu" else 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    with np.errstate(over="ignore"):
        e = np.exp(-v)
        return z / (1 + e), np.abs(v) * (1 - 1 / (1 + e))


def bf16(x):
    """positive 64-bit values rounded to the nearest bf16, ties to even"""
    m, e = np.frexp(x)
    step = np.ldexp(1.0, np.maximum(e - 8, -133))
    return np.rint(x / step) * step


def bounds(act, bits, sign):
    """bf16 of the smallest and the largest |act| that fp32 may give"""
    z = sign * (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    a, v = act64(act, z)
    a = np.abs(a)
    err = (3 * v + 8) * 2.0 ** -24 + (2.0 ** -18 if act == "gelu" else 0.0)
    err = np.minimum(err, 1.0)
    keep = a >= 2.0 ** -120            # (below, fp32 results lose digits or are 0)
    lo, hi = bf16(a * (1 - err)), bf16(a * (1 + err))
    return np.where(keep, lo, 0.0), np.where(keep, hi, 0.0), keep


@pytest.mark.parametrize("act", list(PEAK))
def test_one_of_the_keys_has_the_maximum(act):
    peak = PEAK[act]
    up = np.arange(0, 0x7F80, dtype=np.uint32)
    # z >= 0: growing.  z < 0: growing in |z| up to the peak, falling beyond it.
    for bits, sign in ((up, 1.0), (up[:peak + 1], -1.0), (up[peak + 1:][::-1], -1.0)):
        lo, hi, keep = bounds(act, bits, sign)
        before = np.maximum.accumulate(hi)[:-1]
        bad = np.nonzero(keep[1:] & (before > lo[1:]))[0]
        assert bad.size == 0, [hex(int(bits[i + 1])) for i in bad[:8]]


def test_values():
    assert abs(act64("gelu", np.float64(-3.0))[0] + 3.0 * 0.5 * erfc(3 / math.sqrt(2))) < 1e-15
    assert list(bf16(np.array([1.0, 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8]))) == [1.0, 1.0, 1 + 2.0 ** -6]
