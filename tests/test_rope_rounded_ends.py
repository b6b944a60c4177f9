"""Frequencies whose ramp begins and ends at whole channels (on the host: no GPU needed).

A channel i turns L f / 2 pi times in L tokens, so the channel that turns r times is n ln(L / 2 pi r) / ln(base), with n
channels in all.  The ramp goes from that of `high` turns, rounded down, to that of `low`, rounded up, both within
0 .. 2 n - 1; parity with released checkpoints' own outputs is unpinned."""
import math

import numpy as np
import pytest

import weight_only_quantization_pack_amd as awq


def ramp(n, base, length, low, high):
    a = math.floor(n * math.log(length / (2 * math.pi * high)) / math.log(base))
    b = math.ceil(n * math.log(length / (2 * math.pi * low)) / math.log(base))
    return min(max(a, 0), 2 * n - 1), min(max(b, 0), 2 * n - 1)


def frequencies(rotary, base, length, factor, low=1.0, high=32.0):
    n = rotary // 2
    a, b = ramp(n, base, length, low, high)
    out = []
    for i in range(n):
        f = base ** (-i / n)
        share = min(1.0, max(0.0, (i - a) / (b - a))) if b > a else float(i > a)      # divided by factor
        out.append(f * (1.0 - share) + f / factor * share)
    return np.array(out)


# fp32 of a 64-bit value: half a step, and the few of 64 bits that powers and logarithms cost
ROUNDING = 2.0 ** -24 + 1e-12


@pytest.mark.parametrize("rotary,base,length,factor,ends", [(64, 10000.0, 4096, 40.0, (10, 23)), (128, 500000.0, 8192, 16.0, None),
                                                            (128, 10000.0, 4096, 16.0, None), (64, 1000000.0, 32768, 4.0, None),
                                                            (32, 10000.0, 262144, 2.0, None), (128, 150000.0, 4096, 32.0, None)])
def test_rounded_ends(rotary, base, length, factor, ends):
    got, magnitude = awq.rope_frequencies(rotary, base, scaling="yarn_rounded", factor=factor, original_length=length, device="cpu")
    got = got.double().numpy()
    want = frequencies(rotary, base, length, factor)
    assert np.all(np.abs(got - want) <= ROUNDING * want)
    assert abs(magnitude - (0.1 * math.log(factor) + 1.0)) <= 2.0 ** -24 * magnitude
    plain = base ** (-np.arange(rotary // 2) * 2.0 / rotary)
    a, b = ramp(rotary // 2, base, length, 1.0, 32.0)
    assert ends is None or (a, b) == ends
    assert np.all(np.abs(got / plain - 1.0)[:a + 1] <= 2 * ROUNDING)            # kept up to the lower end,
    assert np.all(np.abs(got / plain * factor - 1.0)[b:] <= 2 * ROUNDING)       # divided from the upper one on


def test_it_differs_from_ends_that_are_not_rounded():
    """Base 10000, 64 channels, 4096 tokens, factor 40: channel 22 has 12 / 13 of its way behind it with ends 10 and 23, so
    f (1 / 13 + 12 / 13 / 40) = 0.1 f, and 0.9576 of it with 10.47 and 22.51, 0.0663 f: a third less."""
    kw = dict(factor=40.0, original_length=4096.0, device="cpu")
    a, b = (awq.rope_frequencies(64, 10000.0, scaling=s, **kw)[0].numpy() for s in ("yarn_rounded", "yarn"))
    assert np.argmax(np.abs(b / a - 1.0)) == 22 and abs(b[22] / a[22] - 0.0663 / 0.1) < 0.005


@pytest.mark.parametrize("low,high,length", [(1.0, 1.5, 4096.0), (2.0, 2.0000001, 4096.0), (1.0, 32.0, 5.0), (1e-9, 32.0, 4096.0)])
def test_narrow_and_outside(low, high, length):
    """Ends that meet, that lie before the first channel, or behind the last one."""
    got, _ = awq.rope_frequencies(64, 10000.0, scaling="yarn_rounded", factor=8.0, original_length=length, low=low, high=high,
                                  device="cpu")
    want = frequencies(64, 10000.0, length, 8.0, low, high)
    assert np.all(np.abs(got.double().numpy() - want) <= ROUNDING * want)


def test_refused():
    for bad in (dict(factor=0.5), dict(original_length=0.0), dict(low=2.0, high=2.0), dict(low=0.0)):
        with pytest.raises(awq.AwqError):
            awq.rope_frequencies(64, scaling="yarn_rounded", device="cpu", **{**dict(factor=2.0, original_length=4096.0), **bad})
