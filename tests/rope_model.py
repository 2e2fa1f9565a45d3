"""Rotary positions in 64 bits, from the definition: the oracle of the rotation tests.

Angles p f are reduced exactly, with integers: f is a rational number, and 1/(2 pi)
is carried to 200 bits, so a far position loses nothing."""
import math
from fractions import Fraction

import numpy as np


def _pi(bits: int) -> int:
    """pi 2^bits by Machin's formula, in integers."""
    def atan_inv(n):
        one = (1 << (bits + 16)) // n
        total, k, sign = 0, 1, 1
        while one:
            total += sign * (one // k)
            one //= n * n
            k += 2
            sign = -sign
        return total
    return (4 * (4 * atan_inv(5) - atan_inv(239))) >> 16


_INV_TWO_PI = Fraction(1 << 200, 2 * _pi(200))


def angles(positions, freqs):
    """p f modulo one turn, in radians, [T, pairs] float64 (the exact value rounded once)."""
    out = np.empty((len(positions), len(freqs)))
    for i, f in enumerate(freqs):
        turn = Fraction(float(f)) * _INV_TWO_PI
        num, den = turn.numerator, turn.denominator
        for t, p in enumerate(positions):
            out[t, i] = 2.0 * math.pi * float(Fraction((int(p) * num) % den, den))
    return out


def frequencies(r, base=10000.0, scaling=0, factor=1.0, original=0.0, low=0.0, high=0.0):
    """One pair at a time: 0 plain, 1 linear, 2 base, 3 parts."""
    fs = []
    for i in range(r // 2):
        if scaling == 2:
            b = base * factor ** (r / (r - 2))
            f = math.exp(-2 * i / r * math.log(b))
        else:
            f = math.exp(-2 * i / r * math.log(base))
        if scaling == 1:
            f = f / factor
        if scaling == 3:
            turns = original / (2 * math.pi / f)
            if turns <= low:
                f = f / factor
            elif turns < high:
                g = (turns - low) / (high - low)
                f = (1 - g) * f / factor + g * f
        fs.append(f)
    return fs


def rotate(x, positions, freqs, layout, magnitude=1.0, inverse=False):
    """x [T, H, D] float64 -> rotated; layout 0: halves, 1: interleaved."""
    a = angles(positions, freqs)
    c, s = magnitude * np.cos(a)[:, None], magnitude * np.sin(a)[:, None]
    if inverse:
        s = -s
    n = len(freqs)
    first = np.arange(n) if layout == 0 else 2 * np.arange(n)
    second = first + n if layout == 0 else first + 1
    y = x.copy()
    y[..., first] = x[..., first] * c - x[..., second] * s
    y[..., second] = x[..., first] * s + x[..., second] * c
    return y


def slack(x, positions, freqs, layout, magnitude=1.0):
    """How far an fp32 rotation may be from rotate() before its output is rounded: per element
    m (|a| + |b|) times
      the angle: 2^-32 of a turn, its fp32 value (half an ulp of at most pi), and the frequency
        as a 53-bit fraction of a turn, p f 2^-52: together 2.6 2^-24 + p f 2^-52;
      cos and sin to 2 ulp (2 2^-23) and the magnitude's product (2^-24);
      two products and a sum (2 2^-24);
    which is under 16 2^-24 + p f 2^-52.  Pass-through elements have none."""
    n = len(freqs)
    first = np.arange(n) if layout == 0 else 2 * np.arange(n)
    second = first + n if layout == 0 else first + 1
    far = np.abs(np.asarray(positions, dtype=np.float64))[:, None] * np.asarray(freqs)[None]
    unit = (16 * 2.0 ** -24 + far * 2.0 ** -52)[:, None]
    y = np.zeros_like(x)
    both = magnitude * (np.abs(x[..., first]) + np.abs(x[..., second])) * unit
    y[..., first] = both
    y[..., second] = both
    return y


BF16_HALF = 2.0 ** -8         # half a step of bf16, relative


def check_bf16(got, want, slack_, where=""):
    """A bf16 output: the fp32 slack, then one rounding (subnormals: half of 2^-133)."""
    tol = slack_ + (np.abs(want) + slack_) * BF16_HALF + 2.0 ** -134
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (where, int(bad.sum()), float(np.abs(got - want)[bad].max()))
