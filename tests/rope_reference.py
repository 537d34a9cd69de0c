"""Rotary positions in NumPy and 64 bits, from their definition, for the tests."""

from __future__ import annotations

import numpy as np

U = 2.0 ** -8       # half a step of bf16, relative
HALF_E4M3 = 2.0 ** -4


def frequencies(rot, base=10000.0):
    return base ** (-2.0 * np.arange(rot // 2) / rot)


def split(x, rot, interleaved):
    """The pairs (a, b) of rows [..., d]."""
    if interleaved:
        return x[..., 0:rot:2], x[..., 1:rot:2]
    return x[..., :rot // 2], x[..., rot // 2:rot]


def join(a, b, x, rot, interleaved):
    y = np.array(x)
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = a, b
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = a, b
    return y


def rotate(x, pos, freq, factor=1.0, interleaved=False, back=False):
    """Rows x [..., heads, d] (float64) at positions pos [...]."""
    x = np.asarray(x, dtype=np.float64)
    rot = 2 * len(freq)
    t = np.asarray(pos, dtype=np.float64)[..., None, None] * freq
    c, s = factor * np.cos(t), factor * np.sin(t) * (-1.0 if back else 1.0)
    a, b = split(x, rot, interleaved)
    return join(a * c - b * s, a * s + b * c, x, rot, interleaved)


def slack(x, pos, freq, factor=1.0, interleaved=False, steps=1):
    """What fp32 may be off by before the result is rounded, for each value.

    The angle: turns a position are held to 2^-52 of themselves, and the NumPy
    product to 2^-53: 2^-51 |p f|.  Cut to 2^-32 of a turn it is off by 2^-29.3
    rad, sin and cos by two units of 2^-24 at most and the factor by one; 2^-21.5
    is above that for each of cos and sin, times (|a| + |b|) factor; the two products and the sum add 3 units of 2^-24, the `steps` turns
    from row to row 2^-22 each.  Values that pass through are exact."""
    rot = 2 * len(freq)
    x = np.abs(np.asarray(x, dtype=np.float64))
    a, b = split(x, rot, interleaved)
    angle = np.abs(np.asarray(pos, dtype=np.float64))[..., None, None] * freq * 2.0 ** -51
    e = (a + b) * factor * (angle + 2.0 ** -21.5 + 3 * 2.0 ** -24 + (steps - 1) * 2.0 ** -22)
    return join(e, e, np.zeros_like(x), rot, interleaved)


def close_bf16(got, want, off, what=""):
    """got (bf16 values) is `want` + at most `off`, rounded once."""
    tol = U * np.abs(want) + (1 + U) * off + 2.0 ** -134  # (half a step of bf16's smallest)
    far = np.abs(np.asarray(got, dtype=np.float64) - want) - tol
    assert np.all(np.isfinite(got)) and far.max(initial=-1.0) <= 0, f"{what}: off by {far.max()}"


def need_scale(amax, grow):
    """The scale of a block of keys: fp32(amax grow) <= 448 need, need a power
    of two of at least 2^-100 and (where the product leaves fp32) at most 2^120."""
    with np.errstate(over="ignore"):
        top = float(np.float32(amax) * np.float32(grow))
    e = -100
    while e < 120 and 448.0 * 2.0 ** e < top:
        e += 1
    return 2.0 ** e


def grow_of(factor):
    return max(np.float32(1.0), np.float32(np.sqrt(2.0) * float(np.float32(factor))))
