"""Oracle of the cache in 4 bits (test infrastructure only): what rows are held as, in fp64, straight from
the definition of the steps, the zero codes and the nearest multiples."""
from __future__ import annotations

import numpy as np

LARGEST = {"f32": float(np.finfo(np.float32).max), "bf16": 2.0 ** 127 * (2 - 2.0 ** -7), "f16": 65504.0}


def step(span):
    """The smallest number of four significant bits, 2^-126 at least, that 15 times is no less than span."""
    s = max(span / 15, 2.0 ** -126)
    mant, exp = np.frexp(s)  # s = mant 2^exp, 1/2 <= mant < 1
    for eighths in range(8, 17):
        t = float(np.ldexp(eighths / 16, exp))
        if 15 * t >= span and t >= 2.0 ** -126:
            return t
    raise AssertionError


def nearest(y):
    """To the nearest whole number, halves toward zero."""
    return np.sign(y) * np.ceil(np.abs(y) - 0.5)


def hold(x, group, largest):
    """(values, steps) of rows x [...][d]: what a cache of 4 bits holds for them, and each channel's step. A group
    with an infinity or a NaN is NaN."""
    x = np.asarray(x, np.float64)
    g = x.reshape(-1, group)
    with np.errstate(invalid="ignore"):
        fine = np.isfinite(g).all(1)
        g = np.where(fine[:, None], g, 0.0)
        lo, hi = np.minimum(g.min(1), 0), np.maximum(g.max(1), 0)
        s = np.array([step(v) for v in hi - lo]).reshape(-1, 1)
        most = np.floor(largest / s)
        k = np.minimum(nearest(-lo[:, None] / s), most)
        m = np.clip(nearest(g / s), -k, np.minimum(15 - k, most))
    v = np.where(fine[:, None], m * s, np.nan)
    return v.reshape(x.shape), np.broadcast_to(s, g.shape).reshape(x.shape)
