"""A serving step's operators (include/w4a16_step.h) in plain 64-bit numpy (angles in 80 bits): the oracle of their GPU
tests.  Scalar definitions written out; nothing here comes from the library."""
from __future__ import annotations

import numpy as np

BF16_STEP = 2.0 ** -8       # a rounding to bf16 is off by at most half a step: this much of the value
F32_STEP = 2.0 ** -24


def rope(x, weight, offset, eps, norm, inv_freq, positions, sections, interleaved):
    """(y, bound) of x [T, heads, D] float64; positions [axes, T] ints; inv_freq float64 (of fp32 numbers).

    bound: what fp32 arithmetic may add up to.  The factor of a norm: a sum of D <= 256 squares as 8 fmas a lane and 5
    additions (13 roundings, halved by the root), mean and eps (2, halved), the root's own 2^-23 (2), two products
    and weight + offset (3): under 14 roundings; sine and cosine are off by 2^-23 of the angle's reduction (one
    rounding of a fraction of a turn, 2^-25 turns, 3.2 roundings), their evaluation (2 ulp, 4) and what fp64 leaves of
    positions to 2^31 (2^-24 of a turn, 6.3): under 14; product and fma 2.  32 roundings of |a| + |b| hold all of it."""
    T, heads, D = x.shape
    y = x.copy()
    if norm:
        factor = np.ones(D) if weight is None else weight + offset
        with np.errstate(divide="ignore", invalid="ignore"):
            y = x / np.sqrt((x * x).mean(2, keepdims=True) + eps) * factor
    size = np.abs(y)
    half = len(inv_freq)
    if half:
        axis = np.zeros(half, dtype=int) if sections is None else np.repeat(np.arange(len(sections)), sections)
        angle = positions[axis, :].T.astype(np.longdouble) * np.asarray(inv_freq, dtype=np.longdouble)[None, :]
        c, s = np.cos(angle).astype(np.float64)[:, None, :], np.sin(angle).astype(np.float64)[:, None, :]
        i = np.arange(half)
        at, bt = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        a, b = y[..., at].copy(), y[..., bt].copy()
        y[..., at], y[..., bt] = a * c - b * s, a * s + b * c
        size[..., at] = size[..., bt] = np.abs(a) + np.abs(b)
    return y, 32 * F32_STEP * size
