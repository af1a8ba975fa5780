"""A serving step's operators (include/w4a16_step.h) in plain 64-bit numpy (angles in 80 bits): the oracle of their GPU
tests.  Scalar definitions written out; nothing here comes from the library."""
from __future__ import annotations

import numpy as np

import kv_reference

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


def kept(x, temperature, top_k, top_p, min_p):
    """The tokens of one row (float64) that the limits keep, first to last, and their weights; temperature > 0."""
    order = np.lexsort((np.arange(len(x)), -x))                   # falling logits, ties by the lower index
    with np.errstate(invalid="ignore"):
        away = x[order] - x[order[0]]
    away[x[order] == x[order[0]]] = 0.0                           # (infinity less itself)
    w = np.exp(away / min(temperature, float(np.finfo(np.float32).max)))
    n = len(x)
    if top_k > 0:
        n = min(n, top_k)
    if top_p < 1:
        before = np.concatenate([[0.0], np.cumsum(w[:n])])
        n = min(n, int((before[:n] < top_p * before[n]).sum()))
    if min_p > 0:
        n = min(n, int((w >= min_p).sum()))
    n = max(n, 1)
    return order[:n], w[:n]


def sample(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, share) of one row of float64 logits; parameters are the float64 values of fp32 ones."""
    nan = np.flatnonzero(np.isnan(x))
    if len(nan):
        return int(nan[0]), float("nan")
    if len(x) == 0 or x.max() == -np.inf:
        return -1, 0.0
    if not temperature > 0 or u is None:
        return int(np.argmax(x)), 1.0
    tokens, w = kept(x, temperature, top_k, top_p if top_p < 1 else 1.0, min_p if min_p > 0 else 0.0)
    by_index = np.argsort(tokens)
    tokens, w = tokens[by_index], w[by_index]
    running = np.cumsum(w)
    at = int((running <= u * running[-1]).sum()) if u > 0 else int(np.flatnonzero(running > 0)[0])
    at = min(at, int(np.flatnonzero(w > 0)[-1]))
    return int(tokens[at]), w[at] / running[-1]


def entry_table(table, lens, page, shared, max_own):
    """Entry by entry, [R, longest]: page * P + offset of what each request's entry j < shared + max_own lies in, or -1.

    table [R, width]: row 0's pages up to entry `shared`, each row's own from there on."""
    longest = max([0, *lens])
    out = np.full((len(lens), max(1, longest)), -1)
    for r in range(len(lens)):
        for j in range(min(longest, shared + max_own, table.shape[1] * page)):
            p = table[0 if j < shared else r, j // page]
            out[r, j] = p * page + j % page if p >= 0 else -1
    return out


def shared_attention(q, kc, ks, vc, vs, table, lens, start, scale, shared, max_own):
    """(out, bound) of attention behind shared entries, as kv_reference.attention has them over a cache of one entry a
    page.  (Its bound leaves 2^-21 of exponentials for the join's: the hardware's are off by 2^-23.)"""
    pages, H, P, D = kc.shape
    flat = lambda c: c.transpose(0, 2, 1, 3).reshape(pages * P, H, 1, D)  # noqa: E731
    return kv_reference.attention(q, flat(kc), np.repeat(ks, P, 0), flat(vc), np.repeat(vs, P, 0),
                                  entry_table(table, lens, P, shared, max_own), lens, start, scale, 0)
