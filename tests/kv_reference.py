"""The paged 8-bit key/value cache in plain 64-bit numpy: the oracle of its GPU tests.

Scalar definitions written out (page by page, row by row); nothing here comes
from the library.  A cache is held as token-major arrays of code VALUES
(float64) with one float64 scale a page and head.
"""
from __future__ import annotations

import math

import numpy as np
import torch

QMAX = {"int8": 127.0, "fp8": 448.0}
TORCH = {"int8": torch.int8, "fp8": torch.float8_e4m3fn}
MIN_SCALE = 2.0 ** -100


def scale_of(a: float, kind: str) -> float:
    """Smallest bf16 number >= a / 127 (int8), smallest power of two >= a / 448 (fp8); NaN if a is not finite."""
    if not math.isfinite(a):
        return math.nan
    if a == 0:
        return MIN_SCALE
    m, e = math.frexp(a / QMAX[kind])
    if kind == "int8":
        s = math.ldexp(math.ceil(m * 256), e - 8)
    else:
        s = math.ldexp(1.0, e - 1 if m == 0.5 else e)
    return max(s, MIN_SCALE)


def nearest_code(y, kind: str):
    """Nearest code value of each y, ties to even."""
    y = np.asarray(y, dtype=np.float64)
    if kind == "int8":
        return np.rint(y)
    _, e = np.frexp(y)
    step = np.ldexp(1.0, np.maximum(e, -5) - 4)     # 4 significant bits, none below 2^-9
    return np.rint(y / step) * step


def runs_of(slots, page: int, slots_total: int):
    """(first token, count) of the longest rows of consecutive slots within one page."""
    out, t = [], 0
    while t < len(slots):
        s = int(slots[t])
        if s < 0 or s >= slots_total:
            t += 1
            continue
        n = 1
        while t + n < len(slots) and slots[t + n] == s + n and (s + n) % page:
            n += 1
        out.append((t, n))
        t += n
    return out


def append(x, slots, codes, scales, kind: str):
    """Writes x [T, H, D] into codes [pages, H, P, D] and scales [pages, H] (both float64, in place)."""
    pages, heads, page, _ = codes.shape
    with np.errstate(invalid="ignore"):
        for t, n in runs_of(slots, page, pages * page):
            p, off = divmod(int(slots[t]), page)
            for h in range(heads):
                part = x[t:t + n, h]
                a = np.abs(part)
                s = scale_of(float(a.max()) if np.isfinite(a).all() else math.nan, kind)
                if off:
                    old = scales[p, h]
                    if math.isnan(old):
                        s = old
                    elif math.isnan(s) or s > old:
                        codes[p, h, :off] = 0.0 if math.isnan(s) else nearest_code(codes[p, h, :off] * old / s, kind)
                    else:
                        s = old
                codes[p, h, off:off + n] = 0.0 if math.isnan(s) else nearest_code(part / s, kind)
                scales[p, h] = s


def attention(q, k_codes, k_scales, v_codes, v_scales, table, seq_lens, token_start, scale, window):
    """Output [T, HQ, D] in 64 bits and the error bound of an element (see bound_of), rows outside requests NaN.

    The bound of a bf16 output computed with fp32 sums and 16-bit weights:
      * the final rounding, 2^-8 |out| (twice the half ulp);
      * the weights: each logit is a D-long fp32 dot product with a few more
        fp32 roundings, off by at most d = (D + 16) 2^-24 max_j scale sum|q k|
        and (exp and log in fp32) 2^-21; a relative weight error of that size
        and the rounding of a weight to 11 bits (2^-11) move the numerator and
        the denominator: (2 d + 2^-20 + 2^-11) twice, on sum p |v|;
      * fp32 sums of n terms: n 2^-23 on sum p |v|;
      * weights below the 16-bit type's normal range: n 2^-24 of the largest value.
    """
    q = np.asarray(q, dtype=np.float64)
    T, HQ, D = q.shape
    pages, H, P, _ = k_codes.shape
    G = HQ // H
    out = np.full((T, HQ, D), np.nan)
    tol = np.zeros((T, HQ, D))
    for r in range(len(seq_lens)):
        n = int(token_start[r + 1] - token_start[r])
        for i in range(n):
            t = int(token_start[r]) + i
            pos = int(seq_lens[r]) - n + i
            lo = max(0, pos - window + 1) if window else 0
            js = [j for j in range(lo, pos + 1)
                  if j // P < table.shape[1] and 0 <= table[r, j // P] < pages]
            out[t], tol[t] = 0.0, 0.0
            if not js:
                continue
            js = np.array(js)
            pg, off = table[r, js // P], js % P
            for h in range(H):
                k = k_codes[pg, h, off] * k_scales[pg, h][:, None]
                v = v_codes[pg, h, off] * v_scales[pg, h][:, None]
                for g in range(h * G, (h + 1) * G):
                    with np.errstate(invalid="ignore"):
                        s = scale * (k @ q[t, g])
                        p = np.exp(s - s.max())
                        p /= p.sum()
                        out[t, g] = p @ v
                        d = (D + 16) * 2.0 ** -24 * float((np.abs(k) @ np.abs(q[t, g])).max()) * abs(scale)
                        tol[t, g] = (2.0 ** -8 * np.abs(out[t, g])
                                     + (2 * (2 * d + 2.0 ** -20 + 2.0 ** -11) + len(js) * 2.0 ** -23) * (p @ np.abs(v))
                                     + len(js) * 2.0 ** -24 * np.abs(v).max())
    return out, tol


# ---- device layout <-> the arrays above -------------------------------------------

def to_values(cache, transposed: bool) -> np.ndarray:
    """A device code tensor as token-major float64 code values [pages, H, P, D]."""
    c = cache.detach().cpu()
    c = c.float() if c.dtype == torch.float8_e4m3fn else c
    a = c.numpy().astype(np.float64)
    return np.ascontiguousarray(a.swapaxes(2, 3)) if transposed else a


def to_codes(values: np.ndarray, kind: str, transposed: bool) -> torch.Tensor:
    """Token-major code values as a device code tensor."""
    a = values.swapaxes(2, 3) if transposed else values
    t = torch.from_numpy(np.ascontiguousarray(a)).float()
    return t.to(TORCH[kind]).cuda()


def random_codes(rng, pages, heads, page, dim, kind):
    """Token-major code values and bf16-valued scales of pages filled from normal entries."""
    x = rng.standard_normal((pages, heads, page, dim))
    scales = np.array([[scale_of(float(np.abs(x[p, h]).max()) * math.ldexp(1.0, int(rng.integers(-3, 4))), kind)
                        for h in range(heads)] for p in range(pages)])
    codes = nearest_code(x / np.array([[scale_of(float(np.abs(x[p, h]).max()), kind) for h in range(heads)]
                                       for p in range(pages)])[:, :, None, None], kind)
    return codes, scales


def dev_scales(scales: np.ndarray) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(scales)).to(torch.bfloat16).cuda()


def host_scales(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def plan(ctx, new, free, table, tokens, page):
    """The plan with Python integers: (table, seq_lens, token_start, slot_map, pages_used)."""
    top = 1 << 29
    ctx = [min(max(int(c), 0), top) for c in ctx]
    new = [min(max(int(n), 0), top) for n in new]
    table = np.array(table, dtype=np.int64).copy()
    width = table.shape[1]
    start, taken, slots = [0], 0, []
    for r, (c, n) in enumerate(zip(ctx, new)):
        held, total = -(-c // page), -(-(c + n) // page)
        for b in range(held, width):
            f = taken + b - held
            table[r, b] = free[f] if b < total and f < len(free) else -1
        for pos in range(c, c + n):
            b = pos // page
            if b >= width or table[r, b] < 0:
                slots.append(-1)
            else:
                slots.append(table[r, b] * page + pos % page)
        taken += total - held
        start.append(start[-1] + n)
    slots = (slots + [-1] * tokens)[:tokens]
    return table, [c + n for c, n in zip(ctx, new)], start, slots, taken
