"""GPU tests of the paged 8-bit key/value cache against the 64-bit definitions
of tests/kv_reference.py.

Plan, append and dequant are exact (integers, and codes whose choice fp32
decides as exact arithmetic does), so they are compared for equality; the
attention is held to the bound that kv_reference.attention derives.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import decode_w4a16_affine_amd as w4
import kv_reference as ref
from parity import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    w4.kv_lib()
    yield
    torch.cuda.synchronize()


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32).cuda()


# ---- plan -----------------------------------------------------------------------

@pytest.mark.parametrize("R,page,new_hi,spare,width_cut,extra", [
    (0, 16, 1, 4, 0, 3),           # no requests: totals and empty slots are still written
    (1, 64, 1, 4, 0, 0),
    (1, 16, 700, 4, 0, 5),
    (5, 16, 3, 4, 0, 0),
    (67, 32, 5, 0, 0, 9),
    (257, 64, 40, 4, 0, 0),
    (1030, 128, 2, 4, 0, 1),
    (33, 16, 60, -20, 0, 0),       # the free list is too short
    (33, 16, 60, 4, 3, 0),         # the table is too narrow
    (33, 16, 60, 4, 0, -37),       # fewer slots than tokens
])
def test_plan_matches_the_definition(R, page, new_hi, spare, width_cut, extra):
    say(f"plan R={R} page={page} new<={new_hi} spare={spare} cut={width_cut} extra={extra}")
    rng = np.random.default_rng(R * 1000 + page)
    ctx = rng.integers(-3, 900, R)          # some negative lengths, taken as 0
    new = rng.integers(-1, new_hi + 1, R)
    ctx[rng.random(R) < 0.2] = 0
    c0, n0 = np.maximum(ctx, 0), np.maximum(new, 0)
    need = int(sum(-(-(c + n) // page) - -(-c // page) for c, n in zip(c0, n0)))
    width = max(1, max([int(-(-(c + n) // page)) for c, n in zip(c0, n0)], default=1) + 2 - width_cut * 4)
    free = rng.permutation(10000)[:max(0, need + spare)]
    table = rng.integers(0, 10000, (R, width))
    tokens = max(0, int(n0.sum()) + extra)
    want = ref.plan(ctx, new, free, table.reshape(R, width), tokens, page)
    t = i32(table.reshape(R, width))
    seq, start, slots, used = w4.kv_plan(i32(ctx), i32(new), i32(free), t, tokens, page)
    torch.cuda.synchronize()
    assert np.array_equal(t.cpu().numpy(), want[0])
    assert seq.tolist() == want[1] and start.tolist() == want[2]
    assert slots.tolist() == list(want[3]) and used.tolist() == [want[4]]


# ---- append and dequant -----------------------------------------------------------

def run_append(x_k, x_v, slots, state, kind, strided=True):
    """The library's append on the reference state's copy; returns its codes and scales as the reference holds them."""
    kc, ks, vc, vs = state
    dk, dv = ref.to_codes(kc, kind, False), ref.to_codes(vc, kind, True)
    sk, sv = ref.dev_scales(ks), ref.dev_scales(vs)
    T, H, D = x_k.shape
    if strided:     # parts of one wider row a token
        wide = torch.full((T, 2 * H * D + 64), 7.0, dtype=torch.bfloat16, device="cuda")
        k, v = wide[:, 8:8 + H * D].view(T, H, D), wide[:, 40 + H * D:40 + 2 * H * D].view(T, H, D)
        k.copy_(x_k), v.copy_(x_v)
    else:
        k, v = x_k.cuda(), x_v.cuda()
    w4.w4a16_kv_append(k, v, i32(slots), dk, dv, sk, sv)
    torch.cuda.synchronize()
    return ref.to_values(dk, False), ref.host_scales(sk), ref.to_values(dv, True), ref.host_scales(sv), (dk, dv, sk, sv)


def same(a, b):
    return np.array_equal(a, b, equal_nan=True)


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("H,D,page,T", [(1, 64, 16, 40), (2, 128, 64, 150), (3, 256, 32, 70), (2, 64, 256, 300),
                                        (1, 128, 128, 1500)])
def test_append_codes_and_scales_are_exact(kind, H, D, page, T):
    say(f"append {kind} H={H} D={D} page={page} T={T}")
    rng = np.random.default_rng(H * 7 + D + page + T)
    pages = T // page + 14
    state = [*ref.random_codes(rng, pages, H, page, D, kind), *ref.random_codes(rng, pages, H, page, D, kind)]
    # requests: a long one from the middle of a page on, several single tokens and short runs in running pages,
    # one over a page's end, some skipped tokens
    ids = rng.permutation(pages)
    slots = []
    long = T - 24
    pos, b = page // 2 + 3, 0
    while len(slots) < long:
        slots.append(ids[b] * page + pos)
        pos += 1
        if pos == page:
            pos, b = 0, b + 1
    b += 1
    for off, n in ((0, 1), (1, 1), (5, 3), (page - 1, 1), (3, 2)):
        slots += [ids[b] * page + off + i for i in range(n)]
        b += 1
    slots += [ids[b] * page + page - 2, ids[b] * page + page - 1, ids[b + 1] * page, ids[b + 1] * page + 1]
    slots += [-1, -7, pages * page, 2 ** 31 - 1]
    slots += [-1] * (T - len(slots))
    slots = np.array(slots[:T])
    x_k = torch.from_numpy(rng.standard_normal((T, H, D)) * np.exp2(rng.integers(-4, 5, (T, 1, 1)))).to(torch.bfloat16)
    x_v = torch.from_numpy(rng.standard_normal((T, H, D))).to(torch.bfloat16)
    want = [a.copy() for a in state]
    ref.append(x_k.double().numpy(), slots, want[0], want[1], kind)
    ref.append(x_v.double().numpy(), slots, want[2], want[3], kind)
    for strided in (True, False):
        got = run_append(x_k, x_v, slots, state, kind, strided)
        for name, a, b2 in zip(("k codes", "k scales", "v codes", "v scales"), got[:4], want):
            assert same(a, b2), (name, strided, np.argwhere(~((a == b2) | (np.isnan(a) & np.isnan(b2))))[:3])


@pytest.mark.parametrize("kind", ["int8", "fp8"])
def test_append_of_zeros_ties_extremes_and_non_finite_values(kind):
    H, D, page = 2, 64, 16
    rng = np.random.default_rng(5)
    state = [*ref.random_codes(rng, 6, H, page, D, kind), *ref.random_codes(rng, 6, H, page, D, kind)]
    x = np.zeros((9, H, D))
    # page 0 begins with zeros (the smallest scale), page 1 with powers of two and their halves (ties in int8),
    # page 2 with the largest and smallest bf16 numbers
    x[2, :, :] = np.exp2(-np.arange(D) / 4 // 1)
    x[3, :, :] = 127 / 2 * np.exp2(-(np.arange(D) % 8))
    x[4] = 3.3895313892515355e38
    x[5] = 2.0 ** -126
    # one head of page 3's run holds an infinity, page 4's a NaN, page 5 goes on over an old NaN scale
    x[6, 1, 9] = math.inf
    x[7, 0, 0] = math.nan
    x[8] = 1.0
    state[1][5, 0] = math.nan
    slots = np.array([0, 1, page, page + 1, 2 * page, 2 * page + 1, 3 * page + 4, 4 * page, 5 * page + 2])
    xt = torch.from_numpy(x).to(torch.bfloat16)
    want = [a.copy() for a in state]
    ref.append(xt.double().numpy(), slots, want[0], want[1], kind)
    ref.append(xt.double().numpy(), slots, want[2], want[3], kind)
    got = run_append(xt, xt, slots, state, kind)
    for name, a, b in zip(("k codes", "k scales", "v codes", "v scales"), got[:4], want):
        assert same(a, b), name
    assert got[1][0, 0] == 2.0 ** -100 and math.isnan(got[1][3, 1]) and math.isnan(got[1][4, 0])
    # the pages' values: NaN where the scale is
    k, v = w4.kv_dequant(*got[4], i32([0, 3, 5, 4, -1, 6]))
    k = k.cpu().double().numpy()
    v = v.cpu().double().numpy()
    for i, p in enumerate([0, 3, 5, 4]):
        assert same(k[i], want[0][p] * want[1][p][:, None, None])
        assert same(v[i], want[2][p] * want[3][p][:, None, None])
    assert np.isnan(k[4:]).all() and np.isnan(v[4:]).all()


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("D,page", [(64, 256), (128, 16), (256, 64)])
def test_dequant_is_exact(kind, D, page):
    rng = np.random.default_rng(D + page)
    kc, ks = ref.random_codes(rng, 5, 3, page, D, kind)
    vc, vs = ref.random_codes(rng, 5, 3, page, D, kind)
    k, v = w4.kv_dequant(ref.to_codes(kc, kind, False), ref.to_codes(vc, kind, True), ref.dev_scales(ks),
                         ref.dev_scales(vs), i32([4, 0, 0, 3]))
    at = [4, 0, 0, 3]
    assert np.array_equal(k.cpu().double().numpy(), (kc * ks[:, :, None, None])[at])
    assert np.array_equal(v.cpu().double().numpy(), (vc * vs[:, :, None, None])[at])


# ---- attention --------------------------------------------------------------------

class Problem:
    """Random requests over a random paged cache (host copy in the reference's form)."""

    def __init__(self, seed, kind, H, G, D, page, lens, news, garbage=True):
        rng = np.random.default_rng(seed)
        self.kind, self.H, self.G, self.D, self.page = kind, H, G, D, page
        self.lens, self.news = list(lens), list(news)
        need = [-(-max(n, 0) // page) for n in lens]
        pages = sum(need) + 3
        self.kc, self.ks = ref.random_codes(rng, pages, H, page, D, kind)
        self.vc, self.vs = ref.random_codes(rng, pages, H, page, D, kind)
        ids = rng.permutation(pages)
        self.width = max(1, max(need))
        self.table = np.full((len(lens), self.width), -1)
        at = 0
        for r, n in enumerate(need):
            self.table[r, :n] = ids[at:at + n]
            at += n
        self.start = np.concatenate([[0], np.cumsum(news)]).astype(int)
        self.T = int(self.start[-1])
        self.q = torch.from_numpy(rng.standard_normal((self.T, H * G, D)) * rng.uniform(0.3, 3.0, (1, H * G, 1))
                                  ).to(torch.bfloat16)
        self.garbage = garbage

    def device(self):
        kt, vt = ref.to_codes(self.kc, self.kind, False), ref.to_codes(self.vc, self.kind, True)
        if self.garbage and self.kind == "fp8":     # unoccupied entries of a last page hold NaN codes
            for r, n in enumerate(self.lens):
                if n > 0 and n % self.page and self.table[r, n // self.page] >= 0:
                    p = int(self.table[r, n // self.page])
                    kt.view(torch.uint8)[p, :, n % self.page:, :] = 0x7F
                    vt.view(torch.uint8)[p, :, :, n % self.page:] = 0xFF
        return kt, vt, ref.dev_scales(self.ks), ref.dev_scales(self.vs)

    def want(self, scale, window):
        return ref.attention(self.q.double().numpy(), self.kc, self.ks, self.vc, self.vs, self.table, self.lens,
                             self.start, scale, window)

    def run(self, scale=None, window=0, max_new=None, max_len=None, strided=False, cache=None):
        q = self.q.cuda()
        if strided:
            wide = torch.zeros((self.T, q.shape[1] * self.D + 24), dtype=torch.bfloat16, device="cuda")
            wide[:, 16:16 + q.shape[1] * self.D] = q.view(self.T, -1)
            q = wide[:, 16:16 + q.shape[1] * self.D].view(self.T, q.shape[1], self.D)
        out = w4.kv_attention(q, *(cache or self.device()), i32(self.table), i32(self.lens), i32(self.start),
                              max(self.news) if max_new is None else max_new, max_len=max_len, scale=scale,
                              window=window)
        torch.cuda.synchronize()
        return out

    def check(self, window=0, scale=None, **kw):
        want, tol = self.want(1 / math.sqrt(self.D) if scale is None else scale, window)
        got = self.run(window=window, scale=scale, **kw).cpu().double().numpy()
        off = np.abs(got - want)
        bad = ~(off <= tol)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[0], got[bad][0], want[bad][0], tol[bad][0])
        return float(np.max(off / np.maximum(tol, 1e-300))) if off.size else 0.0


FORMS = [
    # H, G, D, page, lengths (the new tokens included), new tokens
    ("one short token", 1, 1, 64, 16, [1], [1]),
    ("two entries", 2, 4, 128, 64, [2], [1]),
    ("around a tile's end", 2, 4, 128, 64, [63, 64, 65, 127, 129], [1] * 5),
    ("around a chunk's end", 1, 5, 256, 64, [511, 512, 513, 1024, 1025], [1] * 5),
    ("pages that end inside a tile", 2, 8, 64, 16, [7, 16, 17, 90, 250], [1, 1, 2, 3, 1]),
    ("large pages", 1, 4, 128, 256, [255, 300, 700], [1, 4, 1]),
    ("empty requests", 2, 4, 128, 32, [0, 5, 0, 40], [0, 1, 0, 1]),
    ("rows before the first entry", 1, 2, 64, 16, [2, 0, 3], [5, 2, 3]),
    ("verify", 2, 5, 256, 64, [100, 700, 1300], [5, 3, 6]),
    ("verify over 16 rows", 2, 8, 128, 64, [333, 90], [5, 8]),
    ("64 rows", 1, 8, 64, 32, [600, 70], [8, 7]),
    ("a group of 64", 1, 64, 64, 16, [200, 31], [1, 2]),
    ("no groups", 8, 1, 64, 32, [77, 130], [1, 9]),
    ("a prompt", 1, 4, 128, 64, [197], [197]),
    ("prompts behind cached parts", 2, 2, 64, 16, [150, 310], [70, 129]),
    ("prompt and tokens in one step", 1, 5, 256, 32, [300, 40, 99], [1, 40, 33]),
    ("a long prompt", 1, 2, 128, 64, [600], [590]),
]


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("case", FORMS, ids=[f[0].replace(" ", "_") for f in FORMS])
def test_attention(kind, case):
    name, H, G, D, page, lens, news = case
    say("attention", name, kind)
    p = Problem(11, kind, H, G, D, page, lens, news)
    say("  worst error / bound:", round(p.check(), 3), round(p.check(strided=True, scale=0.25), 3))


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("H,G,D,page,lens,news,window", [
    (2, 4, 64, 16, [1, 40, 600, 1111], [1, 1, 1, 1], 30),
    (1, 5, 256, 64, [64, 513, 900], [1, 5, 3], 512),
    (2, 2, 128, 32, [400, 333], [100, 333], 64),
    (1, 4, 128, 64, [300], [300], 1),
])
def test_attention_with_a_window(kind, H, G, D, page, lens, news, window):
    say("attention window", window, kind, lens)
    p = Problem(13, kind, H, G, D, page, lens, news)
    # entries before the window may be gone: their pages are not read
    for r, (n, k) in enumerate(zip(lens, news)):
        gone = max(0, n - k - window + 1) // page
        p.table[r, :gone] = -1
    p.check(window=window)


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("H,G,D,page,lens,news,window,gone", [
    (1, 8, 64, 64, [3000], [70], 0, None),                  # few tokens behind a long cache
    (2, 4, 128, 32, [2100, 1500, 40, 0, 1999], [40, 300, 3, 0, 17], 0, None),      # beside rows of the other form
    (1, 5, 256, 64, [2511], [33], 0, None),
    (1, 2, 64, 16, [1301], [1301], 0, None),                # first rows lie in one part, last ones in several
    (1, 8, 128, 64, [3000, 1100], [100, 9], 700, None),     # a window that begins inside a part
    (1, 8, 128, 16, [2600], [50], 0, (40, 150)),            # no page in a whole part
    (1, 8, 256, 128, [2600], [50], 0, (0, 21)),             # no page at all
])
def test_attention_of_prompts_in_parts(kind, H, G, D, page, lens, news, window, gone):
    say("attention in parts", kind, H, G, D, lens, news, window)
    p = Problem(19, kind, H, G, D, page, lens, news)
    if gone:
        p.table[0, gone[0]:gone[1]] = -1
    one = p.run(window=window)
    p.check(window=window, max_len=max(lens))
    p.check(window=window, max_len=4 * max(lens), strided=True)
    assert torch.equal(p.run(window=window), one)


@pytest.mark.parametrize("kind", ["int8", "fp8"])
def test_attention_skips_missing_pages_and_leaves_empty_rows_zero(kind):
    p = Problem(17, kind, 2, 4, 128, 16, [90, 200, 33, 120], [1, 4, 33, 70])
    p.table[0, 2] = -1
    p.table[1, 5] = 10 ** 6
    p.table[2, :] = -1          # nothing left: zeros
    p.table[3, 0] = -5
    p.check()
    got = p.run()
    assert (got[p.start[2]:p.start[3]] == 0).all()


@pytest.mark.parametrize("new", [1, 40])
def test_attention_of_a_page_with_a_nan_scale(new):
    # rows that attend an entry of the page are NaN, the others are not touched by it
    p = Problem(19, "int8", 1, 4, 64, 16, [64, 70], [new, 1])
    bad = int(p.table[0, 2])        # entries 32..47 of request 0
    p.vs[bad, 0] = math.nan
    got = p.run().float().cpu()
    for i in range(new):
        pos = 64 - new + i
        assert bool(torch.isnan(got[i]).all()) == (pos >= 32), pos
        assert bool(torch.isnan(got[i]).any()) == (pos >= 32), pos
    assert torch.isfinite(got[new:]).all()


@pytest.mark.parametrize("D,G", [(64, 8), (128, 4), (256, 5)])
@pytest.mark.parametrize("kind", ["int8", "fp8"])
def test_rows_do_not_depend_on_the_batch_or_on_the_candidates(kind, D, G):
    """A verify batch's rows equal single-token calls bit for bit, alone or among other requests."""
    lens, news = [700, 65, 1200], [5, 3, 1]
    p = Problem(23, kind, 2, G, D, 64, lens, news)
    cache = p.device()
    whole = p.run(cache=cache)
    q, table = p.q.cuda(), i32(p.table)
    for r, (n, k) in enumerate(zip(lens, news)):
        for i in range(k):
            t = int(p.start[r]) + i
            one = w4.kv_attention(q[t:t + 1], *cache, table[r:r + 1], i32([n - k + i + 1]), i32([0, 1]), 1)
            assert torch.equal(one[0].view(torch.int16), whole[t].view(torch.int16)), (r, i)


def test_attention_bounds_of_the_step_are_respected():
    """Rows past max_new and rows outside every request stay as they were; entries past max_len are not read."""
    p = Problem(29, "int8", 1, 4, 64, 16, [40, 50], [6, 2])
    q = torch.cat([p.q, p.q[:3]]).cuda()        # three rows that no request holds
    out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    cache = p.device()
    need = w4.w4a16_kv_attention_workspace_bytes(q.shape[0], 2, 4, 64, 0, 4, *cache)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    w4.w4a16_kv_attention(q, *cache, i32(p.table), i32(p.lens), i32(p.start), out, ws, 4, max_len=64)
    whole = p.run()
    assert torch.equal(out[:4], whole[:4]) and torch.equal(out[6:8], whole[6:8])
    assert (out[4:6] == 5).all() and (out[8:] == 5).all()
    # entries 33.. are not read: the rows at later positions see the first 33
    short = p.run(max_len=33).cpu().double().numpy()
    js = np.arange(33)
    for r in range(2):
        pg = p.table[r, js // 16]
        k = p.kc[pg, 0, js % 16] * p.ks[pg, 0][:, None]
        v = p.vc[pg, 0, js % 16] * p.vs[pg, 0][:, None]
        for t in range(p.start[r], p.start[r + 1]):
            for g in range(4):
                s = 0.125 * (k @ p.q[t, g].double().numpy())
                w = np.exp(s - s.max())
                # 2^-8 for the output's rounding and 2^-9 for the 16-bit weights, both on the largest value
                assert (np.abs(short[t, g] - w @ v / w.sum()) <= (2.0 ** -8 + 2.0 ** -9) * np.abs(v).max()).all()


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("D,G", [(64, 2), (128, 4), (256, 5)])
def test_one_request_of_fewer_tokens_than_its_bound(kind, D, G):
    """A call sized for a prompt that brings one or a few tokens only."""
    for n, length in ((1, 130), (3, 67), (0, 20)):
        p = Problem(37, kind, 2, G, D, 32, [length], [n])
        if n:
            p.check(max_new=500)
        else:
            assert p.run(max_new=500).numel() == 0


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("D,G", [(64, 2), (128, 2), (256, 2)])
@pytest.mark.parametrize("new", [1, 40])
def test_many_small_weights_beside_a_large_one_count(kind, D, G, new):
    """200000 entries of weight 1.3 * 2^-27 beside one of weight 1 whose value is 0: the answer is theirs alone.

    A weight is rounded to fp16 as a multiple of 2^-24 after a factor of 2^6, so it is off by at most 2^-31, which is
    2^-4 / 1.3 of these; the logits' own error ((D + 16) 2^-24 of 18.5) and the output's rounding add less than 2^-7."""
    say(f"small weights {kind} D={D} G={G} new={new}")
    n, page = 200001, 256
    w = 1.3 * 2.0 ** -27
    pages = -(-n // page)
    k, v, ks, vs = w4.kv_cache(pages, 1, D, page, dtype=ref.TORCH[kind])
    kv = torch.zeros((pages, 1, page, D))
    kv[0, 0, 0, 0] = 64.0
    k.copy_(kv.to(ref.TORCH[kind]))
    kv.fill_(64.0)
    kv[0, 0, 0] = 0.0
    v.copy_(kv.swapaxes(2, 3).to(ref.TORCH[kind]))
    ks.fill_(1.0 / 64), vs.fill_(1.0 / 64)
    q = torch.zeros((new, G, D), dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 1.0
    table = i32(np.random.default_rng(1).permutation(pages).reshape(1, pages)[:, :])
    # (page 0 holds the large entry: it has to come first)
    t = table.cpu().numpy()
    t[0, int(np.argwhere(t[0] == 0)[0, 0])], t[0, 0] = t[0, 0], 0
    out = w4.kv_attention(q, k, v, ks, vs, i32(t), i32([n]), i32([0, new]), new, max_len=n, scale=-math.log(w))
    torch.cuda.synchronize()
    others = n - new + np.arange(new, dtype=np.float64)         # entries beside the first that row i attends
    want = np.broadcast_to((others * w / (1.0 + others * w))[:, None, None], (new, G, D))
    err = np.abs(out.double().cpu().numpy() / want - 1.0).max()
    assert err < 2.0 ** -4 / 1.3 + 2.0 ** -7, err


@pytest.mark.parametrize("kind", ["int8", "fp8"])
def test_offsets_past_32_bits(kind):
    """A cache of over 4 GiB a tensor, the request's pages at its far end."""
    H, D, page, pages = 8, 128, 128, 40000       # 5.2 GB of codes in each tensor
    p = Problem(31, kind, H, 2, D, page, [300, 130], [1, 130], garbage=False)
    kt, vt, ks, vs = p.device()
    cache = [torch.empty((pages, H, page, D), dtype=ref.TORCH[kind], device="cuda"),
             torch.empty((pages, H, D, page), dtype=ref.TORCH[kind], device="cuda"),
             torch.empty((pages, H), dtype=torch.bfloat16, device="cuda"),
             torch.empty((pages, H), dtype=torch.bfloat16, device="cuda")]
    n = kt.shape[0]
    for big, small in zip(cache, (kt, vt, ks, vs)):
        big.view(torch.uint8 if big.dtype != torch.bfloat16 else torch.int16)[pages - n:] = small.view(
            torch.uint8 if big.dtype != torch.bfloat16 else torch.int16)
    near = p.run()
    p.table = np.where(p.table >= 0, p.table + pages - n, -1)
    far = p.run(cache=tuple(cache))
    assert torch.equal(near.view(torch.int16), far.view(torch.int16))
    # append at the far end, and read it back
    x = torch.randn((3, H, D), device="cuda").to(torch.bfloat16)
    slots = (pages - 1) * page + torch.arange(3, dtype=torch.int32, device="cuda")
    w4.w4a16_kv_append(x, x, slots, *cache)
    k, v = w4.kv_dequant(*cache, i32([pages - 1]))
    assert torch.equal(k[0, :, :3], v[0, :, :3])
    step = cache[2][pages - 1].float()[:, None, None] * (0.5 if kind == "int8" else 16.0)
    assert ((k[0, :, :3] - x.transpose(0, 1).float()).abs() <= step).all()


# ---- streams, graphs ----------------------------------------------------------------

class Step:
    """One step of a cache: plan, append and attention on buffers of its own."""

    def __init__(self, seed, kind="int8"):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        R, H, G, D, page, pages = 6, 2, 4, 128, 64, 80
        self.page = page
        self.ctx, self.new = i32([5, 700, 64, 0, 1200, 63]), i32([1, 3, 1, 100, 1, 2])
        self.cache = w4.kv_cache(pages, H, D, page, dtype=ref.TORCH[kind])
        bits = torch.randint(0, 100, self.cache[0].shape, generator=g, device="cuda", dtype=torch.uint8)
        self.cache[0].view(torch.uint8).copy_(bits)
        self.cache[1].view(torch.uint8).copy_(bits.transpose(2, 3))
        self.cache[2].fill_(0.015625), self.cache[3].fill_(0.03125)
        self.held = torch.arange(80, dtype=torch.int32, device="cuda").view(4, 20)
        self.table0 = torch.full((R, 20), -1, dtype=torch.int32, device="cuda")
        self.table0[0, 0] = 0
        self.table0[1, :11] = torch.arange(1, 12)
        self.table0[2, 0] = 12
        self.table0[4, :19] = torch.arange(13, 32)
        self.table0[5, 0] = 32
        self.table = self.table0.clone()
        self.free = torch.arange(79, 40, -1, dtype=torch.int32, device="cuda")
        T = 108
        self.k = torch.randn((T, H, D), generator=g, device="cuda").to(torch.bfloat16)
        self.v = torch.randn((T, H, D), generator=g, device="cuda").to(torch.bfloat16)
        self.q = torch.randn((T, H * G, D), generator=g, device="cuda").to(torch.bfloat16)
        e = lambda n: torch.zeros((n,), dtype=torch.int32, device="cuda")  # noqa: E731
        self.seq, self.start, self.slots, self.used = e(R), e(R + 1), e(T), e(1)
        self.out = torch.zeros_like(self.q)
        need = w4.w4a16_kv_attention_workspace_bytes(T, R, 100, 1280, 0, H * G, *self.cache)
        self.ws = torch.empty(max(1, need), dtype=torch.uint8, device="cuda")
        self.kv0 = [t.clone() for t in self.cache]

    def reset(self):
        for t, t0 in zip(self.cache, self.kv0):
            t.copy_(t0)
        self.table.copy_(self.table0)
        for t in (self.seq, self.start, self.slots, self.used, self.out):
            t.zero_()

    def run(self):
        w4.w4a16_kv_plan(self.ctx, self.new, self.free, self.table, self.seq, self.start, self.slots, self.used,
                         self.page)
        w4.w4a16_kv_append(self.k, self.v, self.slots, *self.cache)
        w4.w4a16_kv_attention(self.q, *self.cache, self.table, self.seq, self.start, self.out, self.ws, 100)

    def snapshot(self):
        torch.cuda.synchronize()
        return [t.detach().clone().view(torch.uint8) for t in
                (*self.cache, self.table, self.seq, self.start, self.slots, self.used, self.out)]


@pytest.mark.parametrize("kind", ["int8", "fp8"])
def test_graph_replays_match_eager(kind):
    s = Step(3, kind)
    s.run()
    want = s.snapshot()
    s.reset()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for rep in range(4):
        s.reset()
        torch.cuda.synchronize()
        graph.replay()
        for i, (a, b) in enumerate(zip(s.snapshot(), want)):
            assert torch.equal(a, b), (rep, i)
    # other lengths in the same graph: the launches are sized by bounds alone
    s.reset()
    s.new.copy_(i32([2, 1, 1, 33, 1, 0]))
    torch.cuda.synchronize()
    graph.replay()
    got = s.snapshot()
    s.reset()
    s.run()
    for i, (a, b) in enumerate(zip(got, s.snapshot())):
        assert torch.equal(a, b), i


def test_two_streams_match_one():
    a, b = Step(5), Step(7, "fp8")
    a.run(), b.run()
    ref_a, ref_b = a.snapshot(), b.snapshot()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for rep in range(3):
        a.reset(), b.reset()
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            a.run()
        with torch.cuda.stream(s2):
            b.run()
        torch.cuda.synchronize()
        for x, y in zip(a.snapshot() + b.snapshot(), ref_a + ref_b):
            assert torch.equal(x, y), rep


@pytest.mark.parametrize("raw", [False, True])
def test_a_call_on_another_stream_keeps_its_memory(raw):
    """Workspaces and outputs of calls on a stream of the caller's are not given to the current one before they ran."""
    p = Problem(23, "int8", 2, 4, 128, 64, [3000, 2500, 1800], [1, 2, 1])
    cache, args = p.device(), (i32(p.table), i32(p.lens), i32(p.start))
    q = p.q.cuda()
    want = w4.kv_attention(q, *cache, *args, 2)
    values = w4.kv_dequant(*cache, i32([1, 0]))
    s = torch.cuda.Stream()
    busy = torch.randn((4096, 4096), device="cuda")
    torch.cuda.synchronize()
    for rep in range(3):
        with torch.cuda.stream(s):
            for _ in range(20):
                busy @ busy              # (the calls wait behind these)
        stream = s.cuda_stream if raw else s
        out = w4.kv_attention(q, *cache, *args, 2, stream=stream)
        got = w4.kv_dequant(*cache, i32([1, 0]), stream=stream)
        others = [torch.full((n,), math.nan, device="cuda") for n in (1 << 16, 1 << 18, 1 << 20, 1 << 22) for _ in range(4)]
        torch.cuda.synchronize()
        assert torch.equal(out, want), rep
        assert torch.equal(got[0], values[0]) and torch.equal(got[1], values[1]), rep
        del others
