"""GPU tests of w4a16_kv_attention_shared (include/w4a16_step.h) against the 64-bit definition and its bounds
(step_reference.shared_attention).  The random requests over a random paged cache are those of test_kv_gpu.py."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import decode_w4a16_affine_amd as w4
import step_reference as ref
from parity import say
from test_kv_gpu import Problem, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    w4.step_lib()
    yield
    torch.cuda.synchronize()


class Shared(Problem):
    """Requests that begin with the first `shared` entries of request 0."""

    def __init__(self, seed, kind, H, G, D, page, lens, news, shared):
        super().__init__(seed, kind, H, G, D, page, lens, news)
        self.shared = shared
        # columns that are not looked at hold numbers outside the cache
        self.given = self.table.copy()
        self.given[1:, :shared // page] = 10 ** 9
        self.full = self.table.copy()

    def device(self):
        cache = super().device()
        if self.kind == "fp8" and self.given is not self.full and self.shared % self.page and self.shared // self.page < self.width:
            for p in self.table[1:, self.shared // self.page]:      # a row's own page has nothing before the end of the shared ones
                if p >= 0:
                    cache[0].view(torch.uint8)[p, :, :self.shared % self.page] = 0x7F
                    cache[1].view(torch.uint8)[p, :, :, :self.shared % self.page] = 0x7F
        return cache

    def bounds(self):
        return dict(max_new=max(self.news), max_shared=self.shared, max_own=max(0, max(self.lens) - self.shared))

    def want_shared(self, scale=None, max_shared=None, max_own=None):
        shared = self.shared if max_shared is None else min(self.shared, max_shared)
        own = self.bounds()["max_own"] if max_own is None else max_own      # (what the call is given)
        return ref.shared_attention(self.q.double().numpy(), self.kc, self.ks, self.vc, self.vs, self.full, self.lens,
                                    self.start, 1 / math.sqrt(self.D) if scale is None else scale, shared, own)

    def run_shared(self, scale=None, cache=None, q=None, **bounds):
        out = w4.kv_attention_shared(self.q.cuda() if q is None else q, *(cache or self.device()), i32(self.given),
                                     i32(self.lens), i32(self.start), i32([self.shared]), scale=scale,
                                     **{**self.bounds(), **bounds})
        torch.cuda.synchronize()
        return out

    def check_shared(self, scale=None, q=None, **bounds):
        want, tol = self.want_shared(scale, bounds.get("max_shared"), bounds.get("max_own"))
        close(self.run_shared(scale, q=q, **bounds), want, tol)


def close(got, want, tol):
    got = got.cpu().double().numpy()
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[0], got[bad][0], want[bad][0], tol[bad][0])


FORMS = [
    # H, G, D, page, lengths (the new tokens included), new tokens, shared
    ("one entry", 1, 1, 64, 16, [1], [1], 1),
    ("nothing shared", 2, 4, 128, 64, [70, 3], [1, 1], 0),
    ("nothing of its own but the token", 2, 4, 128, 64, [101, 101, 101], [1, 1, 1], 100),
    ("a page's end", 2, 4, 128, 64, [130, 200, 129], [1, 1, 1], 128),
    ("inside a page", 1, 5, 256, 64, [140, 321, 129], [1, 1, 2], 101),
    ("inside a tile", 2, 8, 64, 16, [90, 66, 250], [1, 2, 1], 65),
    ("many rows", 2, 4, 128, 32, [500 + 3 * i for i in range(45)], [1] * 45, 490),
    ("many rows of a head", 1, 1, 64, 16, [300 + i % 7 for i in range(150)], [1] * 150, 299),
    ("verify", 2, 5, 256, 64, [800, 700, 930], [5, 3, 6], 690),
    ("verify over 16 rows", 2, 8, 128, 64, [333, 190], [5, 8], 180),
    ("64 rows", 1, 8, 64, 32, [600, 570], [8, 7], 555),
    ("a group of 64", 1, 64, 64, 16, [200, 181], [1, 1], 170),
    ("no groups", 8, 1, 64, 32, [177, 230], [1, 9], 160),
    ("a group of 3", 1, 3, 128, 128, [1000, 900, 901], [1, 4, 21], 870),
    ("large pages", 1, 4, 128, 256, [800, 700], [1, 4], 600),
    ("parts", 1, 2, 64, 16, [3001, 3010], [1, 1], 2990),
    ("parts of large heads", 1, 5, 256, 128, [1700, 1650], [1, 2], 1640),
    ("parts of a tile", 1, 5, 256, 64, [520] * 40, [1] * 40, 500),
    ("parts beside long own entries", 4, 2, 64, 32, [900 + i for i in range(70)], [1] * 70, 330),
    ("parts of many tiles", 8, 4, 64, 128, [4004 + i % 3 for i in range(34)], [1] * 34, 4000),
    ("empty requests", 2, 4, 128, 32, [90, 0, 95, 0, 100], [0, 0, 1, 0, 1], 70),
    ("positions among the shared entries", 1, 4, 64, 16, [200, 50, 3, 120], [1, 4, 5, 2], 150),
    ("rows before the first entry", 1, 2, 64, 16, [40, 1, 3], [1, 3, 5], 30),
]


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("case", FORMS, ids=[f[0] for f in FORMS])
def test_shared_attention(kind, case):
    say("shared attention", kind, case)
    name, H, G, D, page, lens, news, shared = case
    Shared(61, kind, H, G, D, page, lens, news, shared).check_shared()


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("D,G", [(64, 4), (128, 2), (256, 5)])
@pytest.mark.parametrize("bounds", [dict(max_shared=0), dict(max_shared=77), dict(max_own=0), dict(max_own=9),
                                    dict(max_shared=40, max_own=100), dict(max_shared=5000, max_own=9000)])
def test_bounds_of_the_call_are_respected(kind, D, G, bounds):
    """Fewer entries than the requests hold are attended, as the bounds say; larger ones change nothing but the parts."""
    say("shared attention bounds", kind, D, G, bounds)
    p = Shared(63, kind, 2, G, D, 32, [160, 190, 171], [1, 3, 2], 140)
    if bounds.get("max_shared", 140) < 140:      # entries from there on are each row's own
        p.given = p.full
    p.check_shared(**bounds)


def test_rows_past_the_bound_of_new_tokens_stay_as_they_were():
    say("shared attention rows")
    p = Shared(65, "int8", 2, 4, 128, 32, [160, 190], [2, 5], 140)
    cache, q = p.device(), p.q.cuda()
    need = w4.w4a16_kv_attention_shared_workspace_bytes(9, 2, 3, 140, 50, 8, *cache)
    ws = torch.full((need + 64,), 0xAB, dtype=torch.uint8, device="cuda")
    out = torch.full((9, 8, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    wide = torch.zeros((9, 8, 128), dtype=torch.bfloat16, device="cuda")
    wide[:7] = q
    w4.w4a16_kv_attention_shared(wide, *cache, i32(p.given), i32(p.lens), i32(p.start), i32([140]), out, ws[:need], 3, 140, 50)
    want, tol = p.want_shared()
    close(out[:5], want[:5], tol[:5])
    assert (out[5:] == 3).all() and (ws[need:] == 0xAB).all()
    for bad in (ws[:need - 1], None):
        with pytest.raises(w4.W4A16Error):
            w4.w4a16_kv_attention_shared(wide, *cache, i32(p.given), i32(p.lens), i32(p.start), i32([140]), out, bad, 3, 140, 50)


@pytest.mark.parametrize("kind", ["int8", "fp8"])
def test_missing_pages_strides_and_a_negative_scale(kind):
    """Pages outside the cache are not attended, on either side of the shared entries' end."""
    say("shared attention missing pages", kind)
    p = Shared(67, kind, 2, 4, 64, 16, [300, 250, 280, 245], [1, 2, 1, 1], 240)
    p.given[0, 3], p.given[0, 7], p.given[2, 15], p.given[3, 15] = -1, 10 ** 6, -5, 10 ** 6
    p.full[0, 3], p.full[0, 7], p.full[2, 15], p.full[3, 15] = -1, -1, -1, -1
    wide = torch.zeros((p.T, 8 * 64 + 24), dtype=torch.bfloat16, device="cuda")
    wide[:, 16:16 + 512] = p.q.cuda().view(p.T, -1)
    p.check_shared(scale=-0.2, q=wide[:, 16:16 + 512].view(p.T, 8, 64))


@pytest.mark.parametrize("D,G", [(64, 2), (128, 4), (256, 2)])
def test_entries_that_no_row_attends_may_hold_anything(D, G):
    """Positions among the shared entries: E4M3 NaN codes behind all of them do not enter a sum."""
    say("shared attention garbage", D, G)
    p = Shared(69, "fp8", 1, G, D, 64, [90, 70, 41], [1, 1, 2], 30)
    cache = p.device()
    for j in range(90, 128):
        page = int(p.table[0, j // 64])
        cache[0].view(torch.uint8)[page, :, j % 64] = 0x7F
        cache[1].view(torch.uint8)[page, :, :, j % 64] = 0x7F
    p.shared = 128
    p.given = p.full.copy()
    p.given[1:, :2] = -1
    want, tol = p.want_shared(max_own=0)
    close(p.run_shared(cache=cache, max_shared=128, max_own=0), want, tol)
    close(p.run_shared(cache=cache, max_shared=128, max_own=700), want, tol)


def test_a_nan_scale_stays_with_the_rows_that_attend_it():
    say("shared attention NaN")
    p = Shared(71, "int8", 2, 4, 128, 32, [160, 190, 171], [1, 1, 1], 140)
    clean = p.run_shared()
    cache = p.device()
    cache[2][int(p.table[1, 5]), 1] = float("nan")            # keys of request 1's own page, head 1
    got = p.run_shared(cache=cache)
    assert torch.equal(got[[0, 2]], clean[[0, 2]]) and torch.equal(got[1, :4], clean[1, :4])
    assert torch.isnan(got[1, 4:]).all()
    cache[2][int(p.table[0, 1]), 0] = float("nan")            # of a shared page, head 0
    got = p.run_shared(cache=cache)
    assert torch.isnan(got[:, :4]).all() and torch.equal(got[[0, 2], 4:], clean[[0, 2], 4:])


def test_a_batch_of_many_requests():
    """More requests than a wave's lanes, some of them empty, some with one entry; the last ones differ in every way."""
    say("shared attention, many requests")
    rng = np.random.default_rng(3)
    news = rng.choice([0, 1, 1, 1, 2, 4], 300).tolist()
    lens = [n and int(rng.integers(200, 260)) + n for n in news]
    lens[0] = max(lens[0], 230)
    Shared(73, "fp8", 1, 4, 64, 16, lens, news, 190).check_shared()


def test_captured_with_lengths_that_change_and_on_two_streams():
    say("shared attention captured")
    p = Shared(75, "int8", 2, 4, 128, 32, [700, 650, 690, 645], [1, 3, 2, 1], 640)
    p.given = p.full.copy()
    p.given[1:, :640 // 32] = p.full[0, :640 // 32]           # every row knows the shared pages
    cache, q, table, start = p.device(), p.q.cuda(), i32(p.given), i32(p.start)
    lens, shared = i32(p.lens), i32([640])
    bounds = dict(max_new=3, max_shared=640, max_own=700)
    need = w4.w4a16_kv_attention_shared_workspace_bytes(7, 4, 3, 640, 700, 8, *cache)
    ws = [torch.empty((need,), dtype=torch.uint8, device="cuda") for _ in range(2)]
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        w4.w4a16_kv_attention_shared(q, *cache, table, lens, start, shared, out, ws[0], **bounds)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4.w4a16_kv_attention_shared(q, *cache, table, lens, start, shared, out, ws[0], **bounds)
    for i, s in enumerate((640, 333, 0, 608)):                # the same pages either way: the same attention
        shared.fill_(s)
        torch.cuda.synchronize()
        out.fill_(float("nan"))
        graph.replay()
        other = torch.empty_like(q)
        with torch.cuda.stream(side):
            w4.w4a16_kv_attention_shared(q, *cache, table, lens, start, shared, other, ws[1], **bounds)
        torch.cuda.synchronize()
        eager = w4.kv_attention_shared(q, *cache, table, lens, start, shared, **bounds, stream=side)
        side.synchronize()
        assert torch.equal(out, other) and torch.equal(out, eager)
        p.full = p.given
        p.shared = 0
        close(out, *p.want_shared())
        plain = w4.kv_attention(q, *cache, table, lens, start, 3)
        close(plain, *p.want_shared())
