"""GPU tests of the key/value cache at the edges of its contract: steps with more
tokens than their bounds, entries that no row attends, windows and chunks that
candidates cross, launches and appends beyond the common sizes.

The oracle, its bounds and the random problems are those of test_kv_gpu.py.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import decode_w4a16_affine_amd as w4
import kv_reference as ref
from parity import say
from test_kv_gpu import Problem, i32, run_append, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    w4.kv_lib()
    yield
    torch.cuda.synchronize()


def run_into(p, q, out, max_new, max_len=None, window=0, cache=None):
    """The C-ABI call on the caller's q and out (max_len None: what the table's columns hold)."""
    cache = cache or p.device()
    bound = p.width * p.page if max_len is None else max_len
    need = w4.w4a16_kv_attention_workspace_bytes(q.shape[0], len(p.lens), max_new, bound, window, q.shape[1], *cache)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    w4.w4a16_kv_attention(q, *cache, i32(p.table), i32(p.lens), i32(p.start), out, ws, max_new, max_len=max_len,
                          window=window)
    torch.cuda.synchronize()
    return out


def close(got, want, tol):
    """Within the oracle's bound of each element (NaN is not)."""
    got = got.cpu().double().numpy()
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[0], got[bad][0], want[bad][0], tol[bad][0])


@pytest.mark.parametrize("H,G,D,lens,news", [(1, 2, 64, [2, 0, 3], [5, 2, 3]), (1, 4, 128, [10, 3], [40, 6]),
                                             (1, 5, 256, [33, 9], [33, 12])])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 30 + 5])
def test_the_widest_windows_hide_nothing(H, G, D, lens, news, window):
    say("attention window", window, H, G, D, lens, news)
    Problem(53, "int8", H, G, D, 16, lens, news).check(window=window)


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("D,G", [(64, 4), (256, 5)])
def test_lengths_far_past_the_bound_read_nothing_of_a_window(kind, D, G):
    """Positions near 2^31: no entry below max_len lies in their window, and the rows are 0; others are as ever."""
    say("attention, lengths past the bound", kind, D, G)
    p = Problem(57, kind, 2, G, D, 16, [64, 64, 50], [3, 40, 1])
    want, tol = p.want(1 / math.sqrt(D), 100)
    cache = p.device()
    p.lens[:2] = [2 ** 31 - 1, 2 ** 31 - 30]
    out = p.run(window=100, cache=cache)
    assert (out[:43] == 0).all()
    close(out[43:], want[43:], tol[43:])


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("H,G,D,lens,news,max_new", [
    (1, 4, 64, [60], [17], 16),                          # 64 rows of the bound, 68 of the request
    (2, 4, 128, [300, 50, 9, 700], [17, 30, 2, 300], 16),
    (1, 5, 256, [90, 333], [13, 40], 12),
    (1, 64, 64, [40, 41], [2, 1], 1),                    # a bound of one token
    (2, 4, 64, [300, 90, 50], [60, 5, 17], 20),          # a bound of 80 rows: both forms
    (1, 5, 256, [400], [399], 30),
])
def test_requests_of_more_tokens_than_max_new(kind, H, G, D, lens, news, max_new):
    """A request's first max_new rows are written whatever it brings; the others stay as they were."""
    say("attention max_new", kind, H, G, D, lens, news, max_new)
    p = Problem(41, kind, H, G, D, 32, lens, news)
    want, tol = p.want(1 / math.sqrt(D), 0)
    q = p.q.cuda()
    out = run_into(p, q, torch.full(q.shape, 5.0, dtype=torch.bfloat16, device="cuda"), max_new)
    for r, n in enumerate(news):
        a, b = p.start[r], p.start[r] + min(n, max_new)
        close(out[a:b], want[a:b], tol[a:b])
        assert (out[b:p.start[r + 1]] == 5).all(), r


@pytest.mark.parametrize("H,G,D,page,lens,news,window", [
    (2, 4, 64, 16, [600, 1111, 130, 20], [1, 1, 3, 1], 30),
    (1, 8, 128, 32, [900, 700], [8, 5], 100),               # two row groups with begins of their own
    (1, 5, 256, 64, [513, 900], [5, 3], 100),
    (2, 4, 128, 256, [3000], [1], 512),
    (2, 2, 128, 32, [400, 333], [100, 200], 64),            # the rest as tiles
    (1, 4, 64, 64, [700], [150], 33),
    (1, 5, 256, 64, [500, 300], [100, 33], 70),
    (1, 8, 128, 64, [3000, 1100], [100, 9], 700),           # in parts of the cache
    (1, 5, 256, 32, [3001], [40], 650),
])
def test_entries_before_a_window_may_hold_anything(H, G, D, page, lens, news, window):
    """Their pages are still in the table, but hold NaN codes (reused, or never filled)."""
    say("attention, NaN codes before a window", H, G, D, page, lens, news, window)
    p = Problem(43, "fp8", H, G, D, page, lens, news)
    kt, vt, ks, vs = p.device()
    for r, (n, k) in enumerate(zip(lens, news)):
        for j in range(max(0, n - k - window + 1)):
            pg, off = int(p.table[r, j // page]), j % page
            kt.view(torch.uint8)[pg, :, off] = 0x7F
            vt.view(torch.uint8)[pg, :, :, off] = 0xFF if j % 2 else 0x7F
    cache = (kt, vt, ks, vs)
    p.check(window=window, cache=cache)
    p.check(window=window, cache=cache, max_len=max(lens))


@pytest.mark.parametrize("H,G,D,lens,news,T", [
    (1, 4, 64, [40], [5], 3),
    (2, 4, 128, [90, 40], [5, 3], 4),           # the second request has no row at all
    (1, 5, 256, [70, 333], [3, 6], 5),
    (2, 4, 128, [90], [70], 50),                # as tiles
    (1, 5, 256, [30, 300], [2, 40], 31),
])
def test_entries_of_tokens_past_the_rows_of_q_may_hold_anything(H, G, D, lens, news, T):
    """Tokens past T have no slot, so nothing was appended for them: their entries hold NaN codes."""
    say("attention, fewer rows than tokens", H, G, D, lens, news, T)
    p = Problem(47, "fp8", H, G, D, 32, lens, news)
    want, tol = p.want(1 / math.sqrt(D), 0)
    kt, vt, ks, vs = p.device()
    for r, (n, k) in enumerate(zip(lens, news)):
        for i in range(k):
            if p.start[r] + i >= T:
                j = n - k + i
                kt.view(torch.uint8)[int(p.table[r, j // 32]), :, j % 32] = 0x7F
                vt.view(torch.uint8)[int(p.table[r, j // 32]), :, :, j % 32] = 0x7F
    q = p.q[:T].cuda()
    out = run_into(p, q, torch.empty_like(q), max(news), cache=(kt, vt, ks, vs))
    close(out, want[:T], tol[:T])


@pytest.mark.parametrize("page", [16, 64, 256])
def test_plan_gives_no_slot_in_pages_outside_every_cache(page):
    """Page numbers whose slots would pass 32 bits (held, and from the free list), beside the largest one that fits."""
    top = 2 ** 31 // page           # the first that does not fit
    say("plan, pages outside every cache", page)
    table = i32([[top, 7, -1], [top - 1, -1, -1], [2 ** 31 - 1, -1, -1]])
    seq, start, slots, used = w4.kv_plan(i32([page - 2, page - 1, 1]), i32([3, 2, 1]), i32([2 * top, top + 3, 5]),
                                         table, 6, page)
    torch.cuda.synchronize()
    assert table.tolist() == [[top, 2 * top, -1], [top - 1, top + 3, -1], [2 ** 31 - 1, -1, -1]]
    assert slots.tolist() == [-1, -1, -1, 2 ** 31 - 1, -1, -1] and used.tolist() == [2]


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("window", [0, 400])
def test_rows_do_not_depend_on_where_partial_results_lie(kind, window):
    """Partial results are placed by token or by request, whichever needs less: rows are the same in both."""
    say("placement of partial results", kind, window)
    lens = [1026, 700, 2050, 900, 333]
    # tokens, and with 16 or 3 a request, up to 80 or 15 of them by token; tiles beside them
    for news, max_new, sizes in (([5, 1, 16, 40, 2], 40, (64, 65, 80, 81, 300)), ([1, 3, 1, 2, 1], 3, (8, 15, 16, 200)),
                                 ([1, 3, 1, 2, 1], 16, (8, 80, 81))):
        p = Problem(71, kind, 2, 4, 128, 64, lens, news)
        want, tol = p.want(1 / math.sqrt(128), window)
        q = torch.cat([p.q, torch.zeros((300, 8, 128), dtype=torch.bfloat16)]).cuda()
        few = [t for t in range(p.T) if not p.start[3] <= t < p.start[4] or news[3] <= 16]
        first = None
        for T in sizes:
            out = run_into(p, q[:T], torch.full((T, 8, 128), 5.0, dtype=torch.bfloat16, device="cuda"), max_new,
                           window=window)
            close(out[:p.T], want, tol)
            assert (out[p.T:] == 5).all()
            rows = out[few].view(torch.int16)        # (the order of the tiles' sums may depend on the sizes)
            first = rows if first is None else first
            assert torch.equal(rows, first), T


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("D,G", [(64, 8), (128, 4), (256, 5)])
@pytest.mark.parametrize("window", [0, 1, 258, 514, 700])
def test_rows_of_candidates_that_cross_chunks_and_windows(kind, D, G, window):
    """Verify rows equal single-token calls bit for bit where the candidates' entries end, or their windows begin, in
    different chunks (up to 4096 entries, chunks have 256: ends at 512, 1024 and 2048; begins at 256 and 512)."""
    say("candidates across chunks", kind, D, G, window)
    lens, news = [1026, 514, 2050, 40], [5, 4, 3, 1]
    p = Problem(59, kind, 2, G, D, 64, lens, news)
    cache = p.device()
    whole = p.run(cache=cache, window=window)
    q, table = p.q.cuda(), i32(p.table)
    for r, (n, k) in enumerate(zip(lens, news)):
        for i in range(k):
            t = int(p.start[r]) + i
            one = w4.kv_attention(q[t:t + 1], *cache, table[r:r + 1], i32([n - k + i + 1]), i32([0, 1]), 1,
                                  window=window)
            assert torch.equal(one[0].view(torch.int16), whole[t].view(torch.int16)), (r, i)


def test_more_requests_than_one_grid_axis():
    """33000 single tokens (requests past 32768 lie on another axis of the launch) give the rows of smaller calls."""
    R, pages, page, D = 33000, 50, 16, 64
    say("attention of", R, "requests")
    rng = np.random.default_rng(61)
    p = Problem(61, "int8", 1, 1, D, page, [pages * page], [1])
    cache = p.device()
    lens = rng.integers(1, 300, R)
    table = rng.integers(0, pages, (R, 19))
    q = torch.from_numpy(rng.standard_normal((R, 1, D))).to(torch.bfloat16).cuda()
    start = np.arange(R + 1)
    whole = w4.kv_attention(q, *cache, i32(table), i32(lens), i32(start), 1)
    for a, b in ((0, 20000), (20000, R)):
        part = w4.kv_attention(q[a:b], *cache, i32(table[a:b]), i32(lens[a:b]), i32(start[:b - a + 1]), 1)
        assert torch.equal(part.view(torch.int16), whole[a:b].view(torch.int16)), a
    at = [0, 5, 32766, 32767, 32768, 32769, R - 2, R - 1]
    want, tol = ref.attention(q[at].cpu().double().numpy(), p.kc, p.ks, p.vc, p.vs, table[at], lens[at],
                              np.arange(len(at) + 1), 0.125, 0)
    close(whole[at], want, tol)


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("D,page,singles", [(64, 16, 700), (128, 256, 90), (256, 64, 200)])
def test_append_of_over_4096_tokens(kind, D, page, singles):
    """Blocks that look at 64 tokens: a long run, runs of 1 to 5 tokens side by side, skipped slots, another long run."""
    H, T = 2, 4500
    say("append", kind, D, page, T)
    rng = np.random.default_rng(67 + page)
    pages = T // page + singles + 8
    state = [*ref.random_codes(rng, pages, H, page, D, kind), *ref.random_codes(rng, pages, H, page, D, kind)]
    ids = iter(rng.permutation(pages))
    slots = []

    def run(n, off):
        while n > 0:
            here = min(n, page - off)
            p = next(ids)
            slots.extend(p * page + off + i for i in range(here))
            n, off = n - here, 0

    run(1500, 5)
    for s in range(singles):
        run(1 + s % 5, int(rng.integers(0, page - 5)))
        if s % 11 == 0:
            slots.append(-1)
    run(T - len(slots), page - 3)
    slots = np.array(slots)
    x_k, x_v = (torch.from_numpy(rng.standard_normal((T, H, D)) * np.exp2(rng.integers(-3, 4, (T, 1, 1)))
                                 ).to(torch.bfloat16) for _ in range(2))
    want = [a.copy() for a in state]
    ref.append(x_k.double().numpy(), slots, want[0], want[1], kind)
    ref.append(x_v.double().numpy(), slots, want[2], want[3], kind)
    got = run_append(x_k, x_v, slots, state, kind)
    for name, a, b in zip(("k codes", "k scales", "v codes", "v scales"), got[:4], want):
        assert same(a, b), name
