"""GPU tests of w4a16_sample (include/w4a16_step.h) against the 64-bit definition (step_reference.sample).

Tokens have to be equal: borders between them lie within 2^-27 of the definition's at worst (below), and the seeded
numbers keep away from those by more.  A share is one rounding to fp32 away (2^-24), and what its denominator is off by:
each of N weights is held to half of 2^-e, e = 62 - log2(N) rounded up, beside a sum of at least 1."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import decode_w4a16_affine_amd as w4
import step_reference as ref
from parity import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    w4.step_lib()
    yield
    torch.cuda.synchronize()


def f32(values):
    return torch.tensor(np.asarray(values, dtype=np.float32), device="cuda")


def i32(values):
    return torch.tensor(np.asarray(values, dtype=np.int32), device="cuda")


class Problem:
    """Logits (float64 values of the given type) and parameters of each row (None: off)."""

    def __init__(self, x, dtype, u, temperature=None, top_k=None, top_p=None, min_p=None, pad=0):
        x = torch.as_tensor(np.asarray(x))
        M, N = x.shape
        wide = torch.full((M, N + pad), 1e30, dtype=dtype, device="cuda")
        self.logits = wide[:, pad:]
        self.logits.copy_(x)
        self.x = self.logits.cpu().double().numpy()
        self.u = None if u is None else np.asarray(u, dtype=np.float32)
        self.floats = [None if v is None else np.asarray(v, dtype=np.float32) for v in (temperature, top_p, min_p)]
        self.top_k = top_k

    def args(self):
        t, p, m = (None if v is None else f32(v) for v in self.floats)
        return (self.logits, None if self.u is None else f32(self.u), t, None if self.top_k is None else i32(self.top_k), p, m)

    def want(self):
        out = []
        for r in range(len(self.x)):
            t, p, m = (None if v is None else float(v[r]) for v in self.floats)
            out.append(ref.sample(self.x[r], None if self.u is None else float(self.u[r]), 1.0 if t is None else t,
                                  0 if self.top_k is None else int(self.top_k[r]), 1.0 if p is None else p,
                                  0.0 if m is None else m))
        return out

    def check(self):
        tokens, share = w4.sample(*self.args())
        tokens, share = tokens.cpu().numpy(), share.cpu().numpy()
        for r, (token, part) in enumerate(self.want()):
            assert tokens[r] == token, (r, tokens[r], token, share[r], part)
            if np.isnan(part):
                assert np.isnan(share[r])
            else:
                N = self.x.shape[1]
                off = ref.F32_STEP + N * 2.0 ** (max(N - 1, 0).bit_length() - 63) + 2.0 ** -50
                assert abs(share[r] - part) <= off * part, (r, share[r], part)
        return tokens


def rows(seed, M, N, spread=2.0):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(M, N)) * spread
    for r in range(M):      # some that stand out
        at = rng.integers(0, N, size=min(N, 30))
        x[r, at] = 5 + 6 * rng.random(len(at))
    return x, rng.random(M), rng


SIZES = [(1, 1), (3, 2), (5, 7), (2, 63), (4, 64), (3, 65), (7, 1000), (2, 1023), (2, 1024), (3, 1025), (4, 4096), (3, 8191),
         (2, 8193), (3, 50001), (2, 100003), (2, 262144), (1, 1 << 20)]
DTYPES = [torch.float32, torch.bfloat16]


@pytest.mark.parametrize("M,N", SIZES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("params", ["free", "top_k", "large_k", "top_p", "min_p", "k_p", "large_k_p", "all"])
def test_sizes_and_limits(M, N, dtype, params):
    say("sample", M, N, dtype, params)
    x, u, rng = rows(N, M, N)
    kw = dict(temperature=rng.uniform(0.4, 1.5, M))
    if params in ("top_k", "k_p", "all"):
        kw["top_k"] = rng.integers(1, 70, M)
    if params in ("large_k", "large_k_p"):
        kw["top_k"] = rng.integers(max(1, N // 3), N + 5, M)
    if params in ("top_p", "k_p", "large_k_p", "all"):
        kw["top_p"] = rng.uniform(0.3, 0.99, M)
    if params in ("min_p", "all"):
        kw["min_p"] = rng.uniform(0.0005, 0.3, M)
    Problem(x, dtype, u, **kw, pad=N % 5).check()


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_that_ask_for_different_things(dtype):
    say("sample mixed", dtype)
    M, N = 96, 33333
    x, u, rng = rows(5, M, N)
    Problem(x, dtype, u, temperature=rng.choice([0.0, 0.3, 1.0, 2.5], M), top_k=rng.choice([0, -3, 1, 2, 40, 2000, N, 10 ** 9], M),
            top_p=rng.choice([1.0, 2.0, np.nan, 0.0, -1.0, 0.1, 0.9, 0.999], M),
            min_p=rng.choice([0.0, -1.0, np.nan, 1e-6, 0.05, 0.5, 1.0, 1.5, np.inf], M)).check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N", [(3, 9001), (3, 200001), (1, 1 << 20)])
@pytest.mark.parametrize("spread,temperature,limits", [
    (0.1, 1.0, dict(top_p=0.95)), (0.5, 1.0, dict(top_p=0.5)), (1.0, 3.0, dict(top_p=0.99)), (3.0, 0.1, dict(top_k=50)),
    (3.0, 0.1, dict(top_k=1000)), (3.0, 0.05, dict(top_k=3000, top_p=0.9)), (6.0, 0.02, dict(top_p=0.99, min_p=1e-9)),
    (0.3, 1.0, dict(min_p=0.2)), (0.1, 1.0, dict(min_p=0.9, top_k=8000)), (0.01, 2.0, dict(top_k=100, top_p=0.7)),
    (0.3, 1.0, dict(top_k=7000, top_p=0.6, min_p=0.4)), (0.0, 1.0, dict(top_k=5000, top_p=0.35))])
def test_flat_and_steep_rows(dtype, M, N, spread, temperature, limits):
    """Thousands of tokens of nearly the same weight, and weights that vanish long before a limit is reached."""
    say("sample flat or steep", dtype, M, N, spread, temperature, limits)
    rng = np.random.default_rng(N + int(100 * spread))
    Problem(rng.normal(size=(M, N)) * spread, dtype, rng.random(M), temperature=[temperature] * M,
            **{k: [v] * M for k, v in limits.items()}).check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N", [9001, 150001])
@pytest.mark.parametrize("value", [-np.inf, "lowest", -1e4, -25.0])
def test_rows_masked_but_for_a_few(dtype, N, value):
    """A grammar's mask: limits that are not reached before the masked tokens, which have no weight or (-25) a small one."""
    say("sample masked", dtype, N, value)
    rng = np.random.default_rng(N)
    M = 6
    x = np.full((M, N), float(torch.finfo(dtype).min) if value == "lowest" else value)
    for r in range(M):
        at = rng.integers(0, N, size=[1, 3, 30, 200, 1500, 4000][r])
        x[r, at] = 3 * rng.normal(size=len(at))
    Problem(x, dtype, rng.random(M), temperature=[1.0, 0.2, 1.0, 0.8, 1.3, 0.6], top_k=[50, 1000, 400, 1000, 5000, 6000],
            top_p=[1.0, 0.9, 1.0, 0.9999999, 1.0, 0.95], min_p=[0.0, 0.0, 1e-30, 0.0, 0.0, 0.01]).check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N", [5, 700, 20000])
def test_equal_logits(dtype, N):
    """Ties everywhere: limits cut between equal tokens by their index."""
    say("sample ties", dtype, N)
    rng = np.random.default_rng(7)
    M = 24
    x = rng.integers(0, 3, size=(M, N)).astype(np.float64)
    x[:8] = 1.25
    x[20:] = np.where(rng.random((4, N)) < 0.5, 0.0, -0.0)
    Problem(x, dtype, rng.random(M), top_k=rng.choice([0, 1, N // 2, max(1, N - 1)], M),
            top_p=rng.choice([1.0, 0.5, 0.25, 0.75], M), temperature=rng.choice([1.0, 0.7], M)).check()


@pytest.mark.parametrize("dtype", DTYPES)
def test_uniforms_at_their_ends(dtype):
    """0 gives the first kept token of weight, 1 and beyond the last, also of a row masked at both ends."""
    say("sample ends", dtype)
    x, _, rng = rows(9, 12, 5000)
    x[:, :17] = -np.inf
    x[:, 4000:] = -np.inf
    u = [0.0, 1.0, 2.0, np.inf, -1.0, np.nan, 1 - 2.0 ** -24, 2.0 ** -149] + [0.5] * 4
    p = Problem(x, dtype, u)
    p.u[5] = 0.0      # (the definition's first token is what NaN gives too)
    want = p.want()
    p.u[5] = np.nan
    tokens, _ = w4.sample(*p.args())
    assert tokens.cpu().tolist() == [t for t, _ in want]
    assert tokens[0] == 17 and tokens[1] == 3999 and tokens[3] == 3999


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N", [1, 40, 9000])
def test_infinities_nan_and_masked_rows(dtype, N):
    say("sample special values", dtype, N)
    x, u, rng = rows(11, 12, N)
    low = float(torch.finfo(dtype).min)
    x[0] = -np.inf
    x[1] = low                                        # a mask of the type's lowest value: equal tokens
    x[2, :] = low
    x[2, N // 2] = 3.0
    x[3, N // 3] = np.inf
    x[4, ::2] = np.inf                                # several: each with the same weight
    x[5, N // 2:] = np.nan
    x[6] = -np.inf
    x[6, N - 1] = -5.0
    x[7] = np.nan
    x[8, ::2] = -np.inf
    x[9] = low / 2
    x[9, 0] = low
    x[10] *= 1e30
    x[11] *= 1e-30
    p = Problem(x, dtype, u)
    tokens = p.check()
    assert tokens[0] == -1
    p = Problem(x, dtype, u, temperature=[1e-38, 1e-45, 3e38, np.inf, 1.0, 0.0, 0.5, 0.0, np.inf, 1e30, 1e30, 1e-30],
                top_k=[3] * 12, top_p=[0.9] * 12, min_p=[0.01] * 12)
    p.check()
    p = Problem(x, dtype, u, temperature=[np.inf] * 12)
    p.check()
    assert (Problem(x, dtype, None).check()[[1, 3]] == [0, N // 3]).all()


@pytest.mark.parametrize("M,N,params", [(8200, 9, True), (8200, 9, False), (300, 260001, False), (65536, 1, True)])
def test_rows_that_take_turns(M, N, params):
    """More rows than go through the launches together; a few of each turn's ends are looked at."""
    say("sample turns", M, N, params)
    rng = np.random.default_rng(M)
    x = torch.from_numpy(rng.normal(size=(min(M, 512), N)).astype(np.float32)).cuda()
    x = x.repeat(-(-M // len(x)), 1)[:M].contiguous()
    u, t = rng.random(M).astype(np.float32), rng.uniform(0.3, 2, M).astype(np.float32)
    k = rng.integers(0, 9, M) if params else None
    tokens, share = w4.sample(x, f32(u), f32(t), None if k is None else i32(k), f32(t / 2) if params else None)
    turn = 8192 // -(-N // 8192)
    for r in sorted({0, 1, turn - 1, turn, turn + 1, M // 2, M - 2, M - 1} & set(range(M))):
        p = Problem(x[r:r + 1].cpu(), torch.float32, u[r:r + 1], t[r:r + 1], None if k is None else k[r:r + 1],
                    t[r:r + 1] / 2 if params else None)
        assert int(tokens[r]) == p.want()[0][0], r
        one, part = w4.sample(*p.args())
        assert int(one[0]) == int(tokens[r]) and float(part[0]) == float(share[r])
    assert ((tokens >= 0) & (tokens < N)).all()


def test_shares_follow_the_distribution():
    """Uniforms spread evenly over [0, 1) give each token as often as its weight says (within one)."""
    say("sample frequencies")
    n, N = 4096, 50
    rng = np.random.default_rng(3)
    x = np.repeat(rng.normal(size=(1, N)) * 2, n, 0)
    p = Problem(x, torch.float32, (np.arange(n) + 0.5) / n)
    tokens, share = w4.sample(*p.args())
    counts = np.bincount(tokens.cpu().numpy(), minlength=N)
    w = np.exp(p.x[0] - p.x[0].max())
    assert (np.abs(counts - n * w / w.sum()) <= 1).all()


def test_nothing_to_do():
    say("sample of no rows")
    tokens, share = w4.sample(torch.empty((0, 50), device="cuda"), torch.empty((0,), device="cuda"))
    assert tokens.shape == (0,) and share.shape == (0,)
    tokens, share = w4.sample(torch.empty((300, 0), device="cuda"), torch.zeros((300,), device="cuda"))
    assert (tokens == -1).all() and (share == 0).all()


def test_without_shares_and_with_a_small_workspace():
    say("sample workspace")
    x, u, rng = rows(13, 4, 30000)
    p = Problem(x, torch.float32, u, top_p=[0.9] * 4)
    need = w4.w4a16_sample_workspace_bytes(4, 30000)
    ws = torch.full((max(need, 16) + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    tokens = torch.full((6,), -7, dtype=torch.int32, device="cuda")
    w4.w4a16_sample(*p.args(), tokens[1:5].contiguous(), None, ws)
    got = torch.empty((4,), dtype=torch.int32, device="cuda")
    w4.w4a16_sample(*p.args(), got, None, ws[:max(need, 16)])
    assert got.cpu().tolist() == [t for t, _ in p.want()]
    assert (ws[max(need, 16):] == 0xFF).all()
    if need:
        with pytest.raises(w4.W4A16Error):
            w4.w4a16_sample(*p.args(), got, None, ws[:need - 1])
        with pytest.raises(w4.W4A16Error):
            w4.w4a16_sample(*p.args(), got, None, None)


def test_captured_and_on_two_streams():
    """A graph follows logits, numbers and parameters that change; calls on two streams at once give the same tokens."""
    say("sample captured")
    x, u, rng = rows(15, 20, 40000)
    p = Problem(x, torch.float32, u, temperature=rng.uniform(0.5, 1, 20), top_k=rng.choice([0, 20, 3000], 20),
                top_p=rng.choice([1.0, 0.9], 20), min_p=rng.choice([0.0, 0.01], 20))
    args = p.args()
    need = w4.w4a16_sample_workspace_bytes(20, 40000)
    ws = [torch.empty((need,), dtype=torch.uint8, device="cuda") if need else None for _ in range(2)]
    tokens, share = torch.empty((20,), dtype=torch.int32, device="cuda"), torch.empty((20,), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        w4.w4a16_sample(*args, tokens, share, ws[0])
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4.w4a16_sample(*args, tokens, share, ws[0])
    for i in range(4):
        args[0].copy_(args[0].roll(777, dims=1) * 1.01)
        args[1].copy_(args[1].roll(1))
        args[3].copy_(args[3].roll(1))
        torch.cuda.synchronize()
        tokens.fill_(-9)
        graph.replay()
        got = torch.empty_like(tokens)
        with torch.cuda.stream(side):                        # while the replay may run
            w4.w4a16_sample(*args, got, None, ws[1])
        torch.cuda.synchronize()
        want, part = w4.sample(*args)
        assert torch.equal(tokens, want) and torch.equal(got, want) and torch.equal(share, part)
    p.x, p.u, p.top_k = args[0].cpu().double().numpy(), args[1].cpu().numpy(), args[3].cpu().numpy()
    assert tokens.cpu().tolist() == [t for t, _ in p.want()]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N", [(5, 262144), (10, 262144), (1, 1 << 20), (5, 24576)])
@pytest.mark.parametrize("temperature", [1.0, 0.01])
def test_far_masks_beside_a_tail_that_counts(dtype, M, N, temperature):
    """One token on top, 8192 others masked by a finite value far below it, the rest 21.5 temperatures below it, and a
    top_p that cuts through these.

    The tail's weight w is held to half of 2^-e, e = 62 - log2(N): N tokens move the border of top_p, and the drawn token
    along the tail, by half of N 2^-e / w each, beside a token for either border's rounding.  The sum of kept weights is
    off by that many tokens."""
    say("sample far masks", dtype, M, N, temperature)
    far = [-690.0, -1000.0, -1e4, None, -7000.0]
    x = np.full((M, N), -21.5 * temperature)
    x[:, :8192] = -np.inf
    x[:, 100] = 0.0
    for r in range(M):
        piece = 1 + r % (N // 8192 - 1)
        x[r, 8192 * piece:8192 * (piece + 1)] = float(torch.finfo(dtype).min) if far[r % 5] is None else far[r % 5] * temperature
    tail = (N - 16384) * np.exp(-21.5)
    u = np.array([0.0, 1.0, 1.0 / (1.0 + 0.2 * tail), 0.5, 1.0 - 2.0 ** -24] * 2)[:M]
    p = Problem(x, dtype, u, temperature=[temperature] * M, top_p=[(1.0 + 0.5 * tail) / (1.0 + tail)] * M)
    level = p.x[:, 8192:].max()      # the tail's logit
    w = np.exp(level / float(p.floats[0][0]))
    off = N * 2.0 ** ((N - 1).bit_length() - 62)
    tokens, share = (t.cpu().numpy() for t in w4.sample(*p.args()))
    for r, (token, part) in enumerate(p.want()):
        if token == 100:
            assert tokens[r] == 100, (r, tokens[r], share[r], part)
        else:
            place = np.flatnonzero(p.x[r] == level)
            assert p.x[r, tokens[r]] == level, (r, tokens[r], token, share[r], part)
            assert abs(np.searchsorted(place, tokens[r]) - np.searchsorted(place, token)) <= off / w + 2, (r, tokens[r], token)
        assert abs(share[r] - part) <= (ref.F32_STEP + off + 3 * w) * part, (r, share[r], part)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N", [1000, 8192, 100003, 1 << 20])
@pytest.mark.parametrize("log2_weight", [-36.9, -37.5])
@pytest.mark.parametrize("limits", [dict(), dict(top_k=400), dict(top_p=1 - 2.0 ** -24), dict(min_p=1e-30), dict(top_k=1 << 20, min_p=1e-30)])
def test_small_weights_among_large_ones_count_as_the_header_says(dtype, N, log2_weight, limits):
    """One token of 8192 on top, the rest near half of the 2^-36 that sums with limits hold weights to: sums are off by
    N 2^-37 then, and by N times half of 2^-49 or 2^-62 N otherwise."""
    say("sample small weights", dtype, N, log2_weight, limits)
    x = np.full((3, N), log2_weight * np.log(2.0))
    x[:, ::8192] = 0.0
    p = Problem(x, dtype, [0.0, 0.3, 0.9], **{k: [v] * 3 for k, v in limits.items()})
    tokens, share = (t.cpu().numpy() for t in w4.sample(*p.args()))
    coarse = limits and limits.get("top_k") != 400
    off = N * (2.0 ** -37 if coarse else max(2.0 ** -50, 2.0 ** ((N - 1).bit_length() - 63)))
    for r, (token, part) in enumerate(p.want()):
        assert tokens[r] == token, (r, tokens[r], token)
        assert abs(share[r] - part) <= (ref.F32_STEP + off * part) * part, (r, share[r], part)      # (part: 1 / the sum)


def test_tokens_and_shares_beside_a_calls_rows_stay_as_they_were():
    """Rows in the middle of wider arrays, with a workspace larger than asked for."""
    say("sample guards")
    x, u, rng = rows(17, 4, 30000)
    limited = dict(top_p=[0.9, 1.0, 0.5, 0.99], top_k=[0, 40, 0, 3000], min_p=[0.0, 0.0, 0.02, 0.0])
    for params in (limited, {}):
        p = Problem(x, torch.float32, u, temperature=[1.0, 0.7, 0.0, 1.3], **params)
        ws = torch.full((w4.w4a16_sample_workspace_bytes(4, 30000) + 64,), 0xFF, dtype=torch.uint8, device="cuda")
        tokens = torch.full((6,), -7, dtype=torch.int32, device="cuda")
        share = torch.full((6,), -7.0, device="cuda")
        w4.w4a16_sample(*p.args(), tokens[1:5], share[1:5], ws)
        want = p.want()
        assert tokens.cpu().tolist() == [-7, *(t for t, _ in want), -7]
        assert share[0] == -7 and share[5] == -7 and (ws[-64:] == 0xFF).all()
        off = ref.F32_STEP + 30000 * 2.0 ** (15 - 63) + 2.0 ** -50
        assert all(abs(float(share[1 + r]) - part) <= off * part for r, (_, part) in enumerate(want))
