"""GPU tests of w4a16_qk_norm_rope (include/w4a16_step.h) against the 64-bit definition (step_reference.rope)."""
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


class Problem:
    """Seeded rows; q and k dense, or parts of one projected row (packed)."""

    def __init__(self, seed, T, HQ, H, D, rot, axes=1, sections=None, packed=False, hi=100000):
        rng = np.random.default_rng(seed)
        x = torch.from_numpy(rng.normal(size=(T, HQ + 2 * H, D)) * rng.uniform(0.1, 5, size=(1, HQ + 2 * H, 1)))
        x = x.to(torch.bfloat16).cuda()
        self.q, self.k = x[:, :HQ], x[:, HQ:HQ + H]
        if not packed:
            self.q, self.k = self.q.contiguous(), self.k.contiguous()
        w = torch.from_numpy(1 + 0.4 * rng.normal(size=(2, D))).to(torch.bfloat16).cuda()
        self.weights = [w[0].contiguous(), w[1].contiguous()]
        self.inv_freq = torch.from_numpy(10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))).float().cuda() if rot else None
        self.positions = torch.from_numpy(rng.integers(0, hi, size=(axes, T))).to(torch.int32).cuda()
        self.sections = sections

    def args(self):
        pos = None if self.inv_freq is None else self.positions if self.sections else self.positions[0]
        return dict(inv_freq=self.inv_freq, positions=pos, sections=self.sections)

    def want(self, x, weight, offset=0.0, eps=1e-6, norm=True, interleaved=False):
        f = np.zeros(0) if self.inv_freq is None else self.inv_freq.cpu().double().numpy()
        return ref.rope(x.cpu().double().numpy(), None if weight is None else weight.cpu().double().numpy(), offset,
                        np.float64(np.float32(eps)), norm, f, self.positions.cpu().numpy(), self.sections, interleaved)


def close(got, want):
    y, bound = want
    got = got.cpu().double().numpy()
    assert got.shape == y.shape
    bad = ~(np.abs(got - y) <= bound + ref.BF16_STEP * (np.abs(y) + bound))
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[0], got[bad][0], y[bad][0], bound[bad][0])


SHAPES = [  # T, HQ, H, D, rot
    (1, 1, 1, 64, 64), (1, 10, 2, 256, 256), (2, 5, 1, 128, 128), (3, 32, 8, 128, 64), (7, 7, 7, 64, 16), (5, 3, 1, 256, 8),
    (63, 9, 3, 128, 120), (65, 16, 4, 64, 32), (33, 8, 2, 256, 64), (1, 64, 1, 64, 56), (1030, 32, 8, 128, 128),
    (4099, 4, 1, 64, 64), (2050, 10, 2, 256, 128), (9001, 1, 1, 128, 128), (1500, 40, 3, 64, 64), (2, 20001, 9999, 64, 64),
]


@pytest.mark.parametrize("T,HQ,H,D,rot", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("packed", [False, True])
def test_norm_and_rotation(T, HQ, H, D, rot, interleaved, packed):
    say("rope", T, HQ, H, D, rot, interleaved, packed)
    p = Problem(3, T, HQ, H, D, rot, packed=packed)
    q, k = w4.qk_norm_rope(p.q, p.k, *p.weights, **p.args(), interleaved=interleaved)
    close(q, p.want(p.q, p.weights[0], interleaved=interleaved))
    close(k, p.want(p.k, p.weights[1], interleaved=interleaved))


@pytest.mark.parametrize("axes,sections,D,rot", [(1, [32], 64, 64), (2, [5, 27], 64, 64), (3, [16, 24, 24], 128, 128),
                                                 (3, [0, 1, 127], 256, 256), (4, [3, 2, 0, 11], 128, 32),
                                                 (4, [1, 1, 1, 1], 64, 8)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T", [1, 70])
def test_positions_of_several_axes(axes, sections, D, rot, interleaved, T):
    say("rope axes", axes, sections, D, rot, interleaved, T)
    p = Problem(5, T, 6, 2, D, rot, axes, sections, hi=3000)
    q, k = w4.qk_norm_rope(p.q, p.k, *p.weights, **p.args(), interleaved=interleaved)
    close(q, p.want(p.q, p.weights[0], interleaved=interleaved))
    close(k, p.want(p.k, p.weights[1], interleaved=interleaved))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_parts_can_be_left_out(D):
    """No norm, no weights, an offset, no rotation, no keys, no queries."""
    say("rope parts", D)
    p = Problem(7, 37, 5, 2, D, D)
    q, k = w4.qk_norm_rope(p.q, p.k, **p.args(), norm=False)
    close(q, p.want(p.q, None, norm=False))
    q, k = w4.qk_norm_rope(p.q, p.k, p.weights[0], None, **p.args(), weight_offset=1.0, eps=0.5)
    close(q, p.want(p.q, p.weights[0], offset=1.0, eps=0.5))
    close(k, p.want(p.k, None, eps=0.5))
    only, none = w4.qk_norm_rope(p.q, None, p.weights[0], **p.args())
    assert none is None
    close(only, p.want(p.q, p.weights[0]))
    none, only = w4.qk_norm_rope(None, p.k, None, p.weights[1], **p.args())
    assert none is None
    close(only, p.want(p.k, p.weights[1]))
    p.inv_freq = None
    q, k = w4.qk_norm_rope(p.q, p.k, *p.weights)
    close(q, p.want(p.q, p.weights[0]))
    close(k, p.want(p.k, p.weights[1]))
    q, k = w4.qk_norm_rope(p.q, p.k, norm=False)          # nothing at all: a copy
    assert torch.equal(q, p.q) and torch.equal(k, p.k)


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_and_negative_positions(interleaved):
    say("rope far positions", interleaved)
    p = Problem(9, 6, 4, 2, 128, 128)
    p.positions[0] = torch.tensor([2 ** 31 - 1, -(2 ** 31), -1, 0, 1 << 20, 1999999999], dtype=torch.int32)
    q, k = w4.qk_norm_rope(p.q, p.k, *p.weights, **p.args(), interleaved=interleaved)
    close(q, p.want(p.q, p.weights[0], interleaved=interleaved))
    close(k, p.want(p.k, p.weights[1], interleaved=interleaved))
    still, _ = w4.qk_norm_rope(p.q, p.k, **p.args(), interleaved=interleaved, norm=False)
    assert torch.equal(still[3], p.q[3])                  # position 0 turns nothing


@pytest.mark.parametrize("T,D,interleaved", [(1, 64, False), (50, 128, True), (3000, 256, False), (3001, 64, True)])
def test_in_place_and_into_wider_rows(T, D, interleaved):
    """The same bits as into new rows; what lies beside the rows keeps its own."""
    say("rope in place", T, D, interleaved)
    p = Problem(11, T, 5, 2, D, D // 2, packed=True)
    q, k = w4.qk_norm_rope(p.q, p.k, *p.weights, **p.args(), interleaved=interleaved)
    wide = torch.full((T, 9, D), 7.0, dtype=torch.bfloat16, device="cuda")
    w4.w4a16_qk_norm_rope(p.q, p.k, *p.weights, p.inv_freq, p.positions[0], wide[:, 1:6], wide[:, 7:], interleaved=interleaved)
    assert torch.equal(wide[:, 1:6], q) and torch.equal(wide[:, 7:], k)
    assert (wide[:, 0] == 7).all() and (wide[:, 6] == 7).all()
    w4.w4a16_qk_norm_rope(p.q, p.k, *p.weights, p.inv_freq, p.positions[0], p.q, p.k, interleaved=interleaved)
    assert torch.equal(p.q, q) and torch.equal(p.k, k)


def test_rows_of_zeros_infinity_and_nan_stay_their_own():
    say("rope special values")
    p = Problem(13, 9, 6, 2, 128, 64)
    clean, _ = w4.qk_norm_rope(p.q, p.k, *p.weights, **p.args())
    p.q[2, 1] = 0
    p.q[4, 3, 100] = float("inf")
    p.q[5, 0, 7] = float("nan")
    p.q[7, 2] = 2.0 ** -80                               # squares below fp32's least number: eps alone is left
    q, _ = w4.qk_norm_rope(p.q, p.k, *p.weights, **p.args())
    assert (q[2, 1] == 0).all()
    assert torch.isnan(q[5, 0]).all()
    assert torch.isnan(q[4, 3, 100])                     # infinity times 1 / infinity
    same = torch.ones(9, 6, dtype=torch.bool, device="cuda")
    for t, h in ((2, 1), (4, 3), (5, 0), (7, 2)):
        same[t, h] = False
    assert torch.equal(q[same], clean[same])
    zero, _ = w4.qk_norm_rope(p.q, p.k, *p.weights, **p.args(), eps=0.0)
    assert torch.isnan(zero[2, 1]).all()                 # 0 / 0, as the formula says


def test_nothing_to_do():
    say("rope of no tokens")
    for T, HQ, H in ((0, 4, 2), (3, 0, 0)):
        q, k = (torch.empty((T, n, 64), dtype=torch.bfloat16, device="cuda") for n in (HQ, H))
        pos = torch.zeros((T,), dtype=torch.int32, device="cuda")
        a, b = w4.qk_norm_rope(q, k, inv_freq=torch.ones(32, device="cuda"), positions=pos)
        assert a.shape == q.shape and b.shape == k.shape


def test_captured_and_on_another_stream():
    """A graph follows positions and rows that change between its replays; another stream gives the same bits."""
    say("rope captured")
    p = Problem(15, 24, 8, 2, 128, 128)
    out = [torch.empty_like(p.q), torch.empty_like(p.k)]
    call = lambda: w4.w4a16_qk_norm_rope(p.q, p.k, *p.weights, p.inv_freq, p.positions[0], *out)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(3):
        p.positions += 977
        p.q.mul_(0.75)
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            q, k = w4.qk_norm_rope(p.q, p.k, *p.weights, **p.args())
        side.synchronize()
        assert torch.equal(out[0], q) and torch.equal(out[1], k)
        other = w4.qk_norm_rope(p.q, p.k, *p.weights, **p.args(), stream=side)
        side.synchronize()
        assert torch.equal(other[0], q) and torch.equal(other[1], k)
    close(out[0], p.want(p.q, p.weights[0]))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("exponent", [-60, -63, -64, -66])
def test_rows_whose_mean_square_is_subnormal(D, exponent):
    """eps 0: the mean square lies below fp32's least normal number, 2^-126, and is still what the row is divided by.

    Elements' squares are multiples of 2^-149 there, each off by 2^-150: beside a mean of 2^(2 exponent) or more that is
    2^(-150 - 2 exponent) of it, for the sum and again for the mean, halved by the root.  (2^-18 at worst.)"""
    say("rope subnormal", D, exponent)
    rng = np.random.default_rng(D - exponent)
    p = Problem(17, 5, 4, 2, D, D // 2)
    for x in (p.q, p.k):
        signs = torch.from_numpy(rng.choice([-1.0, 1.0], size=tuple(x.shape)) * rng.uniform(1, 2, size=tuple(x.shape)))
        x.copy_((signs * 2.0 ** exponent).to(torch.bfloat16))
    q, k = w4.qk_norm_rope(p.q, p.k, *p.weights, **p.args(), eps=0.0)
    for got, x, w in ((q, p.q, p.weights[0]), (k, p.k, p.weights[1])):
        y, bound = p.want(x, w, eps=0.0)
        size = bound / (32 * ref.F32_STEP)
        close(got, (y, bound + size * 2.0 ** (-150 - 2 * exponent)))
