"""Pins of oracle/block.py: rows worked by hand, gradients against central
differences, the rounding bound against a run with every step rounded."""

import math

import numpy as np
import pytest

from oracle import block as B, e4m3


def test_rmsnorm_by_hand():
    # mean square (9 + 16) / 2 = 12.5, eps 0.0025: rstd = 1 / sqrt(12.5025)
    h, r, y = B.rmsnorm([[1.0, 5.0]], [[2.0, -1.0]], [2.0, 0.5], 0.0025)
    assert h.tolist() == [[3.0, 4.0]] and r[0] == np.float32(1 / math.sqrt(12.5025))
    want = [np.float32(np.float32(3) * r[0]) * np.float32(2), np.float32(np.float32(4) * r[0]) * np.float32(0.5)]
    assert np.array_equal(y[0], e4m3.f32_to_bf16_bits_rne(np.array(want, dtype=np.float32)))
    # the stream is rounded before it is normalised: 256 + 1 is 256 in BF16, ties to even
    assert B.rmsnorm([[256.0]], [[1.0]], [1.0], 1e-6)[0].tolist() == [[256.0]]
    assert B.rmsnorm([[256.0]], [[1.0]], [1.0], 1e-6, "f32")[0].tolist() == [[257.0]]
    # zeros: 1 / sqrt(eps); no columns likewise
    h, r, y = B.rmsnorm([[0.0, -0.0]], None, [1.0, 1.0], 0.25)
    assert r.tolist() == [2.0] and y.tolist() == [[0, 0x8000]]
    assert B.rms_reciprocal(np.zeros((2, 0)), 0.25).tolist() == [2.0, 2.0]


@pytest.mark.parametrize("res", [False, True])
def test_rmsnorm_gradient_against_differences(res):
    g = np.random.default_rng(1)
    x, w, dy = 2 * g.normal(size=(4, 9)), g.normal(size=9), g.normal(size=(4, 9))
    dres = g.normal(size=(4, 9)) if res else None
    eps = 0.01

    def rstd(a):
        return 1 / np.sqrt((a * a).mean(1) + eps)

    def loss(a, b):
        return float((a * rstd(a)[:, None] * b * dy).sum() + (0 if dres is None else (a * dres).sum()))

    dx, dw, bound, mag = B.rmsnorm_gradient(dy, x, rstd(x), w, dres)
    step = 1e-6
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = step
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * step) - dx[i]) < 1e-7
    for i in range(9):
        e = np.zeros(9)
        e[i] = step
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * step) - dw[i]) < 1e-7
    # every step rounded stays within the bound
    xs, ws, ds = B.f32(x), B.f32(w), B.f32(dy)
    rr = None if dres is None else B.f32(dres)
    r = B.rms_reciprocal(xs, eps)
    dx, _, bound, _ = B.rmsnorm_gradient(ds, xs, r, ws, rr)
    off = np.abs(B.rmsnorm_backward(ds, xs, r, ws, rr).astype(np.float64) - dx)
    assert (off <= bound).all() and off.max() > 0.01 * bound.max()


def test_route_by_hand():
    x = np.log(np.array([[1.0, 3.0, 1.0, 3.0, 2.0, 6.0]]))
    s = np.array([0.5, 0.75, 0.5, 0.75, 2 / 3, 6 / 7])
    e, w, every = B.route(x, 3, renormalize=False)
    assert e.tolist() == [[5, 1, 3]] and np.allclose(every[0], s) and np.allclose(w[0], s[[5, 1, 3]])
    e, w, _ = B.route(x, 3, score="softmax", scale=2.0)
    assert e.tolist() == [[5, 1, 3]] and np.allclose(w, [[1.0, 0.5, 0.5]])
    # the bias chooses and does not weigh: keys .5 .75 1.5 .75 .67 .86
    e, w, _ = B.route(x, 2, bias=[0, 0, 1.0, 0, 0, 0])
    assert e.tolist() == [[2, 5]] and np.allclose(w, [[0.5 / (0.5 + 6 / 7), 6 / 7 / (0.5 + 6 / 7)]])
    # three groups of two: two best 1.25, 1.25, 1.52; the first of the equal ones
    assert B.route(x, 3, groups=3, top_groups=2)[0].tolist() == [[5, 1, 4]]
    # by the best: 3, 3, 6
    assert B.route(x, 2, groups=3, top_groups=1, group_score="max")[0].tolist() == [[5, 4]]
    # three groups: one expert masked leaves its group the other alone
    x[0, 5] = -np.inf
    assert B.route(x, 3, groups=3, top_groups=2)[0].tolist() == [[1, 3, 0]]
    x[0, :4] = [np.nan, -np.inf, -np.inf, -np.inf]
    e, w, every = B.route(x, 3)
    assert e.tolist() == [[4, -1, -1]] and w.tolist() == [[1.0, 0.0, 0.0]] and every[0, 0] == 0
    x[0, 4] = -np.inf
    for score in ("sigmoid", "softmax"):
        e, w, every = B.route(x, 2, score=score)
        assert e.tolist() == [[-1, -1]] and not w.any() and not every.any()
    x[0, :2] = np.inf
    assert np.allclose(B.route(x, 2, score="softmax")[1], [[0.5, 0.5]])


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_backward_against_differences(score, renormalize):
    g = np.random.default_rng(2)
    x, dw, ds = g.normal(size=(3, 7)), g.normal(size=(3, 4)), g.normal(size=(3, 7))
    experts = np.array([[4, 1, 0, 6], [2, -1, 5, 7], [3, 3, 1, 0]])  # two without an expert, one twice

    def loss(a):
        total = 0.0
        for t in range(3):
            s = B.scores(a[t], score)[1]
            at = [(e, d) for e, d in zip(experts[t], dw[t]) if 0 <= e < 7]
            den = sum(s[e] for e, _ in at) if renormalize else 1.0
            total += sum(1.7 * d * s[e] / den for e, d in at) + float((s * ds[t]).sum())
        return total

    dx, mag = B.route_backward(dw, experts, x, score, renormalize, 1.7, ds)
    assert (np.abs(dx) <= mag * (1 + 1e-12)).all()
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = 1e-6
        assert abs((loss(x + e) - loss(x - e)) / 2e-6 - dx[i]) < 1e-7
    x[1, 2] = -np.inf
    assert B.route_backward(dw, experts, x, score, renormalize, 1.7, ds)[0][1, 2] == 0
