"""Pins of oracle/block.py where the router's scores are near the end of the 64-bit range, against 60-digit decimals."""

from decimal import Decimal, localcontext

import numpy as np
import pytest

from oracle import block as B

# logits of a token's chosen experts; the last one holds scores that are 0 in 64 bits beside one that is not
FAR = [[-705.0, -705.5], [-709.5, -712.0], [-712.0, -712.5, -711.0], [-720.0, -720.5], [-740.0, -744.5], [-744.9, -800.0, -745.0], [3.0, -740.0], [0.5, 40.0, -2.0]]


def decimal_scores(x, score):
    """Scores of the logits x as decimals."""
    if score == "sigmoid":
        return [1 / (1 + (-Decimal(float(v))).exp()) for v in x]
    e = [Decimal(float(v)).exp() for v in x]
    return [v / sum(e) for v in e]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("far", FAR)
def test_shares_of_far_scores(far, score):
    x = np.array([far + [0.0] * 3])  # the others are scored, and not chosen: their bias is lower
    bias = np.array([2.0] * len(far) + [0.0] * 3)
    experts, weights, _ = B.route(x, len(far), bias, score=score, scale=2.5)
    assert sorted(experts[0]) == list(range(len(far)))
    with localcontext() as c:
        c.prec = 60
        s = decimal_scores(x[0], score)
        total = sum(s[e] for e in experts[0])
        for e, w in zip(experts[0], weights[0]):
            want = float(Decimal(2.5) * s[e] / total)
            # (64-bit results: a hundred half steps of 2^-53; below the normal numbers the share's rounding, half a step of
            # 2^-1074, counts 2.5 times, the product's and this one's rounding once)
            assert abs(w - want) <= 1e-14 * want + 3 * 2.0 ** -1074


def test_scores_that_are_zero_in_64_bits():
    """A sigmoid's then weigh nothing; a softmax's have a sum all the same."""
    x = np.array([[-746.0, -800.0, 0.0]])
    bias = np.array([2.0, 2.0, 0.0])
    assert B.route(x, 2, bias)[1].tolist() == [[0.0, 0.0]]
    w = B.route(x, 2, bias, score="softmax")[1][0]
    assert abs(w[0] + w[1] - 1) < 1e-15 and abs(w[1] / np.exp(-54.0) - 1) < 1e-14
    assert B.route(np.full((1, 3), -np.inf), 2)[1].tolist() == [[0.0, 0.0]]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("far", FAR)
def test_gradient_of_far_scores(far, score):
    """Against the formula in decimals, and the weights' central differences in decimals."""
    x = np.array([far + [0.0, 1.0]])
    n, k = x.shape[1], len(far)
    r = np.random.default_rng(k)
    dw, ds = r.normal(size=(1, k)), r.normal(size=(1, n))
    experts = np.arange(k)[None]

    def loss(at):
        s = [1 / (1 + (-v).exp()) for v in at]
        if score == "softmax":
            e = [v.exp() for v in at]
            s = [v / sum(e) for v in e]
        total = sum(s[:k])
        return sum(Decimal(2.5) * Decimal(float(d)) * v / total for d, v in zip(dw[0], s)) + sum(Decimal(float(d)) * v for d, v in zip(ds[0], s))

    dx, mag = B.route_backward(dw, experts, x, score, True, 2.5, ds)
    with localcontext() as c:
        c.prec = 400  # (a share of e^-743 = 10^-323 beside one of 1 moves the sum in its 323rd digit)
        at, step = [Decimal(float(v)) for v in x[0]], Decimal(10) ** -12
        for i in range(n):
            up, down = list(at), list(at)
            up[i] += step
            down[i] -= step
            want = float((loss(up) - loss(down)) / (2 * step))
            # a central difference of step 1e-12 is off by 1e-24 of the third derivative, a few of the magnitudes summed
            assert abs(dx[0, i] - want) <= 1e-13 * mag[0, i] + 3 * 2.0 ** -1074, i
