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
