"""Pins of oracle/moe_layer.py: hand-worked routing tables, gradients against
central differences, and the float32 error bound of SwiGLU's gradient against
an emulation with its transcendental steps pushed one ulp."""

import numpy as np
import pytest

from oracle import moe_layer as M


def test_sort_by_hand():
    experts = np.array([[2, 0], [1, 2], [2, 7], [0, 0]])
    offsets, token, row_of = M.sort(experts, 0, 3, 1, 8)
    assert offsets.tolist() == [0, 3, 4, 7]
    assert token.tolist() == [0, 3, 3, 1, 0, 1, 2, -1]
    assert row_of.tolist() == [[4, 0], [3, 5], [6, -1], [1, 2]]
    # groups of four rows, expert 0 elsewhere, room for two of the three rows of expert 2
    offsets, token, row_of = M.sort(experts, 1, 2, 4, 8)
    assert offsets.tolist() == [0, 4, 8] and token.tolist() == [1, -1, -1, -1, 0, 1, 2, -1]
    offsets, token, row_of = M.sort(experts, 1, 2, 2, 4)
    assert offsets.tolist() == [0, 2, 4] and token.tolist() == [1, -1, 0, 1]
    assert row_of.tolist() == [[2, -1], [0, 3], [-1, -1], [-1, -1]]


def test_combine_by_hand():
    y = np.array([[1.0, 2.0], [3.0, np.nan], [5.0, 6.0]])
    row_of = np.array([[0, 2], [-1, -1], [2, 9]])
    out, mag = M.combine(y, row_of, np.array([[2.0, -1.0], [4.0, 4.0], [0.5, np.inf]]))
    assert out.tolist() == [[-3.0, -2.0], [0.0, 0.0], [2.5, 3.0]] and mag[0].tolist() == [7.0, 10.0]
    assert M.combine(y, row_of)[0].tolist() == [[6.0, 8.0], [0.0, 0.0], [5.0, 6.0]]


@pytest.mark.parametrize("weighted", [True, False])
def test_combine_backward_is_the_gradient(weighted):
    r = np.random.default_rng(3)
    y, dout = r.normal(size=(6, 5)), r.normal(size=(3, 5))
    row_of = np.array([[4, 0], [-1, 2], [5, 1]])
    w = r.normal(size=(3, 2)) if weighted else None
    dy, dw, _ = M.combine_backward(dout, y, row_of, w)
    loss = lambda a, b: float((M.combine(a, row_of, b)[0] * dout).sum())  # noqa: E731
    h = 1e-6
    for i in np.ndindex(y.shape):
        e = np.zeros_like(y)
        e[i] = h
        assert abs((loss(y + e, w) - loss(y - e, w)) / (2 * h) - dy[i]) < 1e-8
    if weighted:
        for i in np.ndindex(w.shape):
            e = np.zeros_like(w)
            e[i] = h
            assert abs((loss(y, w + e) - loss(y, w - e)) / (2 * h) - dw[i]) < 1e-8


def test_swiglu_backward_is_the_gradient():
    r = np.random.default_rng(4)
    x, dy = 3 * r.normal(size=(7, 10)), r.normal(size=(7, 5))
    dx, y, _ = M.swiglu_backward(x, dy)
    silu = lambda a: a[:, :5] / (1 + np.exp(-a[:, :5])) * a[:, 5:]  # noqa: E731
    assert np.allclose(y, silu(x), rtol=1e-14)
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = 1e-6
        assert abs(((silu(x + e) - silu(x - e)) * dy).sum() / 2e-6 - dx[i]) < 1e-7


@pytest.mark.parametrize("push", [-1, 0, 1])
def test_swiglu_backward_float32_bound(push):
    """The kernel's steps in float32, with exp2 and the reciprocal one ulp off either way."""
    r = np.random.default_rng(5)
    g = (r.normal(size=200000) * 8).astype(np.float32).view(np.uint32) & 0xFFFF0000
    g = g.view(np.float32)
    u, d = (((r.normal(size=g.size)).astype(np.float32).view(np.uint32) & 0xFFFF0000).view(np.float32) for _ in range(2))
    f = np.float32
    off = lambda v: np.nextafter(v, f(np.inf) if push > 0 else f(-np.inf)) if push else v  # noqa: E731
    x = -np.abs(g)
    n = np.rint((x * f(1.4426950216293335)).astype(f)).astype(f)
    fma = lambda a, b, c: (a.astype(np.float64) * np.float64(b) + c.astype(np.float64)).astype(f)  # noqa: E731
    fr = fma(x, f(1.92596298909109e-8), fma(x, f(1.4426950216293335), -n))
    t = np.ldexp(off(np.exp2(fr.astype(np.float64)).astype(f)), n.astype(int)).astype(f)
    rr = off((1.0 / (f(1) + t).astype(np.float64)).astype(f))
    tr = (t * rr).astype(f)
    s, c = np.where(g >= 0, rr, tr), np.where(g >= 0, tr, rr)
    silu = (g * s).astype(f)
    dg = ((d * u).astype(f) * (silu.astype(np.float64) * c + s).astype(f)).astype(f)
    du = (d * silu).astype(f)
    want, y, scale = M.swiglu_backward(np.stack([g, u], 1), d[:, None])
    got = np.stack([dg, du], 1)
    assert (np.abs(got - want) <= M.SWIGLU_BWD_REL * scale + 2.0 ** -140).all()
    assert (np.abs((silu * u).astype(f) - y[:, 0]) <= M.SWIGLU_BWD_REL * np.abs(y[:, 0]) + 2.0 ** -140).all()


def test_grouped_wgrad_by_hand():
    dy = np.zeros((1, 256))
    x = np.zeros((2, 256))
    dy[0, [0, 128]] = 2, 3
    x[0, [0, 128]] = 5, 7
    x[1, 129] = 1
    dw, mag = M.grouped_wgrad(dy, np.array([[1.0, 0.5]]), x, np.array([[1.0, 2.0], [1.0, 1.0]]), [0, 0, 128, 256], lambda c: c)
    assert dw.tolist() == [[[0.0, 0.0]], [[10.0, 0.0]], [[21.0, 0.0]]] and mag[2, 0, 0] == 21.0
