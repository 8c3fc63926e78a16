"""The expert layer around the grouped GEMMs -- oracle, test infrastructure.

* Routing table: the (token, choice) pairs of the hosted experts in expert
  order, stable, every group padded to a multiple of ``align``
  (jp-study.kr doc 258368 ¶1-¶2: eight of 256 experts per token, several
  experts per device).
* Combine: out[t] = sum_j w[t,j] y[row_of[t,j]], and its gradient.
* SwiGLU's gradient (tmdrlife.com wr_id=13334 ¶4: the output is recomputed
  from the cached inputs in the backward pass):
  dg = dy u (s + g s (1 - s)), du = dy g s, y = g s u, s = 1 / (1 + e^-g).
* Grouped weight gradient: every group's own sum over its tokens
  (jp-study.kr doc 258368 ¶3).

Everything is plain numpy in 64 bits, row by row.  Pins:
tests/test_oracle_moe_layer.py (hand-worked tables, central differences).
"""

import numpy as np


def sort(experts, first, groups, align, cap):
    """(offsets [groups+1], token [cap], row_of like experts), int64."""
    experts = np.asarray(experts, dtype=np.int64)
    tokens, topk = experts.shape
    token = np.full(cap, -1, dtype=np.int64)
    row_of = np.full((tokens, topk), -1, dtype=np.int64)
    offsets = np.zeros(groups + 1, dtype=np.int64)
    row = 0
    for g in range(groups):
        offsets[g] = min(row, cap)
        for t, j in zip(*np.nonzero(experts == first + g)):  # row-major: by t, then j
            if row < cap:
                token[row] = t
                row_of[t, j] = row
            row += 1
        row = -(-row // align) * align
    offsets[groups] = min(row, cap)
    return offsets, token, row_of


def _rows(y, row_of):
    """(y[row_of] as float64 with zeros for pairs without a row, which pairs have one)."""
    has = (row_of >= 0) & (row_of < y.shape[0])
    out = np.zeros(row_of.shape + (y.shape[1],), dtype=np.float64)
    out[has] = np.asarray(y, dtype=np.float64)[row_of[has]]
    return out, has


def combine(y, row_of, weights=None):
    """(out, sum of |terms|), float64 [tokens, N]."""
    rows, has = _rows(y, row_of)
    w = np.ones(row_of.shape) if weights is None else np.where(has, np.asarray(weights, dtype=np.float64), 0.0)
    terms = rows * w[:, :, None]
    return terms.sum(1), np.abs(terms).sum(1)


def combine_backward(dout, y, row_of, weights=None):
    """(dy [cap, N] before rounding, dweights, sum of |terms| of dweights); rows without a pair are zero."""
    dout = np.asarray(dout, dtype=np.float64)
    rows, has = _rows(y, row_of)
    terms = rows * dout[:, None, :]
    w = np.ones(row_of.shape) if weights is None else np.asarray(weights, dtype=np.float64)
    dy = np.zeros(y.shape, dtype=np.float64)
    for t, j in zip(*np.nonzero(has)):
        dy[row_of[t, j]] = w[t, j] * dout[t]
    return dy, np.where(has, terms.sum(2), 0.0), np.where(has[:, :, None], np.abs(terms), 0.0).sum(2)


def swiglu_backward(x, dy):
    """(dx, y, error scale of dx): the scale is the sum of the magnitudes that
    are added to form each derivative, times |dy| and |u|."""
    x = np.asarray(x, dtype=np.float64)
    dy = np.asarray(dy, dtype=np.float64)
    n = x.shape[1] // 2
    g, u = x[:, :n], x[:, n:]
    t = np.exp(-np.abs(g))
    s = np.where(g >= 0, 1.0, t) / (1.0 + t)
    c = np.where(g >= 0, t, 1.0) / (1.0 + t)  # 1 - s without cancellation
    dg = dy * u * (s + g * s * c)
    du = dy * g * s
    scale = np.concatenate([np.abs(dy * u) * (s + np.abs(g) * s * c), np.abs(du)], axis=1)
    return np.concatenate([dg, du], axis=1), g * s * u, scale


# The float32 form: t = e^-|g| carries 2 ln(2) u of argument reduction and one
# ulp (2u) of the hardware exp2 (u = 2^-24); 1 + t rounds (u) with at most half
# of t's error, the reciprocal adds an ulp (2u): r is off by less than
# (1 + 1.7 + 2) u, t r by (3.4 + 4.7 + 1) u; silu adds one rounding, the
# product with 1 - s its error again and the sum another, dy u and the last
# product two: below (9.1 + 1 + 9.1 + 1 + 2) u of the magnitudes added.
SWIGLU_BWD_REL = 23.0 * 2.0 ** -24


def grouped_wgrad(dy_t, dy_scales, x_t, x_scales, offsets, decode):
    """(dW, sum of |terms|) per group, float64 [G, Nout, Kin]; decode maps codes to values."""
    def values(c, s):
        return decode(c).astype(np.float64) * np.repeat(np.asarray(s, dtype=np.float64), 128, axis=1)
    dy, x = values(dy_t, dy_scales), values(x_t, x_scales)
    lo, hi = np.asarray(offsets)[:-1], np.asarray(offsets)[1:]
    dw = np.stack([dy[:, a:b] @ x[:, a:b].T for a, b in zip(lo, hi)])
    return dw, np.stack([np.abs(dy[:, a:b]) @ np.abs(x[:, a:b]).T for a, b in zip(lo, hi)])
