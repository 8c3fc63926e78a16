"""Between a block's linear layers -- oracle, test infrastructure.

* RMS norm of a residual stream: h = rn(x + residual),
  rstd = rn32(1 / sqrt(mean h^2 + eps)), y = bf16(fl(fl(h rstd) w)), every
  rounding where the operator's definition has one, the sum in extended
  precision.  Its gradient, as defined with its roundings and as the formula
  in 64 bits with the bound between the two.
* The router's choice: scores in 64 bits, groups, ties by index, and its
  gradient (jp-study.kr doc 258368 ¶2: eight of 256 routed experts a token).

Plain numpy, token by token for the router.  Pins: tests/test_oracle_block.py
(hand-worked rows, central differences).
"""

import math

import numpy as np

from . import e4m3

U32 = 2.0 ** -24  # half a step of float32, relative


def f32(v):
    return np.asarray(v, dtype=np.float32)


def round_to(v, kind):
    """float32 values rounded to kind ("bf16" or "f32"), as float32."""
    v = f32(v)
    return v if kind == "f32" else e4m3.bf16_bits_to_f32(e4m3.f32_to_bf16_bits_rne(v))


def rms_reciprocal(h, eps):
    """rn32(1 / sqrt(mean h^2 + eps)) of every row, the sum in extended precision."""
    wide = np.asarray(h, dtype=np.longdouble)
    mean = (wide * wide).sum(1) / wide.shape[1] if wide.shape[1] else np.zeros(len(wide), dtype=np.longdouble)
    return f32(1 / np.sqrt(mean + np.longdouble(eps)))


def normalised_bits(h, rstd, w):
    """BF16 patterns of y = bf16(fl(fl(h rstd) w)) from float32 arrays."""
    with np.errstate(all="ignore"):
        return e4m3.f32_to_bf16_bits_rne((f32(h) * f32(rstd)[:, None]) * f32(w))


def rmsnorm(x, residual, w, eps, stream="bf16"):
    """(h float32, rstd float32, y BF16 patterns) from float32 arrays; residual may be None."""
    h = f32(x) if residual is None else round_to(f32(x) + f32(residual), stream)
    rstd = rms_reciprocal(h, eps)
    return h, rstd, normalised_bits(h, rstd, w)


def rmsnorm_backward(dy, h, rstd, w, dres=None):
    """dx in float32, with the roundings of its definition (before the last one to BF16)."""
    dy, h, w, r = f32(dy), f32(h), f32(w), f32(rstd)[:, None]
    g = dy * w
    dot = (np.asarray(g, dtype=np.longdouble) * np.asarray(h, dtype=np.longdouble)).sum(1, keepdims=True)
    c = f32(dot * np.asarray(r, dtype=np.longdouble) / h.shape[1])
    dx = (g - (h * r) * c) * r
    return dx if dres is None else dx + f32(dres)


def rmsnorm_gradient(dy, h, rstd, w, dres=None):
    """The formula in 64 bits: (dx, dweight, bound of dx's float32 steps, sum of |terms| of dweight).

    Bound: g carries one rounding, t = fl(h r) one, c its own and g's (|g h| summed), t c one more, the difference one,
    the product with r one and the sum with dres one; products of two roundings are covered by the factor."""
    dy, h, w, r = (np.asarray(v, dtype=np.float64) for v in (dy, h, w, np.asarray(rstd)[:, None]))
    g, t = dy * w, h * r
    c = (g * h).mean(1, keepdims=True) * r
    mag = np.abs(g * h).mean(1, keepdims=True) * r
    dx = (g - t * c) * r
    bound = r * U32 * (np.abs(g) + np.abs(t) * (3 * np.abs(c) + mag) + 2 * np.abs(g - t * c))
    if dres is not None:
        dx = dx + np.asarray(dres, dtype=np.float64)
        bound = bound + U32 * np.abs(dx)
    return dx, (dy * t).sum(0), 1.01 * bound, np.abs(dy * t).sum(0)


def scores(x, score):
    """Scores of one token's logits (float64; NaN and -inf have none, +inf counts as the largest float32)."""
    x = np.where(np.isnan(x), -np.inf, np.minimum(np.asarray(x, dtype=np.float64), np.finfo(np.float32).max))
    if score == "sigmoid":
        return x, np.array([0.0 if v == -np.inf else 1 / (1 + math.exp(-v)) if v > -700 else math.exp(v) for v in x])
    if not (x > -np.inf).any():
        return x, np.zeros_like(x)
    e = np.array([0.0 if v == -np.inf else math.exp(v - x.max()) for v in x])
    return x, e / math.fsum(e)


def shares(x, s, score):
    """What each of a token's chosen logits x, of scores s, has of the sum of their scores: in extended precision and
    relative to the largest, since 64 bits hold a score near e^-745 in few bits and below it not at all.  0 where every
    score of a sigmoid is 0 in 64 bits; those of a softmax have a sum whatever else is in the row."""
    if not np.any(np.isfinite(x)) or (score == "sigmoid" and not np.any(s)):
        return np.zeros(len(x))
    wide = np.asarray(x, dtype=np.longdouble)
    low = np.minimum(wide, 0) if score == "sigmoid" else wide
    e = np.exp(low - low.max())
    if score == "sigmoid":
        e = e / (1 + np.exp(-np.abs(wide)))
    return np.asarray(e / e.sum(), dtype=np.float64)


def route(logits, topk, bias=None, score="sigmoid", groups=1, top_groups=1, group_score="top2", renormalize=True, scale=1.0):
    """(experts int64 [tokens, topk], weights float64, scores float64 [tokens, E])."""
    tokens, n = logits.shape
    experts, weights = np.full((tokens, topk), -1, dtype=np.int64), np.zeros((tokens, topk))
    every = np.zeros((tokens, n))
    for t in range(tokens):
        x, s = scores(logits[t], score)
        every[t] = s
        with np.errstate(invalid="ignore"):
            key = x if bias is None else np.where(x > -np.inf, s + np.asarray(bias, dtype=np.float64), -np.inf)
        key = np.where(key > -np.inf, key, -np.inf)  # (NaN is none)
        if groups > 1:
            rank = []
            for g in range(groups):
                at = range(g * (n // groups), (g + 1) * (n // groups))
                val = sorted((s[i] if bias is None and group_score == "top2" else key[i] for i in at if key[i] > -np.inf), reverse=True)
                rank.append(-np.inf if not val else val[0] if group_score == "max" else sum(val[:2]))
            opened = sorted(range(groups), key=lambda g: (-rank[g], g))[:top_groups]
            key = np.array([key[i] if i // (n // groups) in opened else -np.inf for i in range(n)])
        order = [i for i in sorted(range(n), key=lambda i: (-key[i], i)) if key[i] > -np.inf][:topk]
        experts[t, :len(order)] = order
        weights[t, :len(order)] = scale * (shares(x[order], s[order], score) if renormalize else s[order])
    return experts, weights, every


def route_backward(dweights, experts, logits, score="sigmoid", renormalize=True, scale=1.0, dscores=None):
    """(dlogits float64, sum of the magnitudes that are added to form each)."""
    tokens, n = logits.shape
    dx, mag = np.zeros((tokens, n)), np.zeros((tokens, n))
    for t in range(tokens):
        x, s = scores(logits[t], score)
        ds = np.zeros(n) if dscores is None else np.array(dscores[t], dtype=np.float64)
        size = np.abs(ds)
        at = [(int(e), float(d)) for e, d in zip(experts[t], dweights[t]) if 0 <= e < n]
        # what renormalised weights w = s / S bring to x_k is w_k (dw_k - sum_j dw_j w_j), a sigmoid's times 1 - s_k: S itself
        # may be far below what can be divided by
        own, own_size = np.zeros(n), np.zeros(n)
        picked = [e for e, _ in at]
        w = shares(x[picked], s[picked], score) if renormalize else []
        mean = math.fsum(d * v for (_, d), v in zip(at, w))
        mean_size = math.fsum(abs(d) * v for (_, d), v in zip(at, w))
        rest = np.array([0.0 if v == -np.inf else scores(np.array([-v]), "sigmoid")[1][0] for v in x]) if score == "sigmoid" else np.ones(n)  # 1 - s
        for e, d in at:
            if not renormalize:
                ds[e] += scale * d
                size[e] += abs(scale * d)
        for (e, d), v in zip(at, w):
            own[e] += scale * v * (d - mean) * rest[e]
            own_size[e] += abs(scale) * v * (abs(d) + mean_size) * rest[e]
        live = x > -np.inf
        ds, size, own, own_size = (np.where(live, v, 0.0) for v in (ds, size, own, own_size))
        if score == "sigmoid":
            dx[t], mag[t] = own + ds * (s * rest), own_size + size * (s * rest)
        else:
            dx[t], mag[t] = own + s * (ds - math.fsum(ds * s)), own_size + s * (size + math.fsum(size * s))
    return dx, mag
