"""The step of a block between its linear layers, as it is measured: residual addition with root-mean-square norm and
1x128 quantization, its gradient, the normalised rows once more in token-axis tiles (the weight gradients' operand), the
router's choice of experts and its gradient.

`own` false: the plain form, elementary torch operations in float32 (float64 for the sums of squares and for the scores
that choices are made by), rounded once at the end.  `own` true: the calls of fine_grained_fp8_fp8q_amd that a training
or serving program makes."""
import math

import torch

own = False

DEV = "cuda:0"
TILE = 128
E4M3_MAX = 448.0
EPS = 1e-6
NEG = float("-inf")


def listed():
    return [
        # one decoded token: residual and norm ahead of the projections, in the latency of one launch
        dict(name="norm_decode_t1", op="norm", rows=1, width=7168, x="bfloat16", stream="bfloat16", weight="bfloat16", bf16=False, quantize=True, mode="free"),
        # a training batch: new residual stream, codes and scales for the projections, 1 / rms for the backward pass
        dict(name="norm_train_t16384", op="norm", rows=16384, width=7168, x="bfloat16", stream="bfloat16", weight="bfloat16", bf16=False, quantize=True,
             mode="free"),
        # a short batch of odd width, float32 activations without a residual, the output in BF16
        dict(name="norm_odd_t777", op="norm", rows=777, width=1030, x="float32", stream=None, weight="float32", bf16=True, quantize=False, mode="free"),
        # the training batch's backward pass: the stream's own gradient added, the gain's gradient over all tokens
        dict(name="norm_backward_t8192", op="norm_backward", rows=8192, width=7168, dy="bfloat16", h="bfloat16", weight="bfloat16", dres=True, out="bfloat16",
             quantize=False, mode="free"),
        # a small odd layer with a float32 stream
        dict(name="norm_backward_odd_t1001", op="norm_backward", rows=1001, width=1030, dy="bfloat16", h="float32", weight="float32", dres=False,
             out="float32", quantize=False, mode="free"),
        # the dense layers' operand of the weight gradient: all tokens, normalised again from the kept stream
        dict(name="norm_token_t16384", op="norm_token", rows=16384, width=7168, h="bfloat16", weight="bfloat16", groups=0, tokens=16384, mode="pow2"),
        # the experts' operand: rows of a routing table over 1000 tokens, groups padded to 128
        dict(name="norm_token_experts_t1000", op="norm_token", rows=3000, width=2048, h="bfloat16", weight="float32", groups=16, tokens=1000, mode="free"),
        # one decoded token: eight of 256 experts out of four of eight groups, a bias for balance
        dict(name="route_decode_t1", op="route", tokens=1, experts=256, groups=8, top_groups=4, topk=8, score="sigmoid", bias=True, group_score="top2",
             renormalize=True, scale=2.5, logits="float32", masked=False, scores=False),
        # the same router over a training batch
        dict(name="route_train_t16384", op="route", tokens=16384, experts=256, groups=8, top_groups=4, topk=8, score="sigmoid", bias=True, group_score="top2",
             renormalize=True, scale=2.5, logits="float32", masked=False, scores=False),
        # a softmax router without groups, BF16 logits, the scores kept for a balance loss, some tokens of padding
        dict(name="route_softmax_t4099", op="route", tokens=4099, experts=160, groups=1, top_groups=1, topk=6, score="softmax", bias=False, group_score="max",
             renormalize=False, scale=1.0, logits="bfloat16", masked=True, scores=True),
        # gradients of the training batch's logits
        dict(name="route_backward_t16384", op="route_backward", tokens=16384, experts=256, topk=8, score="sigmoid", renormalize=True, scale=2.5,
             logits="float32", out="float32", dscores=False),
        # a small softmax router with the balance loss's gradient of the scores
        dict(name="route_backward_softmax_t1001", op="route_backward", tokens=1001, experts=60, topk=4, score="softmax", renormalize=False, scale=1.0,
             logits="bfloat16", out="bfloat16", dscores=True),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "norm_token", "route", "route_backward"])
    kind = lambda: rng.choice(["bfloat16", "bfloat16", "float32"])  # noqa: E731
    mode = rng.choice(["free", "pow2"])
    if op == "norm":
        quantize = rng.random() < 0.7
        return dict(op=op, rows=_log(rng, 1, 8192), width=_log(rng, 64, 7168), x=kind(), stream=rng.choice(["bfloat16", "float32", None]), weight=kind(),
                    bf16=not quantize or rng.random() < 0.3, quantize=quantize, mode=mode)
    if op == "norm_backward":
        return dict(op=op, rows=_log(rng, 1, 8192), width=_log(rng, 64, 7168), dy=kind(), h=kind(), weight=kind(), dres=rng.random() < 0.6, out=kind(),
                    quantize=rng.random() < 0.3, mode=mode)
    if op == "norm_token":
        groups = rng.choice([0, 0, 4, 16])
        return dict(op=op, rows=_log(rng, 1, 12288), width=_log(rng, 64, 7168), h=kind(), weight=kind(), groups=groups, tokens=_log(rng, 1, 8192), mode=mode)
    experts, groups, top_groups = rng.choice([(8, 1, 1), (20, 5, 2), (60, 1, 1), (64, 8, 3), (160, 8, 3), (256, 8, 4), (256, 1, 1), (384, 1, 1)])
    topk = rng.choice([1, 2, 4, 6, 8])
    score, renormalize, scale = rng.choice(["softmax", "sigmoid"]), rng.random() < 0.6, rng.choice([1.0, 2.5])
    if op == "route":
        bias = rng.random() < 0.6
        return dict(op=op, tokens=_log(rng, 1, 16384), experts=experts, groups=groups, top_groups=top_groups, topk=topk, score=score, bias=bias,
                    group_score="top2" if bias else "max", renormalize=renormalize, scale=scale, logits=kind(), masked=rng.random() < 0.3,
                    scores=rng.random() < 0.3)
    # (one weight that is renormalised to 1 has no gradient)
    return dict(op=op, tokens=_log(rng, 1, 16384), experts=experts, topk=topk, score=score, renormalize=renormalize and topk > 1, scale=scale,
                logits=kind(), out=kind(), dscores=rng.random() < 0.4)


# ---------------------------------------------------------------- inputs ----

def _dtype(name):
    return getattr(torch, name)


def _expert_rows(case):
    """Token of every row of a routing table (host numbers, the same for every seed): groups of uneven length, one in four empty, padded to 128 with -1."""
    g, left = case["groups"], case["rows"]
    share = [0.0 if i % 4 == 3 else 1.0 / (1 + (3 * i) % g) for i in range(g)]
    real = [int(left * s / sum(share)) for s in share]
    real[0] += left - sum(real)
    gen = torch.Generator().manual_seed(11)
    parts = []
    for r in real:
        parts += [torch.randint(0, case["tokens"], (r,), generator=gen), torch.full((-r % TILE,), -1, dtype=torch.long)]
    return torch.cat(parts).int()


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    s = {"case": case}
    op = case["op"]
    if op.startswith("norm"):
        width = case["width"]
        rows = case["tokens"] if op == "norm_token" and case["groups"] else case["rows"]
        s["weight"] = (1.0 + 0.2 * normal(width)).to(_dtype(case["weight"]))
        # tokens of different size, a few wide channels
        size = torch.exp(0.5 * normal(rows, 1)) * torch.exp(0.4 * normal(1, width))
        if op == "norm":
            s["x"] = (size * normal(rows, width)).to(_dtype(case["x"]))
            s["residual"] = (2.0 * size * normal(rows, width)).to(_dtype(case["stream"])) if case["stream"] else None
            return s
        s["h"] = (size * normal(rows, width)).to(_dtype(case["h"]))
        s["rstd"] = _rstd(s["h"])
        if op == "norm_backward":
            s["dy"] = normal(rows, width).to(_dtype(case["dy"]))
            s["dres"] = normal(rows, width).to(_dtype(case["out"])) if case["dres"] else None
        else:
            s["index"] = _expert_rows(case).to(DEV) if case["groups"] else None
        return s
    tokens, experts, topk = case["tokens"], case["experts"], case["topk"]
    logits = normal(tokens, experts) + 0.5 * normal(1, experts)
    if case.get("masked"):  # experts that a token may not take, and tokens of padding
        logits[torch.rand((tokens, experts), generator=gen, device=DEV) < 0.1] = NEG
        logits[torch.rand((tokens,), generator=gen, device=DEV) < 0.05] = NEG
    s["logits"] = logits.to(_dtype(case["logits"]))
    if op == "route":
        s["bias"] = 0.1 * normal(experts) if case["bias"] else None
    else:
        s["experts"] = torch.topk(logits, topk, dim=1).indices.int()
        s["dweights"] = normal(tokens, topk)
        s["dscores"] = 0.01 * normal(tokens, experts) if case["dscores"] else None
    return s


# ------------------------------------------------------------ plain forms ----

def _rstd(h):
    return (1.0 / torch.sqrt(h.double().square().mean(1) + EPS)).float()


def _quantize(x, mode):
    """E4M3 codes (as float8) and scales of 1x128 tiles of the rows of x (float32 holding BF16 values)."""
    rows, cols = x.shape
    tiles = torch.nn.functional.pad(x, (0, -cols % TILE)).view(rows, -1, TILE)
    amax = tiles.abs().amax(dim=2)
    if mode == "free":
        scale = amax / torch.full_like(amax, E4M3_MAX)  # a division by a tensor is one rounding; by a number it may not be
    else:
        m, e = torch.frexp(amax)
        scale = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e - 9 + (m > 0.875).int()), torch.zeros_like(amax))
    q = tiles / torch.where(scale > 0, scale, torch.ones_like(scale))[:, :, None]
    return q.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(rows, -1)[:, :cols], scale


def _plain_scores(x, score):
    """Scores of logits x (float64 or float32; -inf is no score)."""
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - torch.where(top > NEG, top, torch.zeros_like(top)))
    total = e.sum(1, keepdim=True)
    return e / torch.where(total > 0, total, torch.ones_like(total))


def _first(key, count):
    """The `count` largest of every row, ties to the lower index: (values, indices)."""
    value, order = torch.sort(key, dim=1, descending=True, stable=True)
    return value[:, :count], order[:, :count]


def _plain_route(s, case):
    tokens, n, groups = case["tokens"], case["experts"], case["groups"]
    x = s["logits"].double()
    scores = _plain_scores(x, case["score"])
    # without a bias the choice is by the logits themselves: the scores rise with them
    key = x if s["bias"] is None else torch.where(x > NEG, scores + s["bias"].double(), NEG)
    if groups > 1:
        best, _ = _first(key.view(tokens * groups, -1), 2)
        rank = best[:, 0]
        if case["group_score"] == "top2":
            rank = rank + torch.where(best[:, -1] > NEG, best[:, -1], torch.zeros_like(rank))
        _, taken = _first(rank.view(tokens, groups), case["top_groups"])
        open_ = (taken[:, :, None] == torch.arange(groups, device=x.device)).any(1)
        key = torch.where(open_.repeat_interleave(n // groups, dim=1), key, NEG)
    value, experts = _first(key, case["topk"])
    has = value > NEG
    weights = torch.where(has, scores.gather(1, experts), 0.0)
    if case["renormalize"]:
        total = weights.sum(1, keepdim=True)
        weights = weights / torch.where(total > 0, total, 1.0)
    out = {"experts": torch.where(has, experts, -1).int(), "weights": (case["scale"] * weights).float()}
    if case["scores"]:
        out["scores"] = scores.float()
    return out


def _plain_route_backward(s, case):
    scores = _plain_scores(s["logits"].double(), case["score"])  # a sum over chosen experts is taken from each of them: next to nothing may be left
    at, dw = s["experts"].long(), s["dweights"].double()
    if case["renormalize"]:
        picked = scores.gather(1, at)
        total = picked.sum(1, keepdim=True)
        dw = (dw - (dw * picked).sum(1, keepdim=True) / total) / total
    ds = torch.zeros_like(scores).scatter_add(1, at, case["scale"] * dw)
    if s["dscores"] is not None:
        ds = ds + s["dscores"]
    if case["score"] == "sigmoid":
        dx = ds * scores * (1.0 - scores)
    else:
        dx = scores * (ds - (ds * scores).sum(1, keepdim=True))
    return {"dlogits": dx.to(_dtype(case["out"]))}


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "route":
        return _plain_route(s, case)
    if op == "route_backward":
        return _plain_route_backward(s, case)
    w = s["weight"].float()
    if op == "norm":
        out, h = {}, s["x"]
        if s["residual"] is not None:
            out["h"] = h = (h.float() + s["residual"].float()).to(_dtype(case["stream"]))
        out["rstd"] = _rstd(h)
        y = (h.float() * out["rstd"][:, None] * w).to(torch.bfloat16)
        if case["bf16"]:
            out["y"] = y
        if case["quantize"]:
            out["codes"], out["scales"] = _quantize(y.float(), case["mode"])
        return out
    xhat = s["h"].float() * s["rstd"][:, None]
    if op == "norm_backward":
        g = s["dy"].float() * w
        mean = (g.double() * s["h"].double()).sum(1, keepdim=True) * s["rstd"].double()[:, None] / case["width"]
        dx = (g - xhat * mean.float()) * s["rstd"][:, None]
        if s["dres"] is not None:
            dx = dx + s["dres"].float()
        out = {"dx": dx.to(_dtype(case["out"])), "dweight": (s["dy"].float() * xhat).sum(0)}
        if case["quantize"]:
            out["codes"], out["scales"] = _quantize(dx.to(torch.bfloat16).float(), case["mode"])
        return out
    y = (xhat * w).to(torch.bfloat16).float()
    if s["index"] is not None:
        y = torch.where((s["index"] >= 0)[:, None], y[s["index"].clamp(min=0).long()], torch.zeros((), device=y.device))
    codes, scales = _quantize(y.T.contiguous(), case["mode"])
    return {"codes": codes, "scales": scales}


def run(s):
    if not own:
        return _plain(s)
    import fine_grained_fp8_fp8q_amd as fp8q
    case = s["case"]
    op = case["op"]
    if op == "norm":
        y, codes, scales, rstd, h = fp8q.rmsnorm_quantize(s["x"], s["weight"], residual=s["residual"], eps=EPS, bf16=case["bf16"],
                                                          quantize=case["quantize"], scale_mode=case["mode"])
        out = {"rstd": rstd}
        if h is not None:
            out["h"] = h
        if case["bf16"]:
            out["y"] = y
        if case["quantize"]:
            out["codes"], out["scales"] = codes.view(torch.float8_e4m3fn), scales
        return out
    if op == "norm_backward":
        dx, codes, scales, dweight = fp8q.rmsnorm_backward(s["dy"], s["h"], s["rstd"], s["weight"], dres=s["dres"], out_dtype=_dtype(case["out"]),
                                                           quantize=case["quantize"], scale_mode=case["mode"])
        out = {"dx": dx, "dweight": dweight}
        if case["quantize"]:
            out["codes"], out["scales"] = codes.view(torch.float8_e4m3fn), scales
        return out
    if op == "norm_token":
        codes, scales = fp8q.rmsnorm_quantize_t(s["h"], s["rstd"], s["weight"], index=s["index"], scale_mode=case["mode"])
        return {"codes": codes.view(torch.float8_e4m3fn), "scales": scales}
    if op == "route":
        experts, weights, scores = fp8q.moe_route(s["logits"], case["topk"], bias=s["bias"], score=case["score"], groups=case["groups"],
                                                  top_groups=case["top_groups"], group_score=case["group_score"], renormalize=case["renormalize"],
                                                  scale=case["scale"], want_scores=case["scores"])
        out = {"experts": experts, "weights": weights}
        if case["scores"]:
            out["scores"] = scores
        return out
    return {"dlogits": fp8q.moe_route_backward(s["dweights"], s["experts"], s["logits"], score=case["score"], renormalize=case["renormalize"],
                                               scale=case["scale"], dscores=s["dscores"], out_dtype=_dtype(case["out"]))}


# ------------------------------------------------------- 64-bit definition ----

def _quantize64(x, mode):
    """The tile quantizer of BF16 values held in 64 bits: codes and scales as float64 values."""
    rows, cols = x.shape
    count = -(-cols // TILE)
    tiles = torch.zeros((rows, count * TILE), dtype=torch.float64, device=x.device)
    tiles[:, :cols] = x
    tiles = tiles.view(rows, count, TILE)
    amax = tiles.abs().max(dim=2).values
    if mode == "free":
        scale = (amax / E4M3_MAX).float().double()
    else:
        scale = torch.where(amax > 0, torch.exp2(torch.ceil(torch.log2((amax / E4M3_MAX).clamp(min=1e-300)))), amax)
    q = (tiles / scale.clamp(min=1e-300)[:, :, None]).float().to(torch.float8_e4m3fn).double()
    return q.reshape(rows, -1)[:, :cols], scale


def _r32(x):
    return x.float().double()


def _bf16(x):
    return x.float().to(torch.bfloat16).double()


def _normalised64(h, rstd, w):
    """The BF16 rows that are quantized: float32 products, each rounded, as the operator defines them (another rounding would move a scale by a BF16 step)."""
    return _bf16(_r32(h * _r32(rstd)) * w)


def _scores64(x, score):
    return torch.sigmoid(x) if score == "sigmoid" else torch.nan_to_num(torch.softmax(x, dim=1))


def _exact_route(s, case):
    x = s["logits"].double()
    scores = _scores64(x, case["score"])
    key = (x if s["bias"] is None else scores + s["bias"].double()).clone()
    key[x == NEG] = NEG
    tokens, n, groups = case["tokens"], case["experts"], case["groups"]
    if groups > 1:
        per = key.view(tokens, groups, n // groups)
        rank = per.amax(2)
        if case["group_score"] == "top2":
            rank = torch.nan_to_num(per.topk(2, dim=2).values, neginf=0.0).sum(2).masked_fill(rank == NEG, NEG)
        shut = torch.ones((tokens, groups), dtype=torch.bool, device=x.device)
        shut.scatter_(1, rank.topk(case["top_groups"], dim=1).indices, False)
        key = per.masked_fill(shut[:, :, None], NEG).view(tokens, n)
    best = key.topk(case["topk"], dim=1)
    w = scores.gather(1, best.indices) * (best.values > NEG)
    if case["renormalize"]:
        w = torch.nan_to_num(w / w.sum(1, keepdim=True))
    out = {"experts": None, "weights": case["scale"] * w}
    if s["logits"].dtype == torch.bfloat16 and s["bias"] is None and groups > 1:
        out["weights"] = None  # groups of equal rank go by their index, which topk does not keep
    if case["scores"]:
        out["scores"] = scores
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(s, case)
    if op == "route_backward":
        x = s["logits"].double().requires_grad_()
        scores = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, dim=1)
        w = scores.gather(1, s["experts"].long())
        if case["renormalize"]:
            w = w / w.sum(1, keepdim=True)
        loss = (case["scale"] * w * s["dweights"].double()).sum()
        if s["dscores"] is not None:
            loss = loss + (scores * s["dscores"].double()).sum()
        loss.backward()
        return {"dlogits": x.grad}
    w = s["weight"].double()
    if op == "norm":
        out, h = {}, s["x"].double()
        if s["residual"] is not None:
            out["h"] = h + s["residual"].double()
            h = out["h"].float().to(_dtype(case["stream"])).double()  # the norm is of the stream as it is stored
        out["rstd"] = (h.pow(2).sum(1) / case["width"] + EPS).rsqrt()
        y = h * out["rstd"][:, None] * w
        if case["bf16"]:
            out["y"] = y
        if case["quantize"]:
            out["codes"], out["scales"] = _quantize64(_normalised64(h, out["rstd"][:, None], w), case["mode"])
        return out
    h, r = s["h"].double(), s["rstd"].double()[:, None]
    if op == "norm_backward":
        dy = s["dy"].double()
        dx = r * dy * w - r.pow(3) * h * ((dy * w) * h).mean(1, keepdim=True)
        if s["dres"] is not None:
            dx = dx + s["dres"].double()
        out = {"dx": dx, "dweight": torch.einsum("tn,tn->n", dy, h * r)}
        if case["quantize"]:
            g = _r32(dy * w)
            d = _r32(_r32(g - _r32(_r32(h * r) * _r32((g * h).mean(1, keepdim=True) * r))) * r)
            out["codes"], out["scales"] = _quantize64(_bf16(d if s["dres"] is None else d + s["dres"].double()), case["mode"])
        return out
    y = _normalised64(h, r, w)
    if s["index"] is not None:
        y = torch.cat([y, torch.zeros_like(y[:1])])[s["index"].long()]  # -1: the zero row behind the last token
    codes, scales = _quantize64(y.T, case["mode"])
    return {"codes": codes, "scales": scales}


# ------------------------------------------------------------------- work ----

def _size(name):
    return 2 if name == "bfloat16" else 4


def work(case):
    op = case["op"]
    if op.startswith("norm"):
        rows, width = case["rows"], case["width"]
        n, tiles, w = rows * width, rows * -(-width // TILE), width * _size(case["weight"])
        if op == "norm":
            total = n * _size(case["x"]) + w + 4 * rows
            if case["stream"]:
                total += 2 * n * _size(case["stream"])
            total += (2 * n if case["bf16"] else 0) + (n + 4 * tiles if case["quantize"] else 0)
            return {"bytes": total, "flops": 6 * n}
        if op == "norm_backward":
            total = n * (_size(case["dy"]) + _size(case["h"]) + _size(case["out"]) * (2 if case["dres"] else 1)) + w + 4 * rows + 4 * width
            return {"bytes": total + (n + 4 * tiles if case["quantize"] else 0), "flops": 10 * n}
        out_rows = _expert_rows(case).numel() if case["groups"] else rows
        read = min(rows, case["tokens"]) if case["groups"] else rows
        total = read * (width * _size(case["h"]) + 4) + w + out_rows * width + 4 * width * -(-out_rows // TILE) + (4 * out_rows if case["groups"] else 0)
        return {"bytes": total, "flops": 4 * n}
    tokens, n, topk = case["tokens"], case["experts"], case["topk"]
    if op == "route":
        total = tokens * (n * _size(case["logits"]) + 8 * topk) + (4 * n if case["bias"] else 0) + (4 * tokens * n if case["scores"] else 0)
        return {"bytes": total, "flops": 20 * tokens * n}
    # without the gradient of all scores, a sigmoid router's logits and the renormalised softmax's matter at the chosen experts alone
    read = n if case["dscores"] or (case["score"] == "softmax" and not case["renormalize"]) else topk
    total = tokens * (read * _size(case["logits"]) + n * _size(case["out"]) + 8 * topk) + (4 * tokens * n if case["dscores"] else 0)
    return {"bytes": total, "flops": 20 * tokens * read}
