"""The operators of an expert (MoE) layer around the FP8 matrix products, as they are measured: routing table, weighted
sum per token and its gradient, SwiGLU's gradient, and the weight gradient of every expert.

`own` false: the plain form, elementary torch operations in float32, rounded once at the end.  `own` true: the calls of
fine_grained_fp8_fp8q_amd that a training or serving program makes."""
import math

import torch

own = False

DEV = "cuda:0"
TILE = 128
E4M3_MAX = 448.0


def listed():
    return [
        # one decoded token, every expert on this device: the latency of the routing table
        dict(name="sort_decode_t1", op="sort", tokens=1, topk=8, experts=256, hosted=256, first=0, align=1, index="int32"),
        # one device's 16 of 256 experts, a long training batch, groups padded to the 128-token tiles of the weight gradient
        dict(name="sort_train_t16384", op="sort", tokens=16384, topk=8, experts=256, hosted=16, first=32, align=128, index="int64"),
        # one decoded token: its eight expert rows summed
        dict(name="combine_decode_t1", op="combine", tokens=1, topk=8, width=7168, experts=256, hosted=256, weighted=True, out="bfloat16"),
        # a batch of prompts, every expert on this device
        dict(name="combine_prefill_t4096", op="combine", tokens=4096, topk=8, width=7168, experts=64, hosted=64, weighted=True, out="bfloat16"),
        # the dispatch's gradient: rows of 16 hosted experts added back to their tokens in float32, no weights, most tokens without a row
        dict(name="combine_dispatch_grad_t8192", op="combine", tokens=8192, topk=8, width=7168, experts=256, hosted=16, weighted=False, out="float32"),
        # the backward pass's first step, its rows written as E4M3 for the down-projection's activation gradient
        dict(name="combine_backward_fp8_t4096", op="combine_backward", tokens=4096, topk=8, width=7168, experts=64, hosted=64, align=1, quantize=True, mode="free"),
        # a small odd layer, rows in BF16, groups padded to 128
        dict(name="combine_backward_odd_t1001", op="combine_backward", tokens=1001, topk=6, width=1030, experts=32, hosted=16, align=128, quantize=False, mode="free"),
        # gradients from the FP8 cache of the up-projection's output, and the activation recomputed for the weight gradient
        dict(name="swiglu_backward_cache_32768", op="swiglu_backward", rows=32768, inter=2048, cache=True, want_y=True),
        # a short ragged batch, the BF16 input kept
        dict(name="swiglu_backward_bf16_777", op="swiglu_backward", rows=777, inter=1000, cache=False, want_y=False),
        # up-projections of 16 experts, 8192 tokens' share: few rows an expert, the float32 gradients' own size decides
        dict(name="grouped_wgrad_up_4096", op="grouped_wgrad", rows=4096, groups=16, nout=4096, kin=7168, mode="free"),
        # down-projections, a long batch with power-of-two scales: the matrix products decide
        dict(name="grouped_wgrad_down_32768", op="grouped_wgrad", rows=32768, groups=16, nout=7168, kin=2048, mode="pow2"),
        # small experts with odd widths
        dict(name="grouped_wgrad_small_900", op="grouped_wgrad", rows=900, groups=8, nout=360, kin=520, mode="free"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["sort", "combine", "combine_backward", "swiglu_backward", "grouped_wgrad"])
    experts = rng.choice([8, 20, 64, 160, 256])
    hosted = max(1, experts // rng.choice([1, 1, 4, 8]))
    topk = rng.choice([1, 2, 4, 6, 8])
    if op == "sort":
        return dict(op=op, tokens=_log(rng, 1, 32768), topk=topk, experts=experts, hosted=hosted, first=rng.choice([0, experts - hosted]),
                    align=rng.choice([1, 16, 128]), index=rng.choice(["int32", "int64"]))
    if op == "combine":
        return dict(op=op, tokens=_log(rng, 1, 4096), topk=topk, width=_log(rng, 64, 7168), experts=experts, hosted=hosted,
                    weighted=rng.random() < 0.7, out=rng.choice(["bfloat16", "float32"]))
    if op == "combine_backward":
        return dict(op=op, tokens=_log(rng, 1, 4096), topk=topk, width=_log(rng, 64, 7168), experts=experts, hosted=hosted,
                    align=rng.choice([1, 128]), quantize=rng.random() < 0.5, mode=rng.choice(["free", "pow2"]))
    if op == "swiglu_backward":
        cache = rng.random() < 0.5
        inter = TILE * rng.randint(1, 16) if cache else _log(rng, 32, 2048)
        return dict(op=op, rows=_log(rng, 1, 32768), inter=inter, cache=cache, want_y=rng.random() < 0.5)
    return dict(op=op, rows=_log(rng, 1, 16384), groups=rng.choice([1, 4, 8, 16]), nout=_log(rng, 64, 4096), kin=_log(rng, 64, 4096),
                mode=rng.choice(["free", "pow2"]))


# ---------------------------------------------------------------- inputs ----

def _pad(n, to):
    return (n + to - 1) // to * to


def _capacity(case):
    """Rows of the expert-sorted buffer: every pair that can land here, or half as many again as the mean where only a share does."""
    pairs, align = case["tokens"] * case["topk"], case.get("align", 1)
    if case["hosted"] < case["experts"]:
        share = pairs * case["hosted"] / case["experts"]
        pairs = min(pairs, int(1.5 * share + 6 * math.sqrt(share) + 8))
    return _pad(pairs + case["hosted"] * (align - 1), align)


def _route(case, gen, spread):
    """Expert of every (token, choice) pair: the best `topk` of a popularity that falls off with the rank, plus noise."""
    rank = torch.randperm(case["experts"], generator=torch.Generator().manual_seed(7)).to(DEV) + 1
    noise = torch.rand((case["tokens"], case["experts"]), generator=gen, device=DEV).clamp_(1e-9, 1 - 1e-7)
    score = -torch.log(-torch.log(noise)) - spread * torch.log(rank.float())
    weights, experts = torch.topk(score, case["topk"], dim=1)
    return experts, torch.softmax(weights, dim=1).float().contiguous()


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


def _group_rows(case):
    """Rows of each group: popularity falls off with the rank, one group in eight is empty (host numbers, the same for every seed)."""
    g, left = case["groups"], case["rows"]
    share = [0.0 if i % 8 == 3 else 1.0 / (1 + (5 * i) % g) for i in range(g)]
    rows = [int(left * s / sum(share)) for s in share]
    rows[0] += left - sum(rows)
    return rows


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    s = {"case": case}
    op = case["op"]
    if op == "sort":
        experts, _ = _route(case, gen, 1.1)
        s["experts"], s["cap"] = experts.to(getattr(torch, case["index"])).contiguous(), _capacity(case)
    elif op in ("combine", "combine_backward"):
        experts, weights = _route(case, gen, 0.0)
        s["cap"] = _capacity(case)
        _, s["token"], s["row_of"] = _plain_sort(experts, case["hosted"], 0, case.get("align", 1), s["cap"])
        s["weights"] = weights if case.get("weighted", True) else None
        s["y"] = normal(s["cap"], case["width"]).to(torch.bfloat16)
        if op == "combine_backward":
            s["dout"] = normal(case["tokens"], case["width"]).to(torch.bfloat16)
    elif op == "swiglu_backward":
        x = (1.7 * normal(case["rows"], 2 * case["inter"])).to(torch.bfloat16)
        s["dy"] = normal(case["rows"], case["inter"]).to(torch.bfloat16)
        if case["cache"]:
            codes, s["x_scales"] = _quantize(x.float(), "pow2")
            s["x"] = codes.contiguous().view(torch.uint8)
        else:
            s["x"], s["x_scales"] = x, None
    else:
        rows = _group_rows(case)
        padded = [_pad(r, TILE) for r in rows]
        cap = max(TILE, sum(padded))
        starts = [sum(padded[:i]) for i in range(len(padded) + 1)]
        s["offsets"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
        s["most"] = max(padded)
        real = torch.zeros(cap, device=DEV)
        for r, at in zip(rows, starts):
            real[at:at + r] = 1.0
        for name, width in (("dy", case["nout"]), ("x", case["kin"])):
            codes, s[name + "_scales"] = _quantize((normal(width, cap) * real).to(torch.bfloat16).float(), case["mode"])
            s[name + "_t"] = codes.contiguous().view(torch.uint8)
    return s


# ------------------------------------------------------------ plain forms ----

def _plain_sort(experts, hosted, first, align, cap):
    tokens, topk = experts.shape
    local = experts.reshape(-1).long() - first
    here = (local >= 0) & (local < hosted)
    key, order = torch.sort(torch.where(here, local, hosted), stable=True)
    counts = (key[:, None] == torch.arange(hosted, device=key.device)).sum(0)
    padded = (counts + align - 1) // align * align
    ends = torch.cumsum(padded, 0)
    before = torch.cat([torch.cumsum(counts, 0) - counts, counts.sum()[None]])
    starts = torch.cat([ends - padded, ends[-1:]])
    row = starts[key] + torch.arange(key.numel(), device=key.device) - before[key]
    fits = (key < hosted) & (row < cap)
    row_of = torch.empty_like(order)
    row_of[order] = torch.where(fits, row, -1)
    token = torch.full((cap + 1,), -1, dtype=torch.long, device=key.device)
    token[torch.where(fits, row, cap)] = torch.where(fits, order // topk, -1)
    offsets = torch.cat([ends.new_zeros(1), ends]).clamp(max=cap)
    return offsets.int(), token[:cap].int(), row_of.view(tokens, topk).int()


def _pair_rows(y, row_of, dtype):
    """y[row_of] as [tokens, topk, width], zeros for pairs without a row."""
    return torch.where((row_of >= 0)[:, :, None], y[row_of.clamp(min=0).long()].to(dtype), torch.zeros((), dtype=dtype, device=y.device))


def _to_rows(pairs, row_of, cap):
    """[tokens, topk, width] values written to their rows of [cap, width]; rows without a pair are zero."""
    rows = torch.zeros((cap + 1, pairs.shape[2]), dtype=pairs.dtype, device=pairs.device)
    rows[torch.where(row_of >= 0, row_of, cap).reshape(-1).long()] = pairs.reshape(-1, pairs.shape[2])
    return rows[:cap]


def _values(codes, scales, dtype):
    """Values of [rows, cols] E4M3 codes with 1x128 scales."""
    s = scales.to(dtype).repeat_interleave(TILE, dim=1)[:, :codes.shape[1]]
    return codes.view(torch.float8_e4m3fn).to(dtype) * s


def _by_group(values, offsets, most):
    """[width, cap] -> [groups, width, most]: each group's columns, zeros behind its end."""
    lo, hi = offsets[:-1].long(), offsets[1:].long()
    at = lo[:, None] + torch.arange(most, device=values.device)
    inside = at < hi[:, None]
    picked = values[:, torch.where(inside, at, 0).reshape(-1)].view(values.shape[0], *at.shape)
    return torch.where(inside, picked, torch.zeros((), dtype=values.dtype, device=values.device)).permute(1, 0, 2).contiguous()


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "sort":
        offsets, token, row_of = _plain_sort(s["experts"], case["hosted"], case["first"], case["align"], s["cap"])
        return {"offsets": offsets, "token": token, "row_of": row_of}
    if op == "combine":
        rows = _pair_rows(s["y"], s["row_of"], torch.float32)
        if s["weights"] is not None:
            rows = rows * s["weights"][:, :, None]
        return {"out": rows.sum(1).to(getattr(torch, case["out"]))}
    if op == "combine_backward":
        dout = s["dout"].float()[:, None, :]
        dweights = (_pair_rows(s["y"], s["row_of"], torch.float32) * dout).sum(2)
        dy = _to_rows(dout * s["weights"][:, :, None], s["row_of"], s["cap"]).to(torch.bfloat16)
        if not case["quantize"]:
            return {"dy": dy, "dweights": dweights}
        codes, scales = _quantize(dy.float(), case["mode"])
        return {"codes": codes, "scales": scales, "dweights": dweights}
    if op == "swiglu_backward":
        x = s["x"].float() if s["x_scales"] is None else _values(s["x"], s["x_scales"], torch.float32)
        gate, up = x[:, :case["inter"]], x[:, case["inter"]:]
        dy, sig = s["dy"].float(), 1.0 / (1.0 + torch.exp(-gate))
        dx = torch.cat([dy * up * sig * (1.0 + gate * (1.0 - sig)), dy * gate * sig], dim=1).to(torch.bfloat16)
        return {"dx": dx, "y": (gate * sig * up).to(torch.bfloat16)} if case["want_y"] else {"dx": dx}
    dy = _by_group(_values(s["dy_t"], s["dy_scales"], torch.float32), s["offsets"], s["most"])
    x = _by_group(_values(s["x_t"], s["x_scales"], torch.float32), s["offsets"], s["most"])
    return {"dw": torch.bmm(dy, x.transpose(1, 2).contiguous())}


def run(s):
    if not own:
        return _plain(s)
    import fine_grained_fp8_fp8q_amd as fp8q
    case = s["case"]
    op = case["op"]
    if op == "sort":
        offsets, token, row_of = fp8q.moe_sort(s["experts"], case["hosted"], first=case["first"], align=case["align"], rows_cap=s["cap"])
        return {"offsets": offsets, "token": token, "row_of": row_of}
    if op == "combine":
        return {"out": fp8q.moe_combine(s["y"], s["row_of"], s["weights"], out_dtype=getattr(torch, case["out"]))}
    if op == "combine_backward":
        dy, codes, scales, dweights = fp8q.moe_combine_backward(s["dout"], s["y"], s["row_of"], s["weights"], s["token"],
                                                                bf16=not case["quantize"], quantize=case["quantize"], scale_mode=case["mode"])
        if not case["quantize"]:
            return {"dy": dy, "dweights": dweights}
        return {"codes": codes.view(torch.float8_e4m3fn), "scales": scales, "dweights": dweights}
    if op == "swiglu_backward":
        dx, y, _, _ = fp8q.swiglu_backward(s["x"], s["dy"], x_scales=s["x_scales"], want_y=case["want_y"])
        return {"dx": dx, "y": y} if case["want_y"] else {"dx": dx}
    acc = "fp32" if case["mode"] == "free" else "fp32_pow2"
    return {"dw": fp8q.grouped_wgrad(s["dy_t"], s["dy_scales"], s["x_t"], s["x_scales"], s["offsets"], acc=acc)}


# ------------------------------------------------------- 64-bit definition ----

def _quantize64(x, mode):
    """The tile quantizer of BF16 values held in 64 bits: codes and scales as float64 values."""
    rows, cols = x.shape
    width = -(-cols // TILE)
    tiles = torch.zeros((rows, width * TILE), dtype=torch.float64, device=x.device)
    tiles[:, :cols] = x
    tiles = tiles.view(rows, width, TILE)
    amax = tiles.abs().max(dim=2).values
    if mode == "free":
        scale = (amax / E4M3_MAX).float().double()
    else:
        scale = torch.where(amax > 0, torch.exp2(torch.ceil(torch.log2((amax / E4M3_MAX).clamp(min=1e-300)))), amax)
    q = (tiles / scale.clamp(min=1e-300)[:, :, None]).float().to(torch.float8_e4m3fn).double()
    return q.reshape(rows, -1)[:, :cols], scale


def exact(case, seed):
    op = case["op"]
    if op == "sort":
        return None
    s = prepare(case, seed)
    if op == "combine":
        out = torch.zeros((case["tokens"], case["width"]), dtype=torch.float64, device=DEV)
        for j in range(case["topk"]):
            t = torch.nonzero(s["row_of"][:, j] >= 0)[:, 0]
            part = s["y"][s["row_of"][t, j].long()].double()
            out[t] += part if s["weights"] is None else part * s["weights"][t, j, None].double()
        return {"out": out}
    if op == "combine_backward":
        dy = torch.zeros((s["cap"], case["width"]), dtype=torch.float64, device=DEV)
        dweights = torch.zeros((case["tokens"], case["topk"]), dtype=torch.float64, device=DEV)
        for j in range(case["topk"]):
            t = torch.nonzero(s["row_of"][:, j] >= 0)[:, 0]
            r = s["row_of"][t, j].long()
            dout = s["dout"][t].double()
            dy[r] = dout * s["weights"][t, j, None].double()
            dweights[t, j] = (dout * s["y"][r].double()).sum(1)
        if not case["quantize"]:
            return {"dy": dy, "dweights": dweights}
        codes, scales = _quantize64(dy.to(torch.bfloat16).double(), case["mode"])
        return {"codes": codes, "scales": scales, "dweights": dweights}
    if op == "swiglu_backward":
        n = case["inter"]
        x = s["x"].double() if s["x_scales"] is None else _values(s["x"], s["x_scales"], torch.float64)
        g, u, d = x[:, :n], x[:, n:], s["dy"].double()
        sig = torch.sigmoid(g)
        dx = torch.empty_like(x)
        dx[:, :n] = d * u * (sig + g * sig * torch.sigmoid(-g))
        dx[:, n:] = d * g * sig
        return {"dx": dx, "y": g * u * sig} if case["want_y"] else {"dx": dx}
    dw = torch.zeros((case["groups"], case["nout"], case["kin"]), dtype=torch.float64, device=DEV)
    at = s["offsets"].tolist()
    dy, x = _values(s["dy_t"], s["dy_scales"], torch.float64), _values(s["x_t"], s["x_scales"], torch.float64)
    for g in range(case["groups"]):
        dw[g] = dy[:, at[g]:at[g + 1]] @ x[:, at[g]:at[g + 1]].T.contiguous()
    return {"dw": dw}


# ------------------------------------------------------------------- work ----

def work(case):
    op = case["op"]
    if op == "sort":
        pairs = case["tokens"] * case["topk"]
        return {"bytes": pairs * (4 if case["index"] == "int32" else 8) + 4 * (pairs + _capacity(case) + case["hosted"] + 1), "flops": 0}
    if op in ("combine", "combine_backward"):
        pairs, width = case["tokens"] * case["topk"], case["width"]
        rows = pairs * case["hosted"] / case["experts"]
        if op == "combine":
            out = 2 if case["out"] == "bfloat16" else 4
            return {"bytes": 2 * rows * width + out * case["tokens"] * width + (8 if case["weighted"] else 4) * pairs,
                    "flops": 2 * rows * width}
        cap = _capacity(case)
        written = cap * (width + 4 * -(-width // TILE)) if case["quantize"] else 2 * cap * width
        return {"bytes": 2 * rows * width + 2 * case["tokens"] * width + written + 12 * pairs + 4 * cap, "flops": 3 * rows * width}
    if op == "swiglu_backward":
        n = case["rows"] * case["inter"]
        read = 2 * n + 8 * n / TILE if case["cache"] else 4 * n
        return {"bytes": read + 2 * n + 4 * n + (2 * n if case["want_y"] else 0), "flops": 20 * n}
    rows = case["rows"]
    return {"bytes": rows * (case["nout"] + case["kin"]) * (1 + 4 / TILE) + 4 * case["groups"] * case["nout"] * case["kin"],
            "flops": 2 * rows * case["nout"] * case["kin"]}
