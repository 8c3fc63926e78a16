"""The expert layer around the grouped GEMMs on the GPU: routing table,
weighted sum and its gradient, SwiGLU's gradient, per-expert weight gradient,
and a whole expert layer, against the 64-bit oracle (oracle/moe_layer.py)."""

import numpy as np
import pytest
import torch

import fine_grained_fp8_fp8q_amd as fp8q
from oracle import e4m3, moe_layer as M, quantize as Q
from tests.gpu_util import (assert_codes_equal, assert_scales_equal, dev, dev_bf16, host, host_bf16_bits, host_codes,
                            need_gpu, say)

pytestmark = pytest.mark.gpu
U32, U16 = 2.0 ** -24, 2.0 ** -8  # half a step of float32 and BF16, relative
TINY16 = 2.0 ** -134              # half the smallest BF16 subnormal


@pytest.fixture(autouse=True)
def _gpu(request):
    need_gpu()
    say(f"[moe layer] {request.node.name}")


def bf16(r, shape, std=1.0):
    return e4m3.f32_to_bf16_bits_rne((r.normal(size=shape) * std).astype(np.float32))


def f64(bits):
    return e4m3.bf16_bits_to_f64(bits)


def spread(t, pad, fill):
    """t [rows, cols] as a view of a wider buffer filled with `fill`."""
    buf = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device=t.device)
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]]


def routing(r, tokens, topk, experts, zipf=0.0):
    score = r.gumbel(size=(tokens, experts)) - zipf * np.log(1 + r.permutation(experts))
    return np.argsort(-score, axis=1, kind="stable")[:, :topk].astype(np.int64)


# ------------------------------------------------------------------ sort ----

def check_sort(experts, first, groups, align, cap, dtype=torch.int64):
    got = fp8q.moe_sort(dev(experts).to(dtype), groups, first=first, align=align, rows_cap=cap)
    want = M.sort(experts, first, groups, align, cap)
    for name, g, w in zip(("offsets", "token", "row_of"), got, want):
        assert g.dtype == torch.int32 and np.array_equal(host(g), w), name


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("tokens,topk,experts,first,groups,align", [
    (1, 1, 1, 0, 1, 1), (1, 8, 256, 0, 256, 1), (3, 2, 5, 2, 1, 128), (63, 1, 7, 0, 7, 16), (64, 6, 20, 10, 10, 4),
    (257, 8, 256, 32, 16, 128), (511, 8, 64, 0, 64, 1), (513, 8, 512, 0, 512, 128), (1000, 9, 33, 1, 31, 3),
    (5000, 3, 40, 0, 40, 1), (16384, 8, 256, 32, 16, 128), (20011, 7, 300, 0, 300, 16)])
def test_sort(dtype, tokens, topk, experts, first, groups, align):
    e = routing(np.random.default_rng(tokens), tokens, topk, experts, zipf=1.1)
    cap = -(-(tokens * topk + groups * (align - 1)) // align) * align
    check_sort(e, first, groups, align, cap, dtype)


@pytest.mark.parametrize("tokens", [40, 9000])
def test_sort_drops_what_does_not_fit_and_takes_any_expert_number(tokens):
    r = np.random.default_rng(8)
    e = r.integers(-3, 9, size=(tokens, 4))  # repeats within a token, numbers below and above
    e[0] = [2 ** 40, -2 ** 62, 2 ** 62 - 1, 3]
    for align in (1, 8):
        for cap in (0, 8, tokens // 8 * 8, tokens * 8):
            check_sort(e, 1, 6, align, cap)
    check_sort(np.full((tokens, 4), 5), 5, 1, 1, tokens * 4)      # all to one expert
    check_sort(np.full((tokens, 4), 77), 0, 5, 128, 128)          # none here


def test_sort_without_tokens_or_experts():
    offsets, token, row_of = fp8q.moe_sort(torch.empty((0, 8), dtype=torch.int64, device="cuda:0"), 3, align=128, rows_cap=256)
    assert host(offsets).tolist() == [0] * 4 and host(token).tolist() == [-1] * 256 and row_of.shape == (0, 8)
    offsets, token, row_of = fp8q.moe_sort(torch.zeros((2, 3), dtype=torch.int32, device="cuda:0"), 0)
    assert host(offsets).tolist() == [0] and host(row_of).tolist() == [[-1] * 3] * 2


def test_sort_of_a_column_slice():
    e = routing(np.random.default_rng(2), 700, 8, 64)
    wide = dev(e)
    got = fp8q.moe_sort(wide[:, :5], 64, rows_cap=3500)
    for g, w in zip(got, M.sort(e[:, :5], 0, 64, 1, 3500)):
        assert np.array_equal(host(g), w)
    with pytest.raises(ValueError, match="contiguous rows"):
        fp8q.moe_sort(wide[:, ::2], 64)
    with pytest.raises(fp8q.Fp8qError):  # rows over one another
        fp8q.moe_sort(wide[:1].expand(700, 8), 64)
    with pytest.raises(fp8q.Fp8qError):
        fp8q.moe_sort(wide, 64, align=128, rows_cap=100)


def check_sort_by_rules(experts, first, groups, align, cap):
    """The same conditions without the oracle's loops, for many pairs: every hosted pair has a row of its group, the
    rows of a group are its pairs in ascending order, and everything else is -1."""
    offsets, token, row_of = (host(v).astype(np.int64) for v in fp8q.moe_sort(dev(experts), groups, first=first, align=align, rows_cap=cap))
    flat, topk = experts.reshape(-1), experts.shape[1]
    counts = np.array([(flat == first + g).sum() for g in range(groups)])
    starts = np.concatenate([[0], np.cumsum(-(-counts // align) * align)])
    assert np.array_equal(offsets, np.minimum(starts, cap))
    want_token, want_row = np.full(cap, -1), np.full(flat.size, -1)
    for g in range(groups):
        p = np.flatnonzero(flat == first + g)
        rows = starts[g] + np.arange(p.size)
        fits = rows < cap
        want_row[p[fits]] = rows[fits]
        want_token[rows[fits]] = p[fits] // topk
    assert np.array_equal(row_of.reshape(-1), want_row) and np.array_equal(token, want_token)


@pytest.mark.parametrize("tokens,topk,experts,first,groups,align", [
    (150001, 8, 64, 0, 64, 128), (400003, 3, 9, 2, 5, 1), (262145, 4, 512, 0, 512, 16), (1100000, 1, 3, 0, 3, 1), (2048, 2, 4, 0, 4, 1),
    (2049, 2, 4, 0, 4, 1), (2000, 1, 8, 0, 8, 2048), (9000, 2, 5, 1, 3, 1500), (40, 2, 160, 0, 160, 1024)])
def test_sort_of_many_pairs(tokens, topk, experts, first, groups, align):
    """More pairs than the kernel keeps in registers between its passes (above a million), both sides of the
    size from which more than one workgroup counts, and long paddings."""
    e = np.random.default_rng(tokens).integers(0, experts, size=(tokens, topk))
    cap = -(-(tokens * topk + groups * align) // align) * align
    check_sort_by_rules(e, first, groups, align, cap)
    check_sort_by_rules(e, first, groups, align, cap // 3 // align * align)


# --------------------------------------------------------------- combine ----

COMBINE = [(1, 8, 7168, 256, 256), (5, 1, 8, 4, 4), (3, 3, 1, 4, 2), (17, 6, 1030, 32, 16), (64, 8, 2048, 8, 8), (33, 12, 513, 20, 20),
           (100, 2, 129, 64, 3), (9, 17, 4104, 18, 18)]


def pairs(r, tokens, topk, experts, hosted, align=1):
    e = routing(r, tokens, topk, experts)
    cap = -(-(tokens * topk + hosted * (align - 1)) // align) * align
    offsets, token, row_of = M.sort(e, 0, hosted, align, cap)
    return offsets, token, row_of, cap


def assert_near(got, want, bound, what):
    got = np.asarray(got, dtype=np.float64)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off, first {np.argwhere(bad)[0]}: {got[bad][0]} for {want[bad][0]}"


@pytest.mark.parametrize("ydt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("odt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,topk,n,experts,hosted", COMBINE)
def test_combine(ydt, odt, tokens, topk, n, experts, hosted):
    r = np.random.default_rng(n)
    _, token, row_of, cap = pairs(r, tokens, topk, experts, hosted)
    yv = f64(bf16(r, (cap, n))) if ydt == torch.bfloat16 else r.normal(size=(cap, n)).astype(np.float32).astype(np.float64)
    yv[token < 0] = np.nan  # rows that no pair names
    y = torch.from_numpy(yv).to("cuda:0").to(ydt)
    w = r.random(size=(tokens, topk)).astype(np.float32)
    for weights in (w, None):
        want, mag = M.combine(yv, row_of, weights)
        # topk fused multiply-adds, then one rounding
        bound = 1.01 * topk * U32 * mag + ((U16 * np.abs(want) * (1 + topk * U32)) if odt == torch.bfloat16 else 0) + 2.0 ** -149
        wd = None if weights is None else dev(weights)
        for pad in (0, 8, 3):
            out = spread(torch.zeros((tokens, n), dtype=odt, device="cuda:0"), pad, 7.0)
            got = fp8q.moe_combine(spread(y, pad, float("nan")), dev(row_of.astype(np.int32)), wd, out=out)
            assert got.data_ptr() == out.data_ptr()
            assert_near(host(got.float()), want, bound, f"pad {pad}")
            if pad:
                assert (host(out._base[:, n:].float()) == 7.0).all()
        assert torch.equal(fp8q.moe_combine(y, dev(row_of.astype(np.int32)), wd, out_dtype=odt), got)


def test_combine_rows_outside_and_non_finite_values():
    y = torch.tensor([[1.0, np.inf], [2.0, np.nan], [3.0, -np.inf]], dtype=torch.float32, device="cuda:0")
    rows = dev(np.array([[0, -1], [2 ** 31 - 1, 3], [0, 2], [1, 0]], dtype=np.int32))
    w = dev(np.array([[2, np.nan], [np.inf, np.nan], [1, 1], [0, 1]], dtype=np.float32))
    got = host(fp8q.moe_combine(y, rows, w, out_dtype=torch.float32))
    assert got[0].tolist() == [2.0, np.inf] and got[1].tolist() == [0.0, 0.0]
    assert got[2][0] == 4.0 and np.isnan(got[2][1]) and got[3][0] == 1.0 and np.isnan(got[3][1])
    b = fp8q.moe_combine(y.bfloat16(), rows, w)
    assert np.isinf(host(b.float())[0, 1]) and np.isnan(host(b.float())[3, 1])


def test_combine_empty():
    y = torch.zeros((0, 16), dtype=torch.bfloat16, device="cuda:0")
    rows = torch.zeros((5, 2), dtype=torch.int32, device="cuda:0")
    assert (host(fp8q.moe_combine(y, rows).float()) == 0).all()
    assert (host(fp8q.moe_combine(y, rows[:, :0], out_dtype=torch.float32)) == 0).all()
    assert fp8q.moe_combine(y, rows[:0]).shape == (0, 16)


def test_no_rows_and_no_row_stride():
    """rows_cap = 0 with ld_y = 0: the sum and its gradient with respect to the weights are zero."""
    lib = fp8q.load_library()
    rows = torch.zeros((5, 2), dtype=torch.int32, device="cuda:0")
    dout = torch.ones((5, 16), dtype=torch.bfloat16, device="cuda:0")
    out, dw = torch.full((5, 16), 7.0, device="cuda:0"), torch.full((5, 2), 7.0, device="cuda:0")
    stream = torch.cuda.current_stream().cuda_stream
    assert lib.fp8q_moe_combine(None, 1, 0, 16, 0, rows.data_ptr(), None, 5, 2, 0, out.data_ptr(), 16, stream) == fp8q.OK
    assert lib.fp8q_moe_combine_backward(dout.data_ptr(), 1, 5, 16, 16, out.data_ptr(), 1, 0, 0, rows.data_ptr(), None, 2, None,
                                         None, 0, 0, None, 0, None, dw.data_ptr(), stream) == fp8q.OK
    assert (host(out) == 0).all() and (host(dw) == 0).all()


# ------------------------------------------------------ combine backward ----

@pytest.mark.parametrize("ddt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("ydt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,topk,n,experts,hosted", COMBINE)
def test_combine_backward(ddt, ydt, tokens, topk, n, experts, hosted):
    r = np.random.default_rng(n + 1)
    align = 128 if hosted < 100 else 1
    _, token, row_of, cap = pairs(r, tokens, topk, experts, hosted, align)
    yv, dv = f64(bf16(r, (cap, n))), f64(bf16(r, (tokens, n)))
    w = r.random(size=(tokens, topk)).astype(np.float32)
    yv[token < 0] = np.nan
    y, dout = torch.from_numpy(yv).to("cuda:0").to(ydt), torch.from_numpy(dv).to("cuda:0").to(ddt)
    rows_d, token_d = dev(row_of.astype(np.int32)), dev(token.astype(np.int32))
    # additions behind one another: eight a chunk in each lane (a workgroup of at least 64 lanes goes over the row in
    # steps of 512 columns or more), six between lanes, three between waves
    depth = 8 * (-(-n // 512)) + 10
    for weights, mode, pad in ((w, "free", 0), (None, "pow2", 5), (w, "pow2", 8)):
        want_dy, want_dw, mag = M.combine_backward(dv, yv, row_of, weights)
        w32 = (np.ones_like(w) if weights is None else weights)
        bits = np.zeros((cap, n), dtype=np.uint16)
        has = row_of >= 0
        for t, j in zip(*np.nonzero(has)):  # one float32 product, one rounding to BF16
            bits[row_of[t, j]] = e4m3.f32_to_bf16_bits_rne(w32[t, j] * dv[t].astype(np.float32))
        dy, codes, scales, dw = fp8q.moe_combine_backward(spread(dout, pad, 3.0), spread(y, pad, float("nan")), rows_d,
                                                          None if weights is None else dev(weights), token_d,
                                                          quantize=True, scale_mode=mode)
        assert np.array_equal(host_bf16_bits(dy), bits)
        oc, os_ = Q.quantize_rows(bits, Q.FREE if mode == "free" else Q.POW2)
        assert_codes_equal(host_codes(codes), oc, "codes")
        assert_scales_equal(host(scales), os_, "scales")
        assert_near(host(dw), want_dw, 1.01 * depth * U32 * mag + 2.0 ** -149, "dweights")
        assert (host(dw)[~has] == 0).all()
        # each output alone is the same
        only = fp8q.moe_combine_backward(dout, y, rows_d, None if weights is None else dev(weights), token_d, bf16=False,
                                         quantize=True, scale_mode=mode, want_dweights=False)
        assert only[0] is None and only[3] is None
        assert torch.equal(only[1], codes) and torch.equal(only[2], scales)


def test_combine_backward_leaves_rows_alone_without_the_token_list():
    r = np.random.default_rng(1)
    rows = np.array([[2, -1], [0, 5]], dtype=np.int32)  # row 5 is outside: 4 rows
    dout, y = dev_bf16(bf16(r, (2, 48))), dev_bf16(bf16(r, (4, 48)))
    lib, dy = fp8q.load_library(), torch.full((4, 56), 9.0, dtype=torch.bfloat16, device="cuda:0")
    dw = torch.full((2, 2), 9.0, device="cuda:0")
    rows_d = dev(rows)
    st = lib.fp8q_moe_combine_backward(dout.data_ptr(), 1, 2, 48, 48, y.data_ptr(), 1, 4, 48, rows_d.data_ptr(), None, 2, None,
                                       dy.data_ptr(), 56, 0, None, 0, None, dw.data_ptr(), None)
    assert st == fp8q.OK
    got = host(dy.float())
    assert (got[:, 48:] == 9).all() and (got[[1, 3]] == 9).all()
    assert torch.equal(dy[2, :48], dout[0]) and torch.equal(dy[0, :48], dout[1])
    assert host(dw)[0, 1] == 0 and host(dw)[1, 1] == 0


def test_combine_backward_empty():
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda:0")  # noqa: E731
    none = torch.full((3, 2), -1, dtype=torch.int32, device="cuda:0")
    minus = torch.full((7,), -1, dtype=torch.int32, device="cuda:0")
    dy, codes, scales, dw = fp8q.moe_combine_backward(z(3, 40) + 1, z(7, 40), none, None, minus, quantize=True)
    assert not host(dy.float()).any() and not host_codes(codes).any() and not host(scales).any() and not host(dw).any()
    dy, _, _, dw = fp8q.moe_combine_backward(z(0, 40), z(7, 40), none[:0], None, minus)
    assert not host(dy.float()).any() and dw.shape == (0, 2)
    assert not host(fp8q.moe_combine_backward(z(3, 40), z(0, 40), none)[3]).any()


@pytest.mark.parametrize("ddt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("ydt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [1, 7, 16, 520, 1027])
def test_combine_backward_non_finite_values(ddt, ydt, n):
    """Infinities and NaN in dout, y and the weights follow float32 arithmetic in the BF16 rows and in the weights'
    gradient; those of pairs without a row and of rows without a pair reach nothing."""
    r = np.random.default_rng(n)
    tokens, topk, cap = 8, 3, 40
    row_of = r.permutation(cap)[:tokens * topk].reshape(tokens, topk).astype(np.int32)
    row_of[1, 0], row_of[5, 2], row_of[6] = -1, cap, [2 ** 31 - 1, -2 ** 31, -7]
    has = (row_of >= 0) & (row_of < cap)
    token = np.full(cap, -1, dtype=np.int32)
    token[row_of[has]] = np.nonzero(has)[0]
    dv, yv = f64(bf16(r, (tokens, n))), f64(bf16(r, (cap, n)))
    w = r.random(size=(tokens, topk)).astype(np.float32)
    yv[row_of[7], 0] = 0.5  # (their products with 2^127 below stay finite)
    dv[0, n // 2], dv[2, 0], dv[3, n - 1], dv[6] = np.inf, np.nan, -np.inf, np.nan
    yv[row_of[4, 0], n - 1], yv[row_of[4, 1], 0], yv[row_of[7, 2], n // 3], yv[token < 0] = np.inf, np.nan, -np.inf, np.nan
    yv[row_of[3, 1], n - 1] = 0.0  # against an infinity of dout
    w[1, 0], w[4, 2], w[5, 0], w[7, 0], w[0, 1], w[6] = np.nan, np.inf, np.nan, -np.inf, 0.0, np.inf
    dv[7, 0] = 2.0 ** 127  # finite, and 2^127 times 3 is not
    w[7, 1] = 3.0
    y, dout = torch.from_numpy(yv).to("cuda:0").to(ydt), torch.from_numpy(dv).to("cuda:0").to(ddt)
    with np.errstate(invalid="ignore", over="ignore"):
        want = np.zeros((cap, n), dtype=np.float32)
        for t, j in zip(*np.nonzero(has)):
            want[row_of[t, j]] = w[t, j] * dv[t].astype(np.float32)
        terms = np.where(has[:, :, None], dv[:, None, :] * yv[np.where(has, row_of, 0)], 0.0)
        want_dw = terms.sum(2)
    bound = 1.01 * (8 * (-(-n // 512)) + 10) * U32 * np.abs(np.where(np.isfinite(terms), terms, 0.0)).sum(2) + 2.0 ** -149
    for pad in (0, 5):
        dy, _, _, dw = fp8q.moe_combine_backward(spread(dout, pad, 3.0), spread(y, pad, 3.0), dev(row_of), dev(w), dev(token))
        assert np.array_equal(host(dy.float()), host(torch.from_numpy(want).bfloat16().float()), equal_nan=True), pad
        dw = host(dw).astype(np.float64)
        fin = np.isfinite(want_dw)
        assert np.array_equal(dw[~fin], want_dw[~fin], equal_nan=True), pad
        assert_near(dw[fin], want_dw[fin], bound[fin], "dweights")
        assert (dw[~has] == 0).all()


@pytest.mark.parametrize("tokens", [1, 3, 1024, 1025])
def test_combine_backward_of_rows_without_columns(tokens):
    """The weight gradients of an empty width are zeros, on both sides of 2048 pairs."""
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda:0")  # noqa: E731
    rows = torch.arange(2 * tokens, dtype=torch.int32, device="cuda:0").view(tokens, 2) - 1
    token = torch.full((2 * tokens,), -1, dtype=torch.int32, device="cuda:0")
    for quantize in (False, True):
        torch.full((tokens, 2), 7.0, device="cuda:0")  # (what the next allocation may find)
        dy, codes, scales, dw = fp8q.moe_combine_backward(z(tokens, 0), z(2 * tokens, 0), rows, None, token, quantize=quantize)
        assert dy.shape == (2 * tokens, 0) and dw.shape == (tokens, 2) and not host(dw).any()
        assert codes is None if not quantize else codes.shape == (2 * tokens, 0) and scales.shape == (2 * tokens, 0)


# ------------------------------------------------------- SwiGLU backward ----

# (the FP8 cache has whole tiles)
@pytest.mark.parametrize("rows,inter,cache", [(r, i, c) for r, i in ((1, 128), (3, 256), (130, 128), (77, 1024), (2, 2048)) for c in (None, "free", "pow2")] +
                         [(50, 7, None), (1, 1, None), (19, 1000, None), (33, 136, None)])
def test_swiglu_backward(rows, inter, cache):
    r = np.random.default_rng(rows * inter)
    xb, dyb = bf16(r, (rows, 2 * inter), 3.0), bf16(r, (rows, inter))
    if cache:
        xc, xs = Q.quantize_rows(xb, Q.FREE if cache == "free" else Q.POW2)
        x64 = (e4m3.decode(xc).astype(np.float32).reshape(rows, -1, 128) * xs[:, :, None]).reshape(rows, -1).astype(np.float64)
        x, scales = dev(xc), dev(xs)
    else:
        x64, x, scales = f64(xb), dev_bf16(xb), None
    want, y64, mag = M.swiglu_backward(x64, f64(dyb))
    dy = dev_bf16(dyb)
    for pad in (0, 8, 3):
        dx, y, _, _ = fp8q.swiglu_backward(spread(x, pad, 1), spread(dy, pad, 1.0), x_scales=scales, want_y=True)
        err = M.SWIGLU_BWD_REL * mag
        assert_near(host(dx.float()), want, err + U16 * (np.abs(want) + err) + TINY16, f"dx, pad {pad}")
        err = M.SWIGLU_BWD_REL * np.abs(y64)
        assert_near(host(y.float()), y64, err + U16 * (np.abs(y64) + err) + TINY16, f"y, pad {pad}")
    if inter % 128 == 0:
        bits = host_bf16_bits(dx)
        for mode in ("free", "pow2"):
            got = fp8q.swiglu_backward(x, dy, x_scales=scales, bf16=mode == "free", quantize=True, scale_mode=mode)
            oc, os_ = Q.quantize_rows(bits, Q.FREE if mode == "free" else Q.POW2)
            assert_codes_equal(host_codes(got[2]), oc, mode)
            assert_scales_equal(host(got[3]), os_, mode)
            assert got[1] is None and (got[0] is None or torch.equal(got[0], dx))
    only = fp8q.swiglu_backward(x, dy, x_scales=scales, bf16=False, want_y=True)
    assert only[0] is None and torch.equal(only[1], y)


def test_swiglu_backward_far_gates():
    """Gates from where the exponential is subnormal to where it vanishes."""
    g = np.concatenate([-np.arange(60, 130, 0.5), np.arange(60, 130, 0.5), [0.0, -0.0, 1e-30, -1e-30, 3e38, -3e38]])
    gb = e4m3.f32_to_bf16_bits_rne(g.astype(np.float32))
    one = np.full_like(gb, e4m3.f32_to_bf16_bits_rne(np.ones(1, np.float32))[0])
    xb = np.stack([gb, one], 1)
    dx, y, _, _ = fp8q.swiglu_backward(dev_bf16(xb), dev_bf16(one[:, None]), want_y=True)
    want, y64, mag = M.swiglu_backward(f64(xb), f64(one[:, None]))
    # below 2^-126 float32 steps and the reciprocal's flush of subnormals count absolutely: times the gate, at most 2^7
    near = np.abs(g) < 1e30
    assert_near(host(dx.float())[near], want[near], (M.SWIGLU_BWD_REL + U16) * np.maximum(mag, np.abs(want))[near] + 2.0 ** -119, "dx")
    assert_near(host(y.float())[near], y64[near], 1.01 * U16 * np.abs(y64)[near] + 2.0 ** -119, "y")
    far = host(dx.float())[~near]
    assert far[0].tolist() == [1.0, pytest.approx(3e38, rel=2.0 ** -7)] and far[1][0] == 0 and far[1][1] == 0


def test_swiglu_backward_against_differences():
    """The kernel's gradient (BF16) against central differences of SwiGLU in 64 bits."""
    r = np.random.default_rng(12)
    xb, dyb = bf16(r, (4, 256), 2.0), bf16(r, (4, 128))
    dx = host(fp8q.swiglu_backward(dev_bf16(xb), dev_bf16(dyb))[0].float()).astype(np.float64)
    x, dy, h = f64(xb), f64(dyb), 1e-5
    f = lambda g, u: g / (1 + np.exp(-g)) * u  # noqa: E731
    g, u = x[:, :128], x[:, 128:]
    diff = np.concatenate([dy * (f(g + h, u) - f(g - h, u)) / (2 * h), dy * f(g, 1.0)], 1)
    _, _, mag = M.swiglu_backward(x, dy)
    # second-order term: h^2/6 times a third derivative below 1 in magnitude, and cancellation of 2^-53 / h
    assert_near(dx, diff, U16 * np.abs(diff) + M.SWIGLU_BWD_REL * mag + 1e-9 * (np.abs(dy * u).repeat(1, 0) @ np.ones((128, 256)) + 1), "dx")


def test_swiglu_backward_empty():
    for rows, inter in ((0, 128), (5, 0), (0, 0)):
        x = torch.zeros((rows, 2 * inter), dtype=torch.bfloat16, device="cuda:0")
        dy = torch.zeros((rows, inter), dtype=torch.bfloat16, device="cuda:0")
        scales = torch.zeros((rows, 2 * inter // 128), device="cuda:0")
        for xx, ss in ((x, None), (x.to(torch.uint8), scales)):
            dx, y, codes, dxs = fp8q.swiglu_backward(xx, dy, x_scales=ss, quantize=True, want_y=True)
            assert dx.shape == codes.shape == (rows, 2 * inter) and y.shape == (rows, inter) and dxs.shape == scales.shape


@pytest.mark.parametrize("pads", [(8, 8, 16), (3, 1, 5), (0, 8, 1)])
def test_outputs_of_any_row_stride_leave_the_gaps_alone(pads):
    """Rows further apart than their length, on and off 16-byte boundaries, for every output of the two gradients."""
    lib, stream = fp8q.load_library(), torch.cuda.current_stream().cuda_stream
    r = np.random.default_rng(sum(pads))

    def buffer(rows, cols, pad, dtype):
        return torch.full((rows, cols + pad), 9, dtype=dtype, device="cuda:0")

    def check(buf, want, what):
        n = want.shape[1]
        assert torch.equal(buf[:, :n], want) and (buf[:, n:] == 9).all(), what

    for n, inter in ((1030, 256), (640, 128)):
        dout, y = dev_bf16(bf16(r, (40, n))), dev_bf16(bf16(r, (50, n)))
        row_of = r.permutation(50)[:40].reshape(40, 1).astype(np.int32)
        row_of[::9] = -1
        token = np.full(50, -1, dtype=np.int32)
        token[row_of[row_of >= 0]] = np.nonzero(row_of >= 0)[0]
        rows, tok, w = dev(row_of), dev(token), torch.rand((40, 1), device="cuda:0")
        dy, codes, scales, dw = fp8q.moe_combine_backward(dout, y, rows, w, tok, quantize=True)
        b_dy, b_codes = buffer(50, n, pads[0], torch.bfloat16), buffer(50, n, pads[1], torch.uint8)
        b_s, b_dw = torch.full_like(scales, 9.0), torch.full_like(dw, 9.0)
        assert lib.fp8q_moe_combine_backward(dout.data_ptr(), 1, 40, n, n, y.data_ptr(), 1, 50, n, rows.data_ptr(), w.data_ptr(), 1, tok.data_ptr(),
                                             b_dy.data_ptr(), n + pads[0], 0, b_codes.data_ptr(), n + pads[1], b_s.data_ptr(), b_dw.data_ptr(),
                                             stream) == fp8q.OK
        check(b_dy, dy, "dy")
        check(b_codes, codes, "codes")
        assert torch.equal(b_s, scales) and torch.equal(b_dw, dw)
        x, g = dev_bf16(bf16(r, (30, 2 * inter))), dev_bf16(bf16(r, (30, inter)))
        dx, out, codes, scales = fp8q.swiglu_backward(x, g, quantize=True, want_y=True)
        b_dx, b_codes = buffer(30, 2 * inter, pads[0], torch.bfloat16), buffer(30, 2 * inter, pads[1], torch.uint8)
        b_y, b_s = buffer(30, inter, pads[2], torch.bfloat16), torch.full_like(scales, 9.0)
        assert lib.fp8q_swiglu_backward(x.data_ptr(), None, 30, inter, 2 * inter, g.data_ptr(), inter, b_dx.data_ptr(), 2 * inter + pads[0],
                                        fp8q.SCALE_POW2, b_codes.data_ptr(), 2 * inter + pads[1], b_s.data_ptr(), b_y.data_ptr(),
                                        inter + pads[2], stream) == fp8q.OK
        check(b_dx, dx, "dx")
        check(b_codes, codes, "dx codes")
        check(b_y, out, "y")
        assert torch.equal(b_s, scales)


# --------------------------------------------------------- grouped wgrad ----

def token_operand(r, width, cap, real, mode, std=1.0):
    x = bf16(r, (cap, width), std)
    x[~real] = 0
    return Q.quantize_token_t(x, Q.FREE if mode == "free" else Q.POW2)


@pytest.mark.parametrize("acc,mode", [("fp32", "free"), ("fp32", "pow2"), ("fp32_pow2", "pow2"), ("fp8_mfma", "free"), ("fp8_mfma_scaled", "pow2")])
@pytest.mark.parametrize("nout,kin,sizes", [(1, 1, [5]), (40, 72, [0, 130, 0, 1]), (256, 256, [128, 256, 384]), (300, 260, [700, 0, 65]),
                                            (257, 225, [0, 0]), (512, 448, [1, 128, 129, 1000]), (3, 600, [640] * 9),
                                            (2000, 4100, [700, 400]),  # (on 128 x 128 tiles, the smaller ones before on 64 x 64)
                                            (2000, 8200, [900, 700]), (4000, 4100, [600])])  # (enough 256 x 256 tiles, and tokens, for the large shape)
def test_grouped_wgrad(acc, mode, nout, kin, sizes):
    r = np.random.default_rng(nout)
    padded = [-(-s // 128) * 128 for s in sizes]
    offsets = np.concatenate([[0], np.cumsum(padded)]).astype(np.int32)
    cap = int(offsets[-1]) + 128
    real = np.zeros(cap, bool)
    for s, o in zip(sizes, offsets):
        real[o:o + s] = True
    real[offsets[-1]:] = True  # rows behind the last group hold anything
    dy_c, dy_s = token_operand(r, nout, cap, real, mode)
    x_c, x_s = token_operand(r, kin, cap, real, mode)
    d = [dev(v) for v in (dy_c, dy_s, x_c, x_s, offsets)]
    got = fp8q.grouped_wgrad(*d, acc=acc)
    # bit for bit the plain weight gradient of each group by itself (the same products in the same order)
    for g, (a, b) in enumerate(zip(offsets[:-1], offsets[1:])):
        alone = fp8q.wgrad(d[0][:, a:b].contiguous(), d[1][:, a // 128:b // 128].contiguous(), d[2][:, a:b].contiguous(),
                           d[3][:, a // 128:b // 128].contiguous(), acc=acc) if b > a else torch.zeros((nout, kin), device="cuda:0")
        assert torch.equal(got[g], alone), f"group {g}"
    if acc.startswith("fp32"):
        want, mag = M.grouped_wgrad(dy_c, dy_s, x_c, x_s, offsets, e4m3.decode)
        assert_near(host(got), want, 1e-5 * mag + 1e-6, acc)
    out = torch.full((len(sizes), nout, kin + 4), 5.0, device="cuda:0")
    fp8q.grouped_wgrad(*d, out=out[:, :, :kin], acc=acc)
    assert torch.equal(out[:, :, :kin], got) and (out[:, :, kin:] == 5).all()
    odd = torch.full((len(sizes), nout, kin + 3), 5.0, device="cuda:0")
    fp8q.grouped_wgrad(*d, out=odd[:, :, :kin], acc=acc)
    assert torch.equal(odd[:, :, :kin], got) and (odd[:, :, kin:] == 5).all()


# (kin 8208: enough 256 x 256 tiles for the forms that the matrix core accumulates; 4112: 128 x 128; the others 64 x 64)
@pytest.mark.parametrize("acc,mode", [("fp32", "free"), ("fp32_pow2", "pow2"), ("fp8_mfma", "free"), ("fp8_mfma_scaled", "pow2")])
@pytest.mark.parametrize("nout,kin,sizes", [(40, 80, [130, 0, 1]), (300, 272, [700, 65]), (129, 16, [128]), (2000, 4112, [700, 400]), (2000, 8208, [900, 700])])
def test_grouped_wgrad_of_partial_tiles_on_line_boundaries(acc, mode, nout, kin, sizes):
    """Row strides of whole 64-byte lines (streaming stores) with tiles that end inside a row and a column: nothing is
    written past the columns, nor past the last row."""
    r = np.random.default_rng(kin)
    padded = [-(-s // 128) * 128 for s in sizes]
    offsets = np.concatenate([[0], np.cumsum(padded)]).astype(np.int32)
    real = np.zeros(int(offsets[-1]), bool)
    for s, o in zip(sizes, offsets):
        real[o:o + s] = True
    d = [dev(v) for v in (*token_operand(r, nout, real.size, real, mode), *token_operand(r, kin, real.size, real, mode), offsets)]
    for ld in (kin, kin + 16):
        buf = torch.full((len(sizes) * nout + 64, ld), 5.0, device="cuda:0")
        out = buf[:len(sizes) * nout].view(len(sizes), nout, ld)[:, :, :kin]
        fp8q.grouped_wgrad(*d, out=out, acc=acc)
        for g, (a, b) in enumerate(zip(offsets[:-1], offsets[1:])):
            alone = fp8q.wgrad(d[0][:, a:b].contiguous(), d[1][:, a // 128:b // 128].contiguous(), d[2][:, a:b].contiguous(),
                               d[3][:, a // 128:b // 128].contiguous(), acc=acc) if b > a else torch.zeros((nout, kin), device="cuda:0")
            assert torch.equal(out[g], alone), f"group {g}, stride {ld}"
        assert (buf[:len(sizes) * nout, kin:] == 5).all() and (buf[len(sizes) * nout:] == 5).all()


def test_grouped_wgrad_broken_tables_stay_inside():
    """Offsets outside the rows, decreasing or off the tiles are clamped and rounded down (a precondition the
    kernel does not report); the answers are those of the clamped table."""
    r = np.random.default_rng(9)
    cap = 512
    dy_c, dy_s = token_operand(r, 40, cap, np.ones(cap, bool), "free")
    x_c, x_s = token_operand(r, 24, cap, np.ones(cap, bool), "free")
    d = [dev(v) for v in (dy_c, dy_s, x_c, x_s)]
    broken = np.array([-5, 200, 100, 2 ** 31 - 1, 300, 600], dtype=np.int32)
    used = [(0, 128), (128, 0), (0, 512), (512, 256), (256, 512)]
    got = fp8q.grouped_wgrad(*d, dev(broken))
    for g, (a, b) in enumerate(used):
        want = fp8q.grouped_wgrad(*d, dev(np.array([a, max(a, b)], dtype=np.int32)))[0]
        assert torch.equal(got[g], want), g


def test_grouped_wgrad_empty():
    c, s = torch.zeros((8, 0), dtype=torch.uint8, device="cuda:0"), torch.zeros((8, 0), device="cuda:0")
    off = torch.zeros(4, dtype=torch.int32, device="cuda:0")
    assert not host(fp8q.grouped_wgrad(c, s, c, s, off)).any()
    assert fp8q.grouped_wgrad(c, s, c, s, off[:1]).shape == (0, 8, 8)


def test_grouped_wgrad_without_outputs():
    c, s = torch.zeros((8, 256), dtype=torch.uint8, device="cuda:0"), torch.zeros((8, 2), device="cuda:0")
    off = torch.tensor([0, 128, 256], dtype=torch.int32, device="cuda:0")
    assert fp8q.grouped_wgrad(c[:0], s[:0], c, s, off).shape == (2, 0, 8)
    assert fp8q.grouped_wgrad(c, s, c[:0], s[:0], off).shape == (2, 8, 0)


@pytest.mark.parametrize("n", [1, 5, 128, 300])
def test_single_columns_of_any_column_stride(n):
    """A tensor of one column has no column stride to speak of: every call with row-major operands takes it, and answers as
    for the contiguous one."""
    r = np.random.default_rng(n)
    col = dev_bf16(bf16(r, (n, 1)))
    odd = dev_bf16(bf16(r, (n, 3)))
    odd[:, :1] = col
    views = [col.t().contiguous().t(), torch.as_strided(col, (n, 1), (1, 77)), torch.as_strided(odd, (n, 1), (3, 2))]
    assert all(v.shape == (n, 1) and torch.equal(v, col) for v in views) and views[1].stride(1) == 77

    def same(call):
        want = call(col)
        for v in views:
            got = call(v)
            assert all(torch.equal(a, b) for a, b in zip(got, want))

    same(lambda v: fp8q.quantize_act(v))
    same(lambda v: fp8q.quantize_act(v, "token_t", "pow2"))
    same(lambda v: fp8q.quantize_weight(v))
    same(lambda v: fp8q.quantize_weight_t(v))
    same(lambda v: fp8q.quantize_linear(v, v))
    index = torch.arange(n, dtype=torch.int32, device="cuda:0").flip(0).contiguous()
    codes, scales = fp8q.quantize_act(col)
    want = fp8q.gather_rows(codes.contiguous(), scales, index)
    for v in (codes, torch.as_strided(codes.contiguous(), (n, 1), (1, 9))):
        assert all(torch.equal(a, b) for a, b in zip(fp8q.gather_rows(v, scales, index), want))
    rows = index[:, None].contiguous()
    same(lambda v: (fp8q.moe_combine(v, rows),))
    same(lambda v: fp8q.moe_combine_backward(v, v, rows)[::3])
    both = torch.cat([col, col], 1)
    same(lambda v: fp8q.swiglu_backward(both, v)[:1])


def test_refusals_of_the_binding():
    y = torch.zeros((8, 16), dtype=torch.bfloat16, device="cuda:0")
    rows = torch.zeros((4, 2), dtype=torch.int32, device="cuda:0")
    w = torch.zeros((4, 2), device="cuda:0")
    for bad in (lambda: fp8q.moe_combine(y.half(), rows), lambda: fp8q.moe_combine(y, rows.long()),
                lambda: fp8q.moe_combine(y, rows, w.double()), lambda: fp8q.moe_combine(y, rows, out=y.float()[:4], out_dtype=torch.bfloat16)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: fp8q.moe_combine(y, rows, w[:3]), lambda: fp8q.moe_combine(y, rows.t()), lambda: fp8q.moe_combine(y.t(), rows),
                lambda: fp8q.moe_combine(y, rows, out=y), lambda: fp8q.moe_combine_backward(y, y, rows),
                lambda: fp8q.moe_combine_backward(y[:4], y, rows, None, rows[:, 0].contiguous()),
                lambda: fp8q.swiglu_backward(y, y), lambda: fp8q.swiglu_backward(y, y[:, :8], quantize=True),
                lambda: fp8q.swiglu_backward(y, y[:, :8], bf16=False), lambda: fp8q.moe_sort(rows, -1), lambda: fp8q.moe_sort(rows, 4, align=0),
                lambda: fp8q.moe_sort(rows, 4, align=(1 << 32) + 1, rows_cap=0), lambda: fp8q.moe_sort(rows, (1 << 32) + 1, rows_cap=8)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(fp8q.Fp8qError):  # rows over one another
        fp8q.moe_combine(y[:1].expand(8, 16), rows)
    with pytest.raises(fp8q.Fp8qError):  # a base that is not 16-byte aligned
        fp8q.moe_combine(y[:, 1:], rows)


# ------------------------------------------------- streams, graphs, a layer ----

def layer_inputs(seed, tokens=300, topk=4, experts=12, hidden=256, inter=128):
    r = np.random.default_rng(seed)
    return (dev_bf16(bf16(r, (tokens, hidden))), dev(routing(r, tokens, topk, experts)), dev(r.random((tokens, topk)).astype(np.float32)),
            dev_bf16(bf16(r, (experts, 2 * inter, hidden), 0.1)), dev_bf16(bf16(r, (experts, hidden, inter), 0.1)),
            dev_bf16(bf16(r, (tokens, hidden))))


def expert_layer(x, experts, weights, w_up, w_down, dout, first, hosted, cap):
    """Forward and backward of the hosted experts, all through the library's entry points but the BF16 row gather."""
    n = lambda w: w[first:first + hosted].reshape(-1, w.shape[2])  # noqa: E731
    up_c, up_s = fp8q.quantize_weight(n(w_up))
    dn_c, dn_s = fp8q.quantize_weight(n(w_down))
    offsets, token, row_of = fp8q.moe_sort(experts, hosted, first=first, align=128, rows_cap=cap)
    group = lambda c, s, like: (c.contiguous().view(hosted, like.shape[1], -1), s.view(hosted, -1, s.shape[1]))  # noqa: E731
    a_c, a_s = fp8q.gather_rows(*fp8q.quantize_act(x), token)
    h = fp8q.grouped_gemm(a_c.contiguous(), a_s, offsets, *group(up_c, up_s, w_up), out=x.new_zeros((cap, w_up.shape[1])))
    z_c, z_s, c_c, c_s = fp8q.swiglu_quantize(h, cache=True)
    y = fp8q.grouped_gemm(z_c.contiguous(), z_s, offsets, *group(dn_c, dn_s, w_down), out=x.new_zeros((cap, w_down.shape[1])))
    out = fp8q.moe_combine(y, row_of, weights)
    # backward
    dy, dy_c, dy_s, dweights = fp8q.moe_combine_backward(dout, y, row_of, weights, token, quantize=True, scale_mode="pow2")

    def transposed(w):
        parts = [fp8q.quantize_weight_t(w[first + e], both=False)[2:] for e in range(hosted)]
        return torch.stack([c.contiguous() for c, _ in parts]), torch.stack([s for _, s in parts])

    dz = fp8q.grouped_gemm(dy_c.contiguous(), dy_s, offsets, *transposed(w_down), out=x.new_zeros((cap, w_down.shape[2])))
    dh, z, dh_c, dh_s = fp8q.swiglu_backward(c_c, dz, x_scales=c_s, quantize=True, want_y=True)
    dxr = fp8q.grouped_gemm(dh_c.contiguous(), dh_s, offsets, *transposed(w_up), out=x.new_zeros((cap, w_up.shape[2])))
    dx = fp8q.moe_combine(dxr, row_of, out_dtype=torch.float32)
    t = lambda v: tuple(p.contiguous() for p in fp8q.quantize_act(v, "token_t"))  # noqa: E731
    xr = torch.where((token >= 0)[:, None], x[token.clamp(min=0).long()], x.new_zeros(()))
    dw_down = fp8q.grouped_wgrad(*t(dy), *t(z), offsets)
    dw_up = fp8q.grouped_wgrad(*t(dh), *t(xr), offsets)
    return out, dx, dweights, dw_up, dw_down


def test_whole_expert_layer_against_float64_autograd():
    """Every output within what E4M3 tiles allow: codes are off by at most half a step (2^-4 relative to their
    value), so a product of two by 2^-3 of the magnitudes summed; in the 2-norm over random signs a few percent.
    The float64 layer is differentiated by torch on the CPU."""
    x, experts, weights, w_up, w_down, dout = layer_inputs(0)
    first, hosted = 2, 8
    cap = 300 * 4 + hosted * 128
    cap = -(-cap // 128) * 128
    got = expert_layer(x, experts, weights, w_up, w_down, dout, first, hosted, cap)
    leaves = [v.double().cpu().requires_grad_() for v in (x, weights, w_up, w_down)]
    xd, wd, ud, dd = leaves
    e = experts.cpu()
    out = torch.zeros_like(xd)
    for i in range(first, first + hosted):
        t, j = torch.nonzero(e == i, as_tuple=True)
        h = xd[t] @ ud[i].T
        g, u = h.chunk(2, 1)
        out = out.index_add(0, t, wd[t, j, None] * ((g * torch.sigmoid(g) * u) @ dd[i].T))
    (out * dout.double().cpu()).sum().backward()
    want = (out.detach(), xd.grad, wd.grad, ud.grad[first:first + hosted], dd.grad[first:first + hosted])
    for name, a, b in zip(("out", "dx", "dweights", "dw_up", "dw_down"), got, want):
        rel = float((a.double().cpu() - b).norm() / b.norm())
        say(f"{name}: {rel:.4f}")
        assert rel < 0.125, name


def test_layer_captured_and_replayed():
    """One graph of the whole layer, replayed on changing inputs with eager work between, equals the eager layer."""
    first, hosted, cap = 0, 6, 300 * 4 + 6 * 128 + (-(300 * 4 + 6 * 128)) % 128
    static = list(layer_inputs(1))
    expert_layer(*static, first, hosted, cap)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        expert_layer(*static, first, hosted, cap)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = expert_layer(*static, first, hosted, cap)
    for seed in (1, 2, 3, 2):
        new = layer_inputs(seed)
        want = expert_layer(*new, first, hosted, cap)
        for s, v in zip(static, new):
            s.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(out, want)):
            assert torch.equal(a, b), (seed, i)


# ---------------------------------------------------------- large offsets ----

def test_rows_past_four_gigabytes():
    """Row offsets that pass 2^31 elements and 2^32 bytes, through the sum, its gradient and SwiGLU's: rows near the
    end against a small call on copies of the same rows, bit for bit."""
    cap, n, tokens = 310_000, 7168, 64
    g = torch.Generator(device="cuda:0").manual_seed(5)
    y = torch.empty((cap, n), dtype=torch.bfloat16, device="cuda:0")
    used = torch.cat([torch.arange(cap - 96, cap), torch.arange(32)]).to("cuda:0")
    some = torch.randn((used.numel(), n), generator=g, device="cuda:0").bfloat16()
    y[used] = some
    small = torch.randperm(used.numel(), generator=g, device="cuda:0").view(tokens, 2).int()
    rows = used[small.long()].int()
    w = torch.rand((tokens, 2), generator=g, device="cuda:0")
    dout = torch.randn((tokens, n), generator=g, device="cuda:0").bfloat16()
    for odt in (torch.bfloat16, torch.float32):
        assert torch.equal(fp8q.moe_combine(y, rows, w, out_dtype=odt), fp8q.moe_combine(some, small, w, out_dtype=odt))
    a = fp8q.moe_combine_backward(dout, y, rows, w, quantize=True)
    b = fp8q.moe_combine_backward(dout, some, small, w, quantize=True)
    assert torch.equal(a[0][used], b[0]) and torch.equal(a[1][used], b[1]) and torch.equal(a[2][used], b[2]) and torch.equal(a[3], b[3])
    del a
    # 310,000 rows of 3584 gates and 3584 ups
    dy = torch.empty((cap, n // 2), dtype=torch.bfloat16, device="cuda:0")
    dys = torch.randn((used.numel(), n // 2), generator=g, device="cuda:0").bfloat16()
    dy[used] = dys
    a, b = fp8q.swiglu_backward(y, dy, want_y=True), fp8q.swiglu_backward(some, dys, want_y=True)
    assert torch.equal(a[0][used], b[0]) and torch.equal(a[1][used], b[1])


def test_grouped_wgrad_past_four_gigabytes():
    """80 gradients of 4096 x 4096: the last ones' offsets pass 2^32 bytes."""
    r = np.random.default_rng(6)
    groups, n = 80, 4096
    offsets = np.minimum(np.arange(groups + 1) * 128, 256).astype(np.int32)
    offsets[-2:] = [256, 384]
    dy_c, dy_s = token_operand(r, n, 384, np.ones(384, bool), "free")
    d = [dev(v) for v in (dy_c, dy_s, dy_c, dy_s, offsets)]
    out = torch.full((groups, n, n), 3.0, device="cuda:0")
    fp8q.grouped_wgrad(*d, out=out)
    for g in (0, 1, groups - 1):
        a, b = int(offsets[g]), int(offsets[g + 1])
        c, s = d[0][:, a:b].contiguous(), d[1][:, a // 128:b // 128].contiguous()
        assert torch.equal(out[g], fp8q.wgrad(c, s, c, s)), g
    assert not out[2:-1].any()


def test_large_sorts_on_two_streams_and_in_two_graphs():
    """Each call has its own workspace: sorts of many pairs at the same time do not meet."""
    ins = [dev(routing(np.random.default_rng(s), 6000, 8, 64)) for s in range(4)]
    want = [fp8q.moe_sort(v, 64, align=128) for v in ins]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append(fp8q.moe_sort(ins[k], 64, align=128))
    torch.cuda.synchronize()
    for k in range(2):
        for g in got[k]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[k]))
    graphs, outs = [], []
    for k in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(fp8q.moe_sort(ins[2 + k], 64, align=128))
        graphs.append(g)
    for _ in range(5):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                graphs[k].replay()
        torch.cuda.synchronize()
        for k in range(2):
            assert all(torch.equal(a, b) for a, b in zip(outs[k], want[2 + k]))
