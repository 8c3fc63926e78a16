"""The router's choice of experts and its gradient on the GPU, against the
token-by-token oracle in 64 bits (oracle/block.py)."""

import numpy as np
import pytest
import torch

import fine_grained_fp8_fp8q_amd as fp8q
from oracle import block as B
from tests.gpu_util import dev, host, need_gpu, say

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
# a float64 value rounded to float32: half a step; the 64-bit steps before it are far below a tenth of that
NEAR32 = 1.1 * 2.0 ** -24
MANY = 16400  # tokens from which every choice of kernels is that of large batches


@pytest.fixture(autouse=True)
def _gpu(request):
    need_gpu()
    say(f"[route] {request.node.name}")


def logits_of(r, tokens, n, dtype, masked=False):
    x = (r.normal(size=(tokens, n)) * 1.5).astype(np.float32)
    if masked:
        x[r.random(x.shape) < 0.2] = -np.inf
        x[r.random(x.shape) < 0.02] = np.nan
        x[r.random(x.shape) < 0.02] = np.inf
        x[r.random(tokens) < 0.1] = -np.inf
    if dtype == BF:
        x = dev(x).to(BF).float().cpu().numpy()
    return x


def on(x, dtype, pad=0):
    buf = torch.full((x.shape[0], x.shape[1] + pad), 100.0, dtype=dtype, device="cuda:0")
    buf[:, :x.shape[1]] = dev(x)
    return buf[:, :x.shape[1]]


def check(x, dtype, topk, bias=None, pad=0, index_dtype=torch.int32, **kw):
    load = torch.full((x.shape[1],), 5, dtype=torch.int32, device="cuda:0")
    bd = None if bias is None else dev(bias)
    e, w, s = fp8q.moe_route(on(x, dtype, pad), topk, bias=bd, index_dtype=index_dtype, want_scores=True, load=load, **kw)
    we, ww, ws = B.route(x, topk, bias, **kw)
    assert e.dtype == index_dtype and e.shape == w.shape == (x.shape[0], topk)
    bad = np.argwhere(host(e) != we)
    assert bad.size == 0, f"{len(bad)} choices differ, first {bad[0]}: {host(e)[bad[0][0]]} for {we[bad[0][0]]}"
    assert (np.abs(host(w.double()) - ww) <= NEAR32 * ww + 2.0 ** -149).all()
    assert (np.abs(host(s.double()) - ws) <= NEAR32 * ws + 2.0 ** -149).all()
    assert np.array_equal(host(load) - 5, np.bincount(we[we >= 0], minlength=x.shape[1]))
    e, w, s = fp8q.moe_route(on(x, dtype, pad), topk, bias=bd, **kw)
    assert s is None and np.array_equal(host(e), we) and (np.abs(host(w.double()) - ww) <= NEAR32 * ww + 2.0 ** -149).all()
    # the same tokens over and over, by the kernels of many tokens (and a last wave that is not full)
    times = -(-MANY // x.shape[0])
    rows = torch.arange(times * x.shape[0] - 1, device="cuda:0") % x.shape[0]
    many = on(x, dtype, pad)[rows]
    bound = dev(NEAR32 * ww + 2.0 ** -149)[rows]
    for want_scores in (False, True):
        load.zero_()
        e, w, s = fp8q.moe_route(many, topk, bias=bd, load=load, want_scores=want_scores, **kw)
        assert torch.equal(e, dev(we)[rows].int()) and bool(((w.double() - dev(ww)[rows]).abs() <= bound).all())
        assert torch.equal(load, torch.bincount(e[e >= 0].long(), minlength=x.shape[1]).int())
        if want_scores:
            assert bool(((s.double() - dev(ws)[rows]).abs() <= NEAR32 * dev(ws)[rows] + 2.0 ** -149).all())


# experts, groups, open groups, topk
SHAPES = [(1, 1, 1, 1), (2, 2, 1, 1), (3, 1, 1, 3), (8, 1, 1, 2), (20, 5, 2, 8), (60, 1, 1, 4), (64, 8, 3, 6), (64, 64, 9, 8), (65, 1, 1, 64), (100, 1, 1, 17), (160, 8, 3, 6),
          (256, 8, 4, 8), (256, 1, 1, 8), (256, 16, 16, 16), (384, 1, 1, 8), (495, 33, 4, 40), (500, 5, 1, 10), (504, 9, 2, 8), (510, 17, 3, 16), (512, 1, 1, 1),
          (512, 64, 8, 64), (510, 3, 2, 8)]


@pytest.mark.parametrize("n,groups,top_groups,topk", SHAPES)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype,biased,renormalize", [(F32, True, True), (F32, False, False), (BF, False, True), (BF, True, False)])
def test_route(n, groups, top_groups, topk, score, dtype, biased, renormalize):
    r = np.random.default_rng(n * 7 + topk)
    for tokens, masked in ((1, False), (37, False), (66, True)):
        x = logits_of(r, tokens, n, dtype, masked)
        bias = (0.2 * r.normal(size=n)).astype(np.float32) if biased else None
        if biased and masked and n > 4:
            bias[r.integers(0, n, size=2)] = -np.inf
            bias[r.integers(0, n)] = np.nan
        # (sums of two scores without a bias: equal ones of BF16 logits are a matter of the last bit)
        for group_score in ("max", "top2") if biased or dtype == F32 else ("max",):
            check(x, dtype, topk, bias, pad=int(r.integers(0, 3)), score=score, groups=groups, top_groups=top_groups, group_score=group_score,
                  renormalize=renormalize, scale=2.5, index_dtype=torch.int64 if biased else torch.int32)


def test_route_ties_go_to_the_lower_index():
    for n, groups in ((64, 1), (256, 8), (100, 1), (17, 1)):
        x = np.zeros((5, n), dtype=np.float32)
        x[1, n // 2:] = 1
        x[2, ::3] = 2
        x[3] = -np.arange(n) % 4
        x[4] = -np.inf
        x[4, -3:] = 1
        for score in ("sigmoid", "softmax"):
            for bias in (None, np.zeros(n, dtype=np.float32)):
                check(x, F32, 8, bias, score=score, groups=groups, top_groups=max(1, groups // 2), group_score="max")


def test_route_of_far_logits():
    """Logits over the whole range of float32: by the logits themselves without a bias, scores that underflow weigh 0."""
    r = np.random.default_rng(3)
    x = (r.normal(size=(40, 64)) * np.exp(20 * r.random((40, 64)))).astype(np.float32)
    x[0] = 3e38
    x[1] = -3e38
    x[2, :9] = [3e38, np.inf, np.inf, -np.inf, 0, -800, -1e-38, 1e-38, 88]
    for score in ("sigmoid", "softmax"):
        for renormalize in (True, False):
            check(x, F32, 8, score=score, renormalize=renormalize)
            check(x, F32, 8, (0.1 * r.normal(size=64)).astype(np.float32), score=score, renormalize=renormalize)


def test_route_near_ties():
    """Biased scores a few 2^-40 apart, far below a float32 step: the order of the 64-bit scores."""
    r = np.random.default_rng(4)
    n = 256
    base = np.float32(0.3) + np.arange(n, dtype=np.float32) * np.float32(2.0 ** -24)
    x = np.stack([base[r.permutation(n)] for _ in range(50)])
    check(x, F32, 8, np.zeros(n, dtype=np.float32), score="sigmoid")
    check(x, F32, 8, np.full(n, 64.0, dtype=np.float32), score="sigmoid")
    check(x, F32, 8, np.full(n, 0.5, dtype=np.float32), score="softmax", groups=8, top_groups=4)


def test_route_large_and_empty():
    r = np.random.default_rng(5)
    e, w, s = fp8q.moe_route(torch.zeros((0, 8), device="cuda:0"), 2, want_scores=True)
    assert e.shape == w.shape == (0, 2) and s.shape == (0, 8)
    e, w, s = fp8q.moe_route(torch.zeros((3, 8), device="cuda:0"), 0, want_scores=True)
    assert e.shape == (3, 0) and host(s).tolist() == [[0.5] * 8] * 3
    e, w, s = fp8q.moe_route(torch.zeros((3, 0), device="cuda:0"), 0)
    assert e.shape == (3, 0)
    # many tokens: rows of a batch as they are alone, and the number of pairs
    x = dev(r.normal(size=(70001, 256)).astype(np.float32))
    bias = dev((0.1 * r.normal(size=256)).astype(np.float32))
    load = torch.zeros(256, dtype=torch.int32, device="cuda:0")
    e, w, _ = fp8q.moe_route(x, 8, bias=bias, groups=8, top_groups=4, load=load)
    assert int(load.sum()) == 70001 * 8 and torch.equal(load, torch.bincount(e.reshape(-1), minlength=256).int())
    for t in (0, 1, 35000, 70000):
        e1, w1, _ = fp8q.moe_route(x[t:t + 1], 8, bias=bias, groups=8, top_groups=4)
        assert torch.equal(e1[0], e[t]) and torch.equal(w1[0], w[t])
    pick = slice(69990, 70001)
    we, ww, _ = B.route(host(x[pick]), 8, host(bias), groups=8, top_groups=4)
    assert np.array_equal(host(e[pick]), we)


@pytest.mark.parametrize("tokens,n,topk", [(1, 256, 8), (511, 256, 8), (512, 256, 8), (1025, 512, 4), (1024, 8, 8), (3001, 60, 3), (4100, 1, 1), (70, 512, 64)])
@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_route_counts_its_pairs(tokens, n, topk, index):
    r = np.random.default_rng(tokens)
    x = logits_of(r, tokens, n, F32, True)
    x[tokens // 2] = -np.inf  # padding, and what is added to
    start = r.integers(0, 1000, size=n).astype(np.int32)
    for bias in (None, np.where(np.arange(n) < 2, 9.0, 0.0).astype(np.float32)):
        load = dev(start)
        e, _, _ = fp8q.moe_route(dev(x), topk, bias=None if bias is None else dev(bias), index_dtype=index, load=load)
        e = host(e).reshape(-1)
        assert (e == -1).any() and np.array_equal(host(load), start + np.bincount(e[e >= 0], minlength=n))


# -------------------------------------------------------------- backward ----

@pytest.mark.parametrize("tokens,n,topk", [(1, 1, 1), (1, 256, 8), (5, 8, 8), (33, 60, 4), (70, 256, 8), (9, 160, 6), (3, 512, 64), (40, 65, 3), (6, 20, 0)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("dtype,odt", [(F32, F32), (BF, BF), (BF, F32), (F32, BF)])
def test_route_backward(tokens, n, topk, score, renormalize, dtype, odt):
    r = np.random.default_rng(n + topk)
    for masked in (False, True):
        x = logits_of(r, tokens, n, dtype, masked)
        if masked:
            x = np.where(np.isposinf(x), np.float32(30.0), x)
        e, _, _ = B.route(x, topk)
        if masked and topk > 2:  # experts that are none, one twice
            e[0, 0], e[-1, 1], e[-1, 2] = n, e[-1, 0], -7
        dw = r.normal(size=(tokens, topk)).astype(np.float32)
        dw[(e < 0) | (e >= n)] = np.nan
        for dscores in (None, r.normal(size=(tokens, n)).astype(np.float32)):
            want, mag = B.route_backward(dw, e, x, score, renormalize, 2.5, dscores)
            got = fp8q.moe_route_backward(dev(dw), dev(e).to(torch.int64 if renormalize else torch.int32), on(x, dtype, int(r.integers(0, 3))), score=score,
                                          renormalize=renormalize, scale=2.5, dscores=None if dscores is None else dev(dscores), out_dtype=odt)
            assert got.dtype == odt
            half = 2.0 ** -8 if odt == BF else 2.0 ** -24
            # 64-bit steps of the magnitudes that are added, a hundred or so of them, and the rounding of the result
            bound = half * 1.01 * np.abs(want) + 200 * 2.0 ** -53 * mag + 2.0 ** -134
            off = np.abs(host(got.double()) - want)
            assert (off <= bound).all(), (masked, float((off / bound).max()))
            assert (host(got.float())[~(x > -np.inf)] == 0).all()


@pytest.mark.parametrize("n,topk", [(256, 8), (60, 4), (128, 16), (100, 3), (512, 17), (130, 5)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_backward_of_many_tokens(n, topk, score, renormalize):
    """Batches in which several tokens share a wave: each token as it is alone."""
    r = np.random.default_rng(n)
    x = logits_of(r, 41, n, F32)
    e, _, _ = B.route(x, topk)
    e[0, 0], e[-1, 1], e[-1, 2] = n, e[-1, 0], -7
    dw = r.normal(size=(41, topk)).astype(np.float32)
    for dscores in (None, r.normal(size=(41, n)).astype(np.float32)):
        want, mag = B.route_backward(dw, e, x, score, renormalize, 2.5, dscores)
        # 64-bit steps of the magnitudes that are added, a hundred or so of them, and the rounding of the result
        bound = 2.0 ** -24 * 1.01 * np.abs(want) + 200 * 2.0 ** -53 * mag + 2.0 ** -134
        for tokens in (2050, MANY):
            rows = np.arange(tokens) % 41
            got = host(fp8q.moe_route_backward(dev(dw[rows]), dev(e[rows]), dev(x[rows]), score=score, renormalize=renormalize, scale=2.5,
                                               dscores=None if dscores is None else dev(dscores[rows])).double())
            assert (np.abs(got - want[rows]) <= bound[rows]).all(), (tokens, dscores is None)


def test_route_backward_gap_and_strides():
    """Output rows of any stride, through the C ABI; nothing behind them is written."""
    r = np.random.default_rng(6)
    for tokens, n, topk, pad in ((33, 60, 4, 3), (5, 256, 8, 8), (1, 7, 2, 1)):
        x, dw = logits_of(r, tokens, n, F32), r.normal(size=(tokens, topk)).astype(np.float32)
        e = B.route(x, topk)[0]
        out = torch.full((tokens, n + pad), 7.0, device="cuda:0")
        args = [dev(dw), dev(e), on(x, F32, pad)]
        st = fp8q.load_library().fp8q_moe_route_backward(args[0].data_ptr(), args[1].data_ptr(), 1, tokens, topk, args[2].data_ptr(), 0, n, n + pad, 1, 1, 2.5, None,
                                                         out.data_ptr(), 0, n + pad, torch.cuda.current_stream().cuda_stream)
        assert st == fp8q.OK
        assert torch.equal(out[:, :n], fp8q.moe_route_backward(args[0], args[1], args[2].contiguous(), scale=2.5)) and bool((out[:, n:] == 7).all())


def test_route_gradient_against_differences():
    """Weights of the kernel itself (float64 would not go through it) moved by central differences of the oracle's."""
    r = np.random.default_rng(7)
    x, dw = r.normal(size=(2, 12)).astype(np.float32), r.normal(size=(2, 3)).astype(np.float32)
    for score in ("sigmoid", "softmax"):
        for renormalize in (True, False):
            e, w, _ = fp8q.moe_route(dev(x), 3, score=score, renormalize=renormalize)
            got = host(fp8q.moe_route_backward(dev(dw), e, dev(x), score=score, renormalize=renormalize))
            picks = host(e)

            def loss(a):
                total = 0.0
                for t in range(2):
                    s = B.scores(a[t], score)[1][picks[t]]
                    total += float((dw[t] * (s / s.sum() if renormalize else s)).sum())
                return total

            for i in np.ndindex(x.shape):
                d = np.zeros(x.shape)
                d[i] = 1e-6
                assert abs((loss(x + d) - loss(x - d)) / 2e-6 - got[i]) < 1e-6


def test_route_refusals_of_the_binding():
    x = torch.zeros((4, 12), device="cuda:0")
    e, w = torch.zeros((4, 2), dtype=torch.int32, device="cuda:0"), torch.zeros((4, 2), device="cuda:0")
    for bad in (lambda: fp8q.moe_route(x.half(), 2), lambda: fp8q.moe_route(x, 2, bias=x[0].double()), lambda: fp8q.moe_route(x, 2, index_dtype=F32),
                lambda: fp8q.moe_route(x, 2, load=torch.zeros(12, device="cuda:0")), lambda: fp8q.moe_route_backward(w.double(), e, x),
                lambda: fp8q.moe_route_backward(w, e.float(), x), lambda: fp8q.moe_route_backward(w, e, x, out_dtype=torch.float16)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: fp8q.moe_route(x, 13), lambda: fp8q.moe_route(x, -1), lambda: fp8q.moe_route(x, 2, groups=2, top_groups=3), lambda: fp8q.moe_route(x, 2, score="relu"),
                lambda: fp8q.moe_route(x, 2, group_score="mean"), lambda: fp8q.moe_route(x, 2, bias=x[0, :4]), lambda: fp8q.moe_route(x.t(), 2),
                lambda: fp8q.moe_route(x, 2, groups=0, top_groups=0), lambda: fp8q.moe_route(x, 2, groups=1 << 32, top_groups=1),
                lambda: fp8q.moe_route_backward(w[:3], e, x), lambda: fp8q.moe_route_backward(w, e[:3], x), lambda: fp8q.moe_route_backward(w, e, x, dscores=x[:3]),
                lambda: fp8q.moe_route_backward(w, e.t().contiguous().t(), x), lambda: fp8q.moe_route(x.cpu(), 2)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: fp8q.moe_route(x, 2, groups=5), lambda: fp8q.moe_route(x, 5, groups=3), lambda: fp8q.moe_route(x, 2, scale=float("nan")),
                lambda: fp8q.moe_route(torch.zeros((2, 513), device="cuda:0"), 2), lambda: fp8q.moe_route(torch.zeros((2, 128), device="cuda:0"), 65),
                lambda: fp8q.moe_route(x[:1].expand(4, 12), 2), lambda: fp8q.moe_route(x, 2, groups=12, top_groups=1), lambda: fp8q.moe_route(x[:, 1:], 2)):
        with pytest.raises(fp8q.Fp8qError):
            bad()
