"""The router and its gradient on the GPU where scores are near the end of the
64-bit range (subnormal, or 0 beside ones that are not), against the oracle in
extended precision."""

import numpy as np
import pytest
import torch

import fine_grained_fp8_fp8q_amd as fp8q
from oracle import block as B
from tests.gpu_util import dev, host, need_gpu, say

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NEAR32 = 1.1 * 2.0 ** -24  # a float64 value rounded to float32, and 64-bit steps far below a tenth of that
TOKENS = (1, 40, 2050, 16400)  # every choice of kernels: one wave a token, several tokens a wave


@pytest.fixture(autouse=True)
def _gpu(request):
    need_gpu()
    say(f"[route far] {request.node.name}")


def far_logits(r, n):
    """40 rows: all logits around one far value, the end of the normal numbers, of the subnormal ones, beyond; whole rows
    and rows with near ones beside them."""
    x = np.zeros((40, n), dtype=np.float32)
    for t, base in enumerate((-640, -700, -705, -708.5, -709.9, -712, -720, -730, -740, -743)):
        for k in range(4):
            x[4 * t + k] = base + r.uniform(-1.5, 1.5, size=n)
            if k == 1:
                x[4 * t + k, ::3] = -800  # (0 in 64 bits, beside some that are not)
            if k == 2:
                x[4 * t + k, 1::5] = r.normal(size=len(x[0, 1::5]))
    x[37] = -800  # 0, all of them
    x[38] = -np.inf
    x[39, :] = -np.inf
    x[39, 3:6] = [-720, -719.5, -3e38]
    return x


@pytest.mark.parametrize("n,groups,top_groups,topk", [(8, 1, 1, 2), (60, 1, 1, 4), (64, 8, 3, 6), (256, 8, 4, 8), (384, 1, 1, 8), (256, 1, 1, 16), (100, 1, 1, 64)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("biased", [False, True])
def test_route_of_far_scores(n, groups, top_groups, topk, score, biased):
    r = np.random.default_rng(n + topk)
    x = far_logits(r, n)
    bias = None
    if biased:  # steps that decide, far above any of the scores that are far
        bias = (r.permutation(n) * 2.0 ** -8 + 2.0).astype(np.float32)
        if score == "softmax":  # near ones stay behind: the chosen ones' scores are all far
            x[:, ::7] = 0.0
            bias[::7] = -2.0
    for renormalize in (True, False):
        kw = dict(score=score, groups=groups, top_groups=top_groups, group_score="max", renormalize=renormalize, scale=2.5)
        want_e, want_w, _ = B.route(x, topk, bias, **kw)
        for tokens in TOKENS:
            rows = np.arange(tokens) % 40 if tokens > 1 else np.array([24])
            for scores in (False, True):
                e, w, _ = fp8q.moe_route(dev(x[rows]), topk, bias=None if bias is None else dev(bias), want_scores=scores, **kw)
                assert np.array_equal(host(e), want_e[rows]), (tokens, scores)
                assert (np.abs(host(w.double()) - want_w[rows]) <= NEAR32 * want_w[rows] + 2.0 ** -149).all(), (tokens, scores)


def test_route_orders_scores_below_the_normal_numbers():
    """Without a step of the bias between them, scores of logits between -745 and -709 choose in their order."""
    x = np.array([[-712, -720, -711, -740, -711.5, -730, -800, -900]], dtype=np.float32)
    for tokens in TOKENS:
        e, w, _ = fp8q.moe_route(dev(np.repeat(x, tokens, 0)), 4, bias=torch.zeros(8, device="cuda:0"))
        assert (host(e) == [2, 4, 0, 1]).all(), tokens
        want = np.exp(np.array([0, -0.5, -1, -9]))
        want /= want.sum()
        assert (np.abs(host(w.double()) - want) <= NEAR32 * want).all()


@pytest.mark.parametrize("n,topk", [(8, 2), (60, 4), (256, 8), (128, 16), (300, 17), (512, 64)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_backward_of_far_scores(n, topk, score, renormalize):
    r = np.random.default_rng(n + topk)
    x = far_logits(r, n)
    if score == "softmax":
        x[:38, ::7] = 0.0
    e = np.stack([r.permutation(n)[:topk] for _ in range(40)])
    if score == "softmax":  # the near ones are not chosen: every chosen score is far
        e = np.stack([r.permutation(np.setdiff1d(np.arange(n), np.arange(0, n, 7)))[:topk] for _ in range(40)])
    e[3, 1], e[36, 0], e[35, 1] = e[3, 0], -1, n
    dw = r.normal(size=(40, topk)).astype(np.float32)
    for dscores in (None, r.normal(size=(40, n)).astype(np.float32)):
        want, mag = B.route_backward(dw, e, x, score, renormalize, 2.5, dscores)
        assert np.isfinite(want).all() and (not renormalize or np.abs(want[20:24]).max() > 1e-3)
        # 64-bit steps of the magnitudes that are added, a hundred or so of them, and the rounding of the result
        bound = 2.0 ** -24 * 1.01 * np.abs(want) + 200 * 2.0 ** -53 * mag + 2.0 ** -134
        for tokens in TOKENS:
            rows = np.arange(tokens) % 40 if tokens > 1 else np.array([24])
            got = host(fp8q.moe_route_backward(dev(dw[rows]), dev(e[rows]), dev(x[rows]), score=score, renormalize=renormalize, scale=2.5,
                                               dscores=None if dscores is None else dev(dscores[rows])).double())
            assert (np.abs(got - want[rows]) <= bound[rows]).all(), (tokens, dscores is None)


def test_route_and_its_gradient_agree_on_far_scores():
    """Weights by the forward pass, moved by differences of the oracle's, against the gradient: two far logits."""
    x, dw = np.array([[-720.0, -720.5, -900.0]], dtype=np.float32), np.array([[1.0, -0.3]], dtype=np.float32)
    e, w, _ = fp8q.moe_route(dev(x), 2, scale=2.5)
    share = host(w.double())[0] / 2.5
    want = 2.5 * share[0] * share[1] * 1.3
    for dscores in (None, torch.zeros((1, 3), device="cuda:0")):
        got = host(fp8q.moe_route_backward(dev(dw), e, dev(x), scale=2.5, dscores=dscores).double())[0]
        assert np.allclose(got, [want, -want, 0], rtol=1e-6, atol=0) and abs(want - 0.764) < 1e-3
