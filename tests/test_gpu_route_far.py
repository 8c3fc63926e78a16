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
