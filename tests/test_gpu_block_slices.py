"""Micro-batches: per-row vectors sliced anywhere go through the binding, and
give the rows of the whole batch bit for bit; eager and captured."""

import numpy as np
import pytest
import torch

import fine_grained_fp8_fp8q_amd as fp8q
from tests.gpu_util import need_gpu, say

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
PARTS = [(0, 1), (1, 2), (3, 50), (6, 7), (50, 201), (201, 403)]


@pytest.fixture(autouse=True)
def _gpu(request):
    need_gpu()
    say(f"[slices] {request.node.name}")


def normal(seed, *shape):
    return torch.randn(shape, generator=torch.Generator(device="cuda:0").manual_seed(seed), device="cuda:0")


def test_norm_gradient_and_token_tiles_of_slices():
    h, dy, w = normal(1, 403, 512).to(BF), normal(2, 403, 512).to(BF), normal(3, 512)
    rstd = fp8q.rmsnorm_quantize(h, w, quantize=False)[3]
    whole = fp8q.rmsnorm_backward(dy, h, rstd, w, quantize=True, want_dweight=False)
    for lo, hi in PARTS:
        part = fp8q.rmsnorm_backward(dy[lo:hi], h[lo:hi], rstd[lo:hi], w, quantize=True)
        assert all(torch.equal(a, b[lo:hi]) for a, b in zip(part[:3], whole[:3])), (lo, hi)
        want = (dy[lo:hi].double() * (h[lo:hi].float() * rstd[lo:hi, None]).double()).sum(0)
        # a rounding a step of at most 202 rows, relative to the magnitudes summed
        mag = (dy[lo:hi].double() * h[lo:hi].double() * rstd[lo:hi, None].double()).abs().sum(0)
        assert bool(((part[3].double() - want).abs() <= 210 * 2.0 ** -24 * mag).all()), (lo, hi)
        tiles = fp8q.rmsnorm_quantize_t(h[lo:hi], rstd[lo:hi], w)
        copied = fp8q.rmsnorm_quantize_t(h[lo:hi].clone(), rstd[lo:hi].clone(), w)
        assert all(torch.equal(a, b) for a, b in zip(tiles, copied)), (lo, hi)
    index = torch.randint(-1, 403, (700,), generator=torch.Generator(device="cuda:0").manual_seed(4), device="cuda:0", dtype=torch.int32)
    for lo, hi in PARTS:
        got, want = fp8q.rmsnorm_quantize_t(h, rstd, w, index=index[lo:hi]), fp8q.rmsnorm_quantize_t(h, rstd, w, index=index[lo:hi].clone())
        assert all(torch.equal(a, b) for a, b in zip(got, want)), (lo, hi)


@pytest.mark.parametrize("topk", [1, 3, 6])
@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_route_gradient_of_slices(topk, index):
    logits, dweights, dscores = normal(5, 403, 64), normal(6, 403, topk), normal(7, 403, 64)
    experts, _, _ = fp8q.moe_route(logits, topk, index_dtype=index)
    for ds in (None, dscores):
        whole = fp8q.moe_route_backward(dweights, experts, logits, dscores=ds)
        for lo, hi in PARTS:
            part = fp8q.moe_route_backward(dweights[lo:hi], experts[lo:hi], logits[lo:hi], dscores=None if ds is None else ds[lo:hi])
            assert torch.equal(part, whole[lo:hi]), (lo, hi)


def test_slices_captured():
    """The copy is part of the graph: a replay reads what the batch's vector holds then."""
    h, dy, w = normal(8, 40, 256).to(BF), normal(9, 40, 256).to(BF), torch.ones(256, device="cuda:0")
    rstd = fp8q.rmsnorm_quantize(h, w, quantize=False)[3].clone()
    call = lambda: fp8q.rmsnorm_backward(dy[5:11], h[5:11], rstd[5:11], w, want_dweight=False)[0]  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for k in range(4):
        rstd.copy_(normal(20 + k, 40).abs() + np.float32(0.1))
        want = call()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
