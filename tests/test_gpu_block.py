"""A block's expert half from its residual stream to its residual stream and
back on the GPU, all through the library's entry points: residual and norm,
router, expert layer, and every gradient, against float64 autograd; eager,
captured and replayed, on two streams and from two graphs."""

import numpy as np
import pytest
import torch

import fine_grained_fp8_fp8q_amd as fp8q
from tests.gpu_util import dev, need_gpu, say

pytestmark = pytest.mark.gpu
EPS = 1e-6
TOKENS, HIDDEN, INTER, EXPERTS, GROUPS, OPEN, TOPK, SCALE = 300, 256, 128, 16, 4, 2, 3, 2.5
CAP = -(-(TOKENS * TOPK + EXPERTS * 127) // 128) * 128


@pytest.fixture(autouse=True)
def _gpu(request):
    need_gpu()
    say(f"[block] {request.node.name}")


def inputs(seed):
    r = np.random.default_rng(seed)
    b = lambda *s, std=1.0: dev((std * r.normal(size=s)).astype(np.float32)).to(torch.bfloat16)  # noqa: E731
    return [b(TOKENS, HIDDEN), b(TOKENS, HIDDEN), (b(HIDDEN, std=0.2) + 1).to(torch.bfloat16), b(EXPERTS, HIDDEN, std=0.1),
            dev((0.05 * r.normal(size=EXPERTS)).astype(np.float32)), b(EXPERTS, 2 * INTER, HIDDEN, std=0.1), b(EXPERTS, HIDDEN, INTER, std=0.1),
            b(TOKENS, HIDDEN), b(TOKENS, HIDDEN)]


def block(x, residual, gain, w_router, bias, w_up, w_down, dout, dh_next):
    """out = experts(norm(h)), h = x + residual; the gradients of <out, dout> + <h, dh_next>."""
    flat = lambda w: w.reshape(-1, w.shape[2])  # noqa: E731
    group = lambda c, s, like: (c.contiguous().view(EXPERTS, like.shape[1], -1), s.view(EXPERTS, -1, s.shape[1]))  # noqa: E731
    tok = lambda v: tuple(p.contiguous() for p in v)  # noqa: E731

    def transposed(w):
        parts = [fp8q.quantize_weight_t(w[e], both=False)[2:] for e in range(EXPERTS)]
        return torch.stack([c.contiguous() for c, _ in parts]), torch.stack([s for _, s in parts])

    _, a_c, a_s, rstd, h = fp8q.rmsnorm_quantize(x, gain, residual=residual, eps=EPS)
    r_c, r_s, rt_c, rt_s = fp8q.quantize_weight_t(w_router)
    logits = fp8q.gemm(a_c.contiguous(), a_s, r_c.contiguous(), r_s, out_dtype=torch.float32)
    experts, weights, _ = fp8q.moe_route(logits, TOPK, bias=bias, groups=GROUPS, top_groups=OPEN, scale=SCALE)
    offsets, token, row_of = fp8q.moe_sort(experts, EXPERTS, align=128, rows_cap=CAP)
    g_c, g_s = fp8q.gather_rows(a_c, a_s, token)
    up = fp8q.grouped_gemm(g_c.contiguous(), g_s, offsets, *group(*fp8q.quantize_weight(flat(w_up)), w_up), out=x.new_zeros((CAP, 2 * INTER)))
    z_c, z_s, c_c, c_s = fp8q.swiglu_quantize(up, cache=True)
    y = fp8q.grouped_gemm(z_c.contiguous(), z_s, offsets, *group(*fp8q.quantize_weight(flat(w_down)), w_down), out=x.new_zeros((CAP, HIDDEN)))
    out = fp8q.moe_combine(y, row_of, weights)
    # backward
    dy, dy_c, dy_s, dweights = fp8q.moe_combine_backward(dout, y, row_of, weights, token, quantize=True)
    dz = fp8q.grouped_gemm(dy_c.contiguous(), dy_s, offsets, *transposed(w_down), out=x.new_zeros((CAP, INTER)))
    dup, z, dup_c, dup_s = fp8q.swiglu_backward(c_c, dz, x_scales=c_s, quantize=True, want_y=True)
    dxr = fp8q.grouped_gemm(dup_c.contiguous(), dup_s, offsets, *transposed(w_up), out=x.new_zeros((CAP, HIDDEN)))
    dn = fp8q.moe_combine(dxr, row_of, out_dtype=torch.float32)
    dw_down = fp8q.grouped_wgrad(*tok(fp8q.quantize_act(dy, "token_t")), *tok(fp8q.quantize_act(z, "token_t")), offsets)
    dw_up = fp8q.grouped_wgrad(*tok(fp8q.quantize_act(dup, "token_t")), *tok(fp8q.rmsnorm_quantize_t(h, rstd, gain, index=token)), offsets)
    # the router's part: its gradient reaches the norm through W_router and the chosen weights (16 logits padded to a tile of 128)
    dlogits = fp8q.moe_route_backward(dweights, experts, logits, scale=SCALE, out_dtype=torch.bfloat16)
    wide = x.new_zeros((TOKENS, 128))
    wide[:, :EXPERTS] = dlogits
    dl_c, dl_s = fp8q.quantize_act(wide)
    rt = torch.zeros((HIDDEN, 128), dtype=torch.uint8, device=x.device)
    rt[:, :EXPERTS] = rt_c
    dn = dn + fp8q.dgrad(dl_c.contiguous(), dl_s, rt, rt_s, out_dtype=torch.float32)
    pad = -TOKENS % 128
    dl_t = torch.nn.functional.pad(dlogits, (0, 0, 0, pad))
    index = torch.cat([torch.arange(TOKENS, device=x.device, dtype=torch.int32), torch.full((pad,), -1, device=x.device, dtype=torch.int32)])
    dw_router = fp8q.wgrad(*tok(fp8q.quantize_act(dl_t, "token_t")), *tok(fp8q.rmsnorm_quantize_t(h, rstd, gain, index=index)))
    dx, _, _, dgain = fp8q.rmsnorm_backward(dn, h, rstd, gain, dres=dh_next)
    return out, h, dx, dgain, dw_router, dw_up, dw_down, experts


def reference(leaves, experts, dout, dh_next):
    """The same block in float64 on the CPU with the experts given, differentiated by torch."""
    x, residual, gain, w_router, _, w_up, w_down = [v.double().cpu().requires_grad_() for v in leaves]
    h = x + residual
    n = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * gain
    s = torch.sigmoid(n @ w_router.T).gather(1, experts)
    w = SCALE * s / s.sum(1, keepdim=True)
    out = torch.zeros_like(h)
    for e in range(EXPERTS):
        t, j = torch.nonzero(experts == e, as_tuple=True)
        g, u = (n[t] @ w_up[e].T).chunk(2, 1)
        out = out.index_add(0, t, w[t, j, None] * ((g * torch.sigmoid(g) * u) @ w_down[e].T))
    ((out * dout.double().cpu()).sum() + (h * dh_next.double().cpu()).sum()).backward()
    return out.detach(), h.detach(), x.grad, gain.grad, w_router.grad, w_up.grad, w_down.grad


def test_block_against_float64_autograd():
    """Every output within what E4M3 tiles allow (codes off by at most half a step, 2^-4, a product of two by 2^-3 of
    the magnitudes summed, over random signs a few percent in the 2-norm)."""
    leaves = inputs(0)
    got = block(*leaves)
    experts = got[-1].long().cpu()
    assert int(experts.min()) >= 0
    want = reference(leaves[:7], experts, leaves[7], leaves[8])
    for name, a, b in zip(("out", "h", "dx", "dgain", "dw_router", "dw_up", "dw_down"), got, want):
        rel = float((a.double().cpu() - b).norm() / b.norm())
        say(f"{name}: {rel:.4f}")
        assert rel < 0.125, name


def test_block_captured_and_replayed():
    """One graph of the block, replayed on changing inputs with eager work between, equals the eager block."""
    static = inputs(1)
    block(*static)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(*static)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block(*static)
    for seed in (1, 2, 3, 2):
        new = inputs(seed)
        want = block(*new)
        for s, v in zip(static, new):
            s.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(out, want)):
            assert torch.equal(a, b), (seed, i)


def test_norm_gradients_on_two_streams_and_in_two_graphs():
    """Each call has its own workspace: gradients at the same time do not meet."""
    g = torch.Generator(device="cuda:0").manual_seed(3)
    args = []
    for rows in (3000, 2500, 3100, 700):
        h = torch.randn((rows, 1536), generator=g, device="cuda:0").to(torch.bfloat16)
        w = torch.randn(1536, generator=g, device="cuda:0")
        rstd = fp8q.rmsnorm_quantize(h, w, quantize=False)[3]
        args.append((torch.randn((rows, 1536), generator=g, device="cuda:0"), h, rstd, w))
    want = [fp8q.rmsnorm_backward(*a) for a in args]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append(fp8q.rmsnorm_backward(*args[k]))
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(v[0], want[k][0]) and torch.equal(v[3], want[k][3]) for v in got[k])
    graphs, outs = [], []
    for k in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(fp8q.rmsnorm_backward(*args[2 + k]))
        graphs.append(graph)
    for _ in range(5):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                graphs[k].replay()
        torch.cuda.synchronize()
        for k in range(2):
            assert torch.equal(outs[k][0], want[2 + k][0]) and torch.equal(outs[k][3], want[2 + k][3])


def test_serving_steps_in_place_captured():
    """A decoded token: the residual stream updated in place and routed, replayed step after step, as the eager steps."""
    g = torch.Generator(device="cuda:0").manual_seed(4)
    r = lambda *s: torch.randn(s, generator=g, device="cuda:0")  # noqa: E731
    w, router, bias = r(7168).to(torch.bfloat16), r(256, 7168).to(torch.bfloat16), 0.1 * r(256)
    steps = [r(1, 7168).to(torch.bfloat16) for _ in range(6)]
    r_c, r_s = fp8q.quantize_weight(router)
    r_c = r_c.contiguous()

    def step(x, stream):
        _, c, s, _, _ = fp8q.rmsnorm_quantize(x, w, residual=stream, h_out=stream)
        logits = fp8q.gemm(c.contiguous(), s, r_c, r_s, out_dtype=torch.float32)
        return (c, s) + fp8q.moe_route(logits, 8, bias=bias, groups=8, top_groups=4, scale=2.5)[:2]

    start = r(1, 7168).to(torch.bfloat16)
    stream, want = start.clone(), []
    for x in steps:
        want.append([v.clone() for v in step(x, stream)] + [stream.clone()])
    x, stream = steps[0].clone(), start.clone()
    step(x, stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x, stream)
    stream.copy_(start)
    for v, expect in zip(steps, want):
        x.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(list(out) + [stream], expect))
