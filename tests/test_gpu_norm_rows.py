"""Every row once: the gain's gradient of small whole numbers, whose float32
sums are exact in any order, against their 64-bit sums by equality, so that one
row lost or taken twice shows; and rows beyond a workgroup's registers in
numbers that make several blocks of them, forward and backward."""

import numpy as np
import pytest
import torch

import fine_grained_fp8_fp8q_amd as fp8q
from oracle import block as B, e4m3, quantize as Q
from tests.gpu_util import assert_codes_equal, assert_scales_equal, dev, host, host_codes, need_gpu, say

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


@pytest.fixture(autouse=True)
def _gpu(request):
    need_gpu()
    say(f"[norm rows] {request.node.name}")


def whole(g, rows, n, dtype, pad):
    """-3 .. 3, as a view of rows `pad` elements longer."""
    t = torch.zeros((rows, n + pad), dtype=dtype, device="cuda:0")[:, :n]
    t.copy_(torch.randint(-3, 4, (rows, n), generator=g, device="cuda:0"))
    return t


# waves and workgroups that go round their rows, with a last turn that is not full; rows of every number of chunks; several
# blocks of long rows, the last ones short or (16385 rows in 512 blocks of 33) without any
@pytest.mark.parametrize("rows,n", [(9000, 40), (70000, 3), (2049, 512), (5000, 520), (2500, 1030), (8193, 1030), (4099, 1536), (1500, 2048), (4097, 2056), (1030, 7168),
                                    (513, 8192), (33, 8200), (100, 8200), (1000, 8200), (16385, 8200), (33, 16400), (100, 16400), (1000, 16400), (700, 16384), (129, 40000)])
@pytest.mark.parametrize("ddt,hdt,odt", [(BF, BF, BF), (F32, F32, F32), (F32, BF, BF), (BF, F32, BF)])
def test_gains_gradient_has_every_row_once(rows, n, ddt, hdt, odt):
    g = torch.Generator(device="cuda:0").manual_seed(rows + n)
    for pad in (0, 3) if rows * n < 1 << 26 else (0,):
        dy, h = whole(g, rows, n, ddt, pad), whole(g, rows, n, hdt, pad)
        # (at most 9 a row: below 2^24, where float32 counts)
        want = sum((dy[i:i + 4096].double() * h[i:i + 4096].double()).sum(0) for i in range(0, rows, 4096))
        one, w = torch.ones(rows, device="cuda:0"), torch.ones(n, device="cuda:0")
        for want_dx in (False, True):
            got = fp8q.rmsnorm_backward(dy, h, one, w, out_dtype=odt, want_dx=want_dx)[3]
            bad = torch.nonzero(got.double() != want).flatten()
            assert bad.numel() == 0, (pad, want_dx, bad.numel(), bad[0].item(), got[bad[0]].item(), want[bad[0]].item())


@pytest.mark.parametrize("rows,n,dtype", [(33, 16400, BF), (100, 16391, BF), (40, 8200, F32), (35, 16400, F32)])
def test_long_rows(rows, n, dtype):
    """Forward, dx and its codes, bit for bit as the oracle has them."""
    r = np.random.default_rng(n + rows)
    v = lambda *s: B.round_to(r.normal(size=s).astype(np.float32), "bf16" if dtype == BF else "f32")  # noqa: E731
    x, res, w, dy = v(rows, n), v(rows, n), B.round_to(v(n), "bf16"), v(rows, n)
    put = lambda a, d=dtype: dev(a).to(d)  # noqa: E731
    h, rstd, bits = B.rmsnorm(x, res, w, EPS, "bf16" if dtype == BF else "f32")
    y, codes, scales, got_r, got_h = fp8q.rmsnorm_quantize(put(x), put(w, BF), residual=put(res), eps=EPS, bf16=True)
    assert np.array_equal(host(got_h.float()), h) and np.array_equal(host(got_r), rstd)
    assert np.array_equal(host(y.float()), e4m3.bf16_bits_to_f32(bits))
    c, s = Q.quantize_rows(bits)
    assert_codes_equal(host_codes(codes), c, "codes")
    assert_scales_equal(host(scales), s, "scales")
    want = B.rmsnorm_backward(dy, h, rstd, w, res)
    dx, codes, scales, dw = fp8q.rmsnorm_backward(put(dy), put(h), dev(rstd), put(w, BF), dres=put(res), quantize=True)
    assert np.array_equal(host(dx.float()), B.round_to(want, "bf16" if dtype == BF else "f32"))
    c, s = Q.quantize_rows(e4m3.f32_to_bf16_bits_rne(want))
    assert_codes_equal(host_codes(codes), c, "codes of dx")
    assert_scales_equal(host(scales), s, "scales of dx")
    _, dw64, _, mag = B.rmsnorm_gradient(dy, h, rstd, w, res)
    # a block's 32 fused steps at most (and t's rounding), then its shares: 64 sums of 8 at most, four at a time and 16
    assert (np.abs(host(dw.double()) - dw64) <= (33 + 8 + 4 + 16) * 2.0 ** -24 * mag * 1.01).all()
