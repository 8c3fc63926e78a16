"""Residual addition with RMS norm and quantization, its gradient, and the
normalised rows in token-axis tiles on the GPU, against oracle/block.py: the
forward pass, dx and the tiles bit for bit."""

import numpy as np
import pytest
import torch

import fine_grained_fp8_fp8q_amd as fp8q
from oracle import block as B, e4m3, quantize as Q
from tests.gpu_util import assert_codes_equal, assert_scales_equal, dev, host, host_bf16_bits, host_codes, need_gpu, say

pytestmark = pytest.mark.gpu
EPS = 1e-6
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _gpu(request):
    need_gpu()
    say(f"[norm] {request.node.name}")


def values(r, shape, dtype, std=1.0):
    """float32 values that dtype holds."""
    v = (std * r.normal(size=shape)).astype(np.float32)
    return B.round_to(v, "bf16") if dtype == BF else v


def rows_like(r, rows, n, dtype, std=1.0):
    """Rows of different size with wide channels."""
    return values(r, (rows, n), F32, 1.0) if n == 0 else B.round_to(
        values(r, (rows, n), F32) * (std * np.exp(0.7 * r.normal(size=(rows, 1)) + 0.5 * r.normal(size=(1, n)))).astype(np.float32),
        "bf16" if dtype == BF else "f32")


def on(v, dtype, pad=0):
    """A float32 array on the GPU in dtype, as a view of rows `pad` elements longer that hold NaN there."""
    buf = torch.full((v.shape[0], v.shape[1] + pad), float("nan"), dtype=dtype, device="cuda:0")
    buf[:, :v.shape[1]] = dev(v)
    return buf[:, :v.shape[1]]


def same_f32(got, want, what):
    got, want = host(got.float()), B.f32(want)
    bad = np.argwhere(~((got == want) | (np.isnan(got) & np.isnan(want))))
    assert got.shape == want.shape and bad.size == 0, f"{what}: {len(bad)} of {want.size} differ, first {bad[0]}: {got[tuple(bad[0])]!r} for {want[tuple(bad[0])]!r}"


def same_rows(got, bits, mode):
    """(y, codes, scales) against BF16 patterns."""
    y, codes, scales = got
    if y is not None:
        same_f32(y, e4m3.bf16_bits_to_f32(bits), "y")
    if codes is not None:
        c, s = Q.quantize_rows(bits, mode)
        assert_scales_equal(host(scales), s, "scales")
        assert_codes_equal(host_codes(codes), c, "codes")


SIZES = [(1, 1), (3, 2), (2, 127), (5, 128), (4, 129), (17, 1030), (9, 513), (1, 7168), (40, 2048), (65, 7168), (2, 8192), (3, 8200), (2, 16391), (1, 40000),
         (300, 64), (1100, 360)]


@pytest.mark.parametrize("rows,n", SIZES)
@pytest.mark.parametrize("xdt,sdt,wdt,mode", [(BF, BF, BF, "free"), (BF, None, F32, "pow2"), (F32, F32, BF, "pow2"), (F32, BF, F32, "free"), (BF, F32, BF, "free"),
                                              (F32, None, F32, "free")])
def test_norm(rows, n, xdt, sdt, wdt, mode):
    r = np.random.default_rng(rows * n)
    x, w = rows_like(r, rows, n, xdt), values(r, (n,), wdt)
    res = None if sdt is None else rows_like(r, rows, n, sdt, 2.0)
    h, rstd, bits = B.rmsnorm(x, res, w, EPS, "bf16" if sdt == BF else "f32")
    for pad in (0, 8, 3):
        xd, rd, wd = on(x, xdt, pad), None if res is None else on(res, sdt, pad), dev(w).to(wdt)
        y, codes, scales, got_r, got_h = fp8q.rmsnorm_quantize(xd, wd, residual=rd, eps=EPS, bf16=True, scale_mode=mode)
        same_f32(got_r, rstd, "rstd")
        same_rows((y, codes, scales), bits, mode)
        if res is None:
            assert got_h is None
            continue
        assert got_h.dtype == sdt
        same_f32(got_h, h, "h")
        # into a tensor of another stride, and over the residual itself
        out = torch.full((rows, n + 5), 7.0, dtype=sdt, device="cuda:0")
        for dst in (out[:, :n], rd):
            got = fp8q.rmsnorm_quantize(xd, wd, residual=rd, eps=EPS, scale_mode=mode, h_out=dst)
            assert got[4] is dst and got[0] is None
            same_f32(dst, h, "h_out")
            assert torch.equal(got[1], codes) and torch.equal(got[2], scales) and torch.equal(got[3], got_r)
        assert (host(out[:, n:].float()) == 7.0).all()
        assert pad == 0 or torch.isnan(rd._base[:, n:]).all()


def call(name, *args):
    lib = fp8q.load_library()
    st = getattr(lib, name)(*[a.data_ptr() if isinstance(a, torch.Tensor) else a for a in args], torch.cuda.current_stream().cuda_stream)
    assert st == fp8q.OK, (name, st)


@pytest.mark.parametrize("rows,n", [(5, 1030), (70, 256), (3, 9000), (1, 513)])
@pytest.mark.parametrize("ldy,ldc", [(0, 0), (8, 16), (3, 1)])
def test_norm_outputs_of_any_row_stride_leave_the_gaps_alone(rows, n, ldy, ldc):
    """Every output alone and all together, through the C ABI."""
    r = np.random.default_rng(n)
    x, res, w = rows_like(r, rows, n, BF), rows_like(r, rows, n, F32), values(r, (n,), F32)
    xd, rd, wd = on(x, BF), on(res, F32), dev(w)
    h, rstd, bits = B.rmsnorm(x, res, w, EPS, "f32")
    for which in ("h", "y", "codes", "rstd", "all"):
        ho, yo = torch.full((rows, n + ldy), 7.0, device="cuda:0"), torch.full((rows, n + ldy), 7.0, dtype=BF, device="cuda:0")
        co, so = torch.full((rows, n + ldc), 9, dtype=torch.uint8, device="cuda:0"), torch.full((rows, (n + 127) // 128), 7.0, device="cuda:0")
        ro = torch.full((rows,), 7.0, device="cuda:0")
        use = lambda k, t: t if which in (k, "all") else None  # noqa: E731
        call("fp8q_rmsnorm_quantize", xd, 1, rows, n, n, rd, 0, n, use("h", ho), n + ldy, wd, 0, EPS, use("y", yo), n + ldy, 0, use("codes", co), n + ldc,
             use("codes", so), use("rstd", ro))
        same_rows((yo[:, :n] if which in ("y", "all") else None, co[:, :n] if which in ("codes", "all") else None, so), bits, "free")
        if which in ("h", "all"):
            same_f32(ho[:, :n], h, "h")
        if which in ("rstd", "all"):
            same_f32(ro, rstd, "rstd")
        assert bool((ho[:, n:] == 7).all()) and bool((yo[:, n:] == 7).all()) and bool((co[:, n:] == 9).all())
        for k, t in (("h", ho), ("y", yo), ("rstd", ro)):
            assert which in (k, "all") or bool((t == 7).all()), k


@pytest.mark.parametrize("scale", [2.0 ** -120, 2.0 ** -60, 2.0 ** 60, 2.0 ** 120])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_of_small_and_large_rows(scale, dtype):
    """The sum of squares holds what float32 would not."""
    r = np.random.default_rng(3)
    x = rows_like(r, 6, 300, dtype, scale)
    w = values(r, (300,), BF)
    for eps in (1e-6, 1e-300):
        _, rstd, bits = B.rmsnorm(x, None, w, eps)
        if not np.isfinite(rstd).all():
            continue
        y, _, _, got, _ = fp8q.rmsnorm_quantize(on(x, dtype), dev(w).to(BF), eps=eps, bf16=True, quantize=False)
        same_f32(got, rstd, "rstd")
        same_f32(y, e4m3.bf16_bits_to_f32(bits), "y")


def test_norm_of_zeros_and_non_finite_rows():
    """A row of zeros, and rows with an infinity or a NaN beside whole ones."""
    r = np.random.default_rng(4)
    x = rows_like(r, 6, 640, BF)
    x[1] = 0
    x[1, 3] = -0.0
    w = values(r, (640,), BF)
    want = B.rmsnorm(x, None, w, EPS)
    x[2, 70], x[4, 630] = np.inf, np.nan
    y, codes, scales, rstd, _ = fp8q.rmsnorm_quantize(on(x, BF), dev(w).to(BF), eps=EPS, bf16=True)
    rows = [0, 1, 3, 5]
    c, s = Q.quantize_rows(want[2])
    assert np.array_equal(host(rstd)[rows], want[1][rows]) and host(rstd)[2] == 0 and np.isnan(host(rstd)[4])
    assert np.array_equal(host_bf16_bits(y)[rows], want[2][rows])
    assert np.array_equal(host_codes(codes)[rows], c[rows]) and np.array_equal(host(scales)[rows], s[rows])
    inf_row = host(y.float())[2]
    assert np.isnan(inf_row[70]) and (np.delete(inf_row, 70) == 0).all() and np.isnan(host(y.float())[4]).all()


def test_norm_empty():
    w = torch.ones(8, device="cuda:0")
    y, codes, scales, rstd, h = fp8q.rmsnorm_quantize(torch.zeros((0, 8), device="cuda:0"), w, bf16=True)
    assert y.shape == (0, 8) and codes.shape == (0, 8) and scales.shape == (0, 1) and rstd.shape == (0,) and h is None
    x = torch.zeros((3, 0), dtype=BF, device="cuda:0")
    y, codes, scales, rstd, h = fp8q.rmsnorm_quantize(x, w[:0], residual=x, eps=0.25, bf16=True)
    assert y.shape == (3, 0) and h.shape == (3, 0) and scales.shape == (3, 0) and host(rstd).tolist() == [2.0] * 3
    dx, codes, scales, dw = fp8q.rmsnorm_backward(torch.zeros((0, 8), device="cuda:0"), torch.zeros((0, 8), device="cuda:0"), w[:0], w, quantize=True)
    assert dx.shape == (0, 8) and codes.shape == (0, 8) and host(dw).tolist() == [0.0] * 8
    dx, _, _, dw = fp8q.rmsnorm_backward(x, x, rstd, w[:0])
    assert dx.shape == (3, 0) and dw.shape == (0,)
    codes, scales = fp8q.rmsnorm_quantize_t(x, rstd, w[:0])
    assert codes.shape == (0, 3) and scales.shape == (0, 1)
    index = torch.zeros(5, dtype=torch.int32, device="cuda:0")
    codes, scales = fp8q.rmsnorm_quantize_t(torch.zeros((0, 8), device="cuda:0"), w[:0], w, index=index)
    assert not host_codes(codes).any() and not host(scales).any() and codes.shape == (8, 5)
    codes, scales = fp8q.rmsnorm_quantize_t(torch.zeros((4, 8), device="cuda:0"), w[:4], w, index=index[:0])
    assert codes.shape == (8, 0) and scales.shape == (8, 0)


def test_a_row_does_not_depend_on_the_others():
    """The same row alone, among a few and among many, in the forward pass, dx and the token tiles' values."""
    r = np.random.default_rng(5)
    for n in (512, 7168, 9008):
        x, w = on(rows_like(r, 3000, n, BF), BF), dev(values(r, (n,), BF)).to(BF)
        dy = on(values(r, (3000, n), BF), BF)
        many = fp8q.rmsnorm_quantize(x, w, residual=dy)
        grads = fp8q.rmsnorm_backward(dy, x, many[3], w, quantize=True, want_dweight=False)
        for lo, hi in ((0, 1), (1234, 1235), (2000, 2003), (2800, 3000), (700, 1500)):
            few = fp8q.rmsnorm_quantize(x[lo:hi], w, residual=dy[lo:hi])
            for a, b in zip(few[1:], many[1:]):
                assert torch.equal(a, b[lo:hi]), (n, lo)
            if lo % 4 == 0:  # (rstd's base has to be on 16 bytes)
                part = fp8q.rmsnorm_backward(dy[lo:hi], x[lo:hi], many[3][lo:hi], w, quantize=True, want_dweight=False)
                for a, b in zip(part[:3], grads[:3]):
                    assert torch.equal(a, b[lo:hi]), (n, lo)


# -------------------------------------------------------------- backward ----

@pytest.mark.parametrize("rows,n", SIZES)
@pytest.mark.parametrize("ddt,hdt,wdt,odt,dres,mode", [(BF, BF, BF, BF, True, "free"), (BF, F32, F32, F32, False, "pow2"), (F32, BF, BF, F32, True, "free"),
                                                       (F32, F32, BF, BF, False, "pow2"), (BF, BF, F32, F32, True, "pow2"), (F32, BF, F32, BF, True, "free")])
def test_norm_backward(rows, n, ddt, hdt, wdt, odt, dres, mode):
    r = np.random.default_rng(rows + n)
    h, w, dy = rows_like(r, rows, n, hdt), values(r, (n,), wdt), values(r, (rows, n), ddt)
    res = values(r, (rows, n), odt) if dres else None
    rstd = B.rms_reciprocal(h, EPS)
    want = B.rmsnorm_backward(dy, h, rstd, w, res)
    dx64, dw64, bound, mag = B.rmsnorm_gradient(dy, h, rstd, w, res)
    for pad in (0, 8, 3):
        args = on(dy, ddt, pad), on(h, hdt, pad), dev(rstd), dev(w).to(wdt)
        rd = None if res is None else on(res, odt, pad)
        dx, codes, scales, dw = fp8q.rmsnorm_backward(*args, dres=rd, out_dtype=odt, quantize=True, scale_mode=mode)
        assert dx.dtype == odt and dw.dtype == F32
        same_f32(dx, B.round_to(want, "bf16" if odt == BF else "f32"), "dx")
        same_rows((None, codes, scales), e4m3.f32_to_bf16_bits_rne(want), mode)
        step = 2.0 ** -8 if odt == BF else 0.0
        off = np.abs(host(dx.double()) - dx64)
        assert (off <= (bound + step * np.abs(dx64)) * (1 + 2.0 ** -8) + 2.0 ** -133).all()
        # one rounding of t, one a product or fused step, one an addition, in any order of the rows
        off = np.abs(host(dw.double()) - dw64)
        assert (off <= (rows + 2) * 2.0 ** -24 * mag * 1.01).all(), float((off / np.maximum(mag, 1e-30)).max())
        # each output alone
        only = fp8q.rmsnorm_backward(*args, dres=rd, out_dtype=odt, want_dx=False, want_dweight=True)
        assert only[0] is None and only[1] is None and torch.equal(only[3], dw)
        only = fp8q.rmsnorm_backward(*args, dres=rd, out_dtype=odt, want_dweight=False)
        assert only[3] is None and torch.equal(only[0], dx)
        only = fp8q.rmsnorm_backward(*args, dres=rd, out_dtype=odt, want_dx=False, want_dweight=False, quantize=True, scale_mode=mode)
        assert torch.equal(only[1], codes) and torch.equal(only[2], scales)


@pytest.mark.parametrize("rows,n", [(9000, 40), (2500, 1030), (70000, 3)])
def test_norm_backward_of_many_rows(rows, n):
    r = np.random.default_rng(n)
    h, w, dy = rows_like(r, rows, n, BF), values(r, (n,), BF), values(r, (rows, n), BF)
    rstd = B.rms_reciprocal(h, EPS)
    args = on(dy, BF), on(h, BF), dev(rstd), dev(w).to(BF)
    dx, _, _, dw = fp8q.rmsnorm_backward(*args)
    same_f32(dx, B.round_to(B.rmsnorm_backward(dy, h, rstd, w), "bf16"), "dx")
    _, dw64, _, mag = B.rmsnorm_gradient(dy, h, rstd, w)
    assert (np.abs(host(dw.double()) - dw64) <= (rows + 2) * 2.0 ** -24 * mag * 1.01).all()
    assert torch.equal(fp8q.rmsnorm_backward(*args)[3], dw)


def test_norm_gradients_hold_their_own_memory():
    """What a caller keeps of the gradients holds no scratch memory."""
    x, w, rstd = torch.randn(600, 1030, device="cuda:0").to(BF), torch.ones(1030, device="cuda:0"), torch.ones(600, device="cuda:0")
    dx, codes, scales, dw = fp8q.rmsnorm_backward(x, x, rstd, w, quantize=True)
    for t, most in ((dx, 600 * 1030 * 2), (codes, 600 * 1040), (scales, 600 * 9 * 4), (dw, 1030 * 4)):
        assert t.untyped_storage().nbytes() <= most


@pytest.mark.parametrize("n", [1030, 1500, 1536])
@pytest.mark.parametrize("ddt,hdt,odt", [(F32, F32, F32), (F32, BF, F32), (BF, F32, BF), (BF, BF, BF)])
def test_norm_backward_of_many_rows_of_three_chunks(n, ddt, hdt, odt):
    rows = 2060
    r = np.random.default_rng(n)
    h, w, dy, res = rows_like(r, rows, n, hdt), values(r, (n,), BF), values(r, (rows, n), ddt), values(r, (rows, n), odt)
    rstd = B.rms_reciprocal(h, EPS)
    want = B.rmsnorm_backward(dy, h, rstd, w, res)
    _, dw64, _, mag = B.rmsnorm_gradient(dy, h, rstd, w, res)
    dx, codes, scales, dw = fp8q.rmsnorm_backward(on(dy, ddt), on(h, hdt), dev(rstd), dev(w).to(BF), dres=on(res, odt), out_dtype=odt, quantize=True)
    same_f32(dx, B.round_to(want, "bf16" if odt == BF else "f32"), "dx")
    same_rows((None, codes, scales), e4m3.f32_to_bf16_bits_rne(want), "free")
    # one rounding of t, one a product or fused step, one an addition, in any order of the rows
    assert (np.abs(host(dw.double()) - dw64) <= (rows + 2) * 2.0 ** -24 * mag * 1.01).all()


def test_norm_backward_in_place_and_strides():
    """dx over the gradient it adds to, and output strides through the C ABI."""
    r = np.random.default_rng(8)
    for rows, n, pad in ((9, 1030, 3), (70, 512, 8), (2, 9000, 0)):
        h, w, dy, res = rows_like(r, rows, n, BF), values(r, (n,), BF), values(r, (rows, n), BF), values(r, (rows, n), F32)
        rstd = B.rms_reciprocal(h, EPS)
        want = B.rmsnorm_backward(dy, h, rstd, w, res)
        c, s = Q.quantize_rows(e4m3.f32_to_bf16_bits_rne(want))
        rd = torch.full((rows, n + pad), 7.0, device="cuda:0")
        rd[:, :n] = dev(res)
        co, so = torch.full((rows, n + pad), 9, dtype=torch.uint8, device="cuda:0"), torch.zeros((rows, (n + 127) // 128), device="cuda:0")
        call("fp8q_rmsnorm_backward", on(dy, BF), 1, rows, n, n, on(h, BF), 1, n, dev(rstd), dev(w).to(BF), 1, rd, n + pad, rd, 0, n + pad, 0, co, n + pad, so, None,
             None, 0)
        same_f32(rd[:, :n], want, "dx")
        assert_codes_equal(host_codes(co[:, :n]), c, "codes")
        assert_scales_equal(host(so), s, "scales")
        assert bool((rd[:, n:] == 7).all()) and bool((co[:, n:] == 9).all())


def test_norm_backward_non_finite_values():
    """An infinity or NaN of a row stays in that row of dx, and in its columns of dweight where it is a dy."""
    r = np.random.default_rng(9)
    rows, n = 50, 700
    h, w, dy = rows_like(r, rows, n, BF), values(r, (n,), BF), values(r, (rows, n), BF)
    rstd = B.rms_reciprocal(h, EPS)
    clean = fp8q.rmsnorm_backward(on(dy, BF), on(h, BF), dev(rstd), dev(w).to(BF))
    dy[7, 33], dy[20, 650] = np.inf, np.nan
    dx, _, _, dw = fp8q.rmsnorm_backward(on(dy, BF), on(h, BF), dev(rstd), dev(w).to(BF))
    keep = np.delete(np.arange(rows), [7, 20])
    assert np.array_equal(host(dx.float())[keep], host(clean[0].float())[keep])
    assert not np.isfinite(host(dx.float())[7]).any() and np.isnan(host(dx.float())[20]).all()
    cols = np.delete(np.arange(n), [33, 650])
    assert np.array_equal(host(dw)[cols], host(clean[3])[cols]) and np.isinf(host(dw)[33]) and np.isnan(host(dw)[650])


def test_norm_gradients_against_differences():
    """dx and dweight of a scalar of the float32 output, against central differences of the same norm in 64 bits."""
    r = np.random.default_rng(10)
    n = 40
    x, w, dy = values(r, (3, n), F32), values(r, (n,), F32), values(r, (3, n), F32)
    rstd = fp8q.rmsnorm_quantize(on(x, F32), dev(w), eps=EPS, quantize=False)[3]
    dx, _, _, dw = fp8q.rmsnorm_backward(on(dy, F32), on(x, F32), rstd, dev(w), out_dtype=F32)

    def loss(a, b):
        return float((a / np.sqrt((a * a).mean(1, keepdims=True) + EPS) * b * dy).sum())

    x64, w64, step = x.astype(np.float64), w.astype(np.float64), 1e-6
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x64)
        e[i] = step
        # differences: 1e-6; the float32 gradient: a few steps of its largest term
        assert abs((loss(x64 + e, w64) - loss(x64 - e, w64)) / (2 * step) - float(dx[i])) < 1e-6 * 20
    for i in range(n):
        e = np.zeros(n)
        e[i] = step
        assert abs((loss(x64, w64 + e) - loss(x64, w64 - e)) / (2 * step) - float(dw[i])) < 1e-6 * 20


# ---------------------------------------------------------- token tiles ----

@pytest.mark.parametrize("rows,n", [(1, 1), (5, 64), (127, 65), (128, 64), (129, 63), (300, 1030), (1000, 136), (16, 7168), (257, 512)])
@pytest.mark.parametrize("hdt,wdt,mode", [(BF, BF, "free"), (F32, BF, "pow2"), (BF, F32, "pow2"), (F32, F32, "free")])
def test_norm_token_tiles(rows, n, hdt, wdt, mode):
    r = np.random.default_rng(rows * n)
    h, w = rows_like(r, rows, n, hdt), values(r, (n,), wdt)
    rstd = B.rms_reciprocal(h, EPS)
    bits = B.normalised_bits(h, rstd, w)
    tables = [None, r.integers(0, rows, size=2 * rows + 3), np.concatenate([r.permutation(rows), np.full(130, -1), [rows, 2 ** 31 - 1, -2 ** 31, 0]])]
    for pad in (0, 8, 3):
        for index in tables:
            want = bits
            if index is not None:
                want = np.where(((index >= 0) & (index < rows))[:, None], bits[np.clip(index, 0, rows - 1)], np.uint16(0))
            c, s = Q.quantize_token_t(want, mode)
            codes, scales = fp8q.rmsnorm_quantize_t(on(h, hdt, pad), dev(rstd), dev(w).to(wdt), index=None if index is None else dev(index.astype(np.int32)),
                                                    scale_mode=mode)
            assert_scales_equal(host(scales), s, "scales")
            assert_codes_equal(host_codes(codes), c, "codes")


def test_norm_token_tiles_equal_the_quantizers():
    """The codes and scales of the library's own quantizer on the forward pass's y, at a size that fills the chip."""
    r = np.random.default_rng(12)
    g = torch.Generator(device="cuda:0").manual_seed(12)
    h = torch.randn((4096, 2048), generator=g, device="cuda:0").to(BF)
    w = dev(values(r, (2048,), BF)).to(BF)
    y, codes, scales, rstd, _ = fp8q.rmsnorm_quantize(h, w, bf16=True, scale_mode="pow2")
    assert all(torch.equal(a, b) for a, b in zip((codes, scales), fp8q.quantize_act(y, "row", "pow2")))
    assert all(torch.equal(a, b) for a, b in zip(fp8q.rmsnorm_quantize_t(h, rstd, w), fp8q.quantize_act(y, "token_t")))


# ----------------------------------------------------- sizes and refusals ----

def test_norm_rows_past_four_gigabytes():
    """Row offsets past 2^31 elements and 2^32 bytes: the last rows against a small call on copies of them."""
    rows, n = 310_000, 7168
    g = torch.Generator(device="cuda:0").manual_seed(5)
    x = torch.zeros((rows, n), dtype=BF, device="cuda:0")
    w = torch.rand(n, generator=g, device="cuda:0").to(BF)
    x[-64:] = torch.randn((64, n), generator=g, device="cuda:0").to(BF)
    x[:64] = x[-64:]
    a, b = fp8q.rmsnorm_quantize(x, w, residual=x), fp8q.rmsnorm_quantize(x[-64:].clone(), w, residual=x[-64:].clone())
    for p, q in zip(a[1:], b[1:]):
        assert torch.equal(p[-64:], q) and torch.equal(p[:64], q)
    rstd = a[3]
    del a
    a, b = fp8q.rmsnorm_backward(x, x, rstd, w, want_dweight=False)[0], fp8q.rmsnorm_backward(x[-64:].clone(), x[-64:].clone(), rstd[-64:].clone(), w)
    assert torch.equal(a[-64:], b[0]) and torch.equal(a[:64], b[0]) and not a[64:-64].any()
    del a
    dw = fp8q.rmsnorm_backward(x, x, rstd, w, want_dx=False)[3]
    assert torch.allclose(dw, 2 * b[3], rtol=1e-5, atol=1e-4)
    index = torch.arange(rows - 128, rows, dtype=torch.int32, device="cuda:0")
    got = fp8q.rmsnorm_quantize_t(x, rstd, w, index=index)
    want = fp8q.rmsnorm_quantize_t(x[-128:].clone(), rstd[-128:].clone(), w)
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_norm_refusals_of_the_binding():
    x = torch.zeros((8, 16), dtype=BF, device="cuda:0")
    w, r = torch.ones(16, device="cuda:0"), torch.ones(8, device="cuda:0")
    for bad in (lambda: fp8q.rmsnorm_quantize(x.half(), w), lambda: fp8q.rmsnorm_quantize(x, w.double()), lambda: fp8q.rmsnorm_quantize(x, w, residual=x.half()),
                lambda: fp8q.rmsnorm_quantize(x, w, residual=x, h_out=x.float()), lambda: fp8q.rmsnorm_backward(x, x, r.double(), w),
                lambda: fp8q.rmsnorm_backward(x, x, r, w, dres=x, out_dtype=F32), lambda: fp8q.rmsnorm_backward(x, x, r, w, out_dtype=torch.float16),
                lambda: fp8q.rmsnorm_quantize_t(x, r, w, index=torch.zeros(8, dtype=torch.int64, device="cuda:0"))):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: fp8q.rmsnorm_quantize(x, w[:8]), lambda: fp8q.rmsnorm_quantize(x.t(), r), lambda: fp8q.rmsnorm_quantize(x, w, residual=x[:4]),
                lambda: fp8q.rmsnorm_quantize(x, w, h_out=x), lambda: fp8q.rmsnorm_quantize(x, w, residual=x, h_out=x[:, :8]),
                lambda: fp8q.rmsnorm_backward(x, x[:4], r, w), lambda: fp8q.rmsnorm_backward(x, x, r[:4], w), lambda: fp8q.rmsnorm_backward(x, x, r, w, dres=x[:4]),
                lambda: fp8q.rmsnorm_backward(x, x, r, w, want_dx=False, want_dweight=False), lambda: fp8q.rmsnorm_quantize_t(x, r, w.view(4, 4)),
                lambda: fp8q.rmsnorm_quantize_t(x, r[::2], w), lambda: fp8q.rmsnorm_quantize(x, w.cpu())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: fp8q.rmsnorm_quantize(x, w, eps=0.0), lambda: fp8q.rmsnorm_quantize(x, w, eps=float("nan")), lambda: fp8q.rmsnorm_quantize(x, w, eps=float("inf")),
                lambda: fp8q.rmsnorm_quantize(x[:1].expand(8, 16), w), lambda: fp8q.rmsnorm_quantize(x[:, 1:], w[:15]),
                lambda: fp8q.rmsnorm_quantize(x, w, residual=x, h_out=torch.empty((1, 16), dtype=BF, device="cuda:0").expand(8, 16))):
        with pytest.raises(fp8q.Fp8qError):
            bad()
