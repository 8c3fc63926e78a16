"""The step between a block's linear layers at the largest sizes its entry points accept."""

import pytest
import torch

import fine_grained_fp8_fp8q_amd as fp8q
from tests.gpu_util import need_gpu, say

pytestmark = pytest.mark.gpu
BF, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
MOST = 2 ** 31 - 1
PERIOD = 1 << 22  # every input repeats after so many rows: so must every output


@pytest.fixture(autouse=True)
def _gpu(request):
    need_gpu()
    say(f"[block sizes] {request.node.name}")
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def repeated(rows, seed, dtype=BF):
    g = torch.Generator(device="cuda:0").manual_seed(seed)
    t = torch.empty(rows, dtype=dtype, device="cuda:0")
    t[:PERIOD] = torch.randn(PERIOD, generator=g, device="cuda:0").to(dtype)
    whole = rows // PERIOD
    t[PERIOD:whole * PERIOD].view(whole - 1, PERIOD).copy_(t[:PERIOD])
    t[whole * PERIOD:] = t[:rows - whole * PERIOD]
    return t


def repeats(t, first):
    """Whether t is `first`, the small call's output, over and over."""
    whole = t.numel() // PERIOD
    return all(torch.equal(t[i * PERIOD:(i + 1) * PERIOD], first) for i in range(whole)) and torch.equal(t[whole * PERIOD:], first[:t.numel() - whole * PERIOD])


def guarded(n, dtype):
    """n elements between others that have to stay as they are."""
    buf = torch.full((n + 128,), 7, dtype=dtype, device="cuda:0")
    return buf, buf[64:64 + n]


def untouched(buf):
    return (buf[:64] == 7).all().item() and (buf[-64:] == 7).all().item()


def call(name, *args):
    args = [a.data_ptr() if isinstance(a, torch.Tensor) else a for a in args]
    assert getattr(fp8q.load_library(), name)(*args, torch.cuda.current_stream().cuda_stream) == fp8q.OK
    torch.cuda.synchronize()
    say(f"[block sizes] {name} done")


def test_norm_of_the_most_rows():
    w = torch.full((1,), 1.5, device="cuda:0")
    x = repeated(MOST, 1)
    small = fp8q.rmsnorm_quantize(x[:PERIOD, None], w, bf16=True, quantize=False)
    (yb, y), (rb, rstd) = guarded(MOST, BF), guarded(MOST, F32)
    call("fp8q_rmsnorm_quantize", x, 1, MOST, 1, 1, None, 1, 1, None, 1, w, 0, 1e-6, y, 1, 0, None, 1, None, rstd)
    assert repeats(y, small[0][:, 0]) and repeats(rstd, small[3]) and untouched(yb) and untouched(rb)
    del y, yb
    # its gradient: that of the gain is a sum of ones
    small = fp8q.rmsnorm_backward(x[:PERIOD, None], x[:PERIOD, None], rstd[:PERIOD].clone(), w)[0]
    one, (db, dx) = torch.ones(MOST, dtype=BF, device="cuda:0"), guarded(MOST, BF)
    call("fp8q_rmsnorm_backward", x, 1, MOST, 1, 1, x, 1, 1, rstd, w, 0, None, 1, dx, 1, 1, 0, None, 1, None, None, None, 0)
    assert repeats(dx, small[:, 0]) and untouched(db)
    del dx, db
    rstd.fill_(1.0)
    dw, need = torch.zeros(4, device="cuda:0"), fp8q.load_library().fp8q_rmsnorm_backward_workspace(MOST, 1)
    work = torch.empty(need // 4, device="cuda:0")
    call("fp8q_rmsnorm_backward", one, 1, MOST, 1, 1, one, 1, 1, rstd, w, 0, None, 1, None, 1, 1, 0, None, 1, None, dw, work, need)
    # (sums of up to 2^24 ones are exact, those above it round to steps of at most 2^8)
    assert 2.0 ** 31 - 2.0 ** 8 <= dw[0].item() <= 2.0 ** 31 and not dw[1:].any()


def test_norm_of_the_longest_rows():
    """2^30 - 1 columns: offsets past 2^32 bytes in a row, gone over in steps."""
    n = 2 ** 30 - 1
    x, w = repeated(n, 2), torch.ones(n, dtype=BF, device="cuda:0")
    (yb, y), rstd = guarded(n, BF), torch.empty(1, device="cuda:0")
    call("fp8q_rmsnorm_quantize", x, 1, 1, n, n, None, 1, n, None, n, w, 1, 1e-6, y, n, 0, None, n, None, rstd)
    # 64-bit sums by the library, of 2^30 squares
    want = 1.0 / (sum((x[i:i + (1 << 26)].double() ** 2).sum().item() for i in range(0, n, 1 << 26)) / n + 1e-6) ** 0.5
    assert abs(rstd.item() - want) <= want * (2.0 ** -24 + 2.0 ** -40)
    assert repeats(y, (x[:PERIOD].float() * rstd).to(BF)) and untouched(yb)


def test_norm_gradient_of_the_longest_row():
    """One row of 2^30 - 1 columns: dw is dy t itself, dx its formula with a sum over all of them."""
    n = 2 ** 30 - 1
    h, dy, rstd = repeated(n, 5), repeated(n, 6), torch.full((1,), 0.875, device="cuda:0")
    w = torch.ones(n, dtype=BF, device="cuda:0")
    (xb, dx), (wb, dw) = guarded(n, BF), guarded(n, F32)
    need = fp8q.load_library().fp8q_rmsnorm_backward_workspace(1, n)
    work = torch.empty(need // 4, device="cuda:0")
    call("fp8q_rmsnorm_backward", dy, 1, 1, n, n, h, 1, n, rstd, w, 1, None, n, dx, 1, n, 0, None, n, None, dw, work, need)
    t = h[:PERIOD].float() * rstd
    assert repeats(dw, dy[:PERIOD].float() * t) and untouched(wb) and untouched(xb)
    dot = sum((dy[i:i + (1 << 26)].double() * h[i:i + (1 << 26)].double()).sum().item() for i in range(0, n, 1 << 26))
    mean = torch.tensor(dot * 0.875 / n, dtype=F32, device="cuda:0")
    assert repeats(dx, ((dy[:PERIOD].float() - t * mean) * rstd).to(BF))


def test_token_tiles_of_the_most_rows():
    rows = 128 * (2 ** 24 - 1)
    h, w, (rb, rstd) = repeated(rows, 3), torch.full((1,), 0.75, device="cuda:0"), guarded(rows, F32)
    rstd.fill_(1.25)
    codes, scales = fp8q.rmsnorm_quantize_t(h[:PERIOD, None], rstd[:PERIOD].clone(), w)
    (cb, c), (sb, s) = guarded(rows, U8), guarded(rows // 128, F32)
    call("fp8q_rmsnorm_quantize_t", h, 1, rows, 1, 1, rstd, w, 0, None, rows, 0, c, rows + 64, s)
    assert repeats(c, codes[0]) and untouched(cb) and untouched(sb)
    period = PERIOD // 128
    assert all(torch.equal(s[i:i + period], scales[0, :min(period, s.numel() - i)]) for i in range(0, s.numel(), period))


def test_route_of_the_most_tokens():
    x = repeated(MOST, 4)
    e0, w0, _ = fp8q.moe_route(x[:PERIOD, None], 1, renormalize=False)
    (eb, e), (wb, w) = guarded(MOST, I32), guarded(MOST, F32)
    call("fp8q_moe_route", x, 1, MOST, 1, 1, None, fp8q.SCORE_SIGMOID, 1, 1, fp8q.GROUP_MAX, 1, 0, 1.0, fp8q.INDEX_I32, e, w, None, None)
    assert repeats(e, e0[:, 0]) and repeats(w, w0[:, 0]) and untouched(eb) and untouched(wb)
    d0 = fp8q.moe_route_backward(w0, e0, x[:PERIOD, None], renormalize=False)
    db, d = guarded(MOST, BF)
    call("fp8q_moe_route_backward", w, e, fp8q.INDEX_I32, MOST, 1, x, 1, 1, 1, fp8q.SCORE_SIGMOID, 0, 1.0, None, d, 1, 1)
    assert repeats(d, d0[:, 0]) and untouched(db)
