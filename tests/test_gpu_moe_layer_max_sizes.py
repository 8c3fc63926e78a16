"""The expert-layer operators at the largest sizes their entry points accept."""

import pytest
import torch

import fine_grained_fp8_fp8q_amd as fp8q
from oracle import quantize as Q
from tests.gpu_util import assert_codes_equal, assert_scales_equal, host, host_bf16_bits, host_codes, need_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(request):
    need_gpu()
    say(f"[moe layer sizes] {request.node.name}")
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def chunks(n, size=1 << 28):
    return [(a, min(a + size, n)) for a in range(0, n, size)]


def ar(a, b):
    return torch.arange(a, b, dtype=torch.int32, device="cuda:0")


def test_sort_pads_up_to_the_largest_row():
    """One pair, one expert, padded to 2^31 - 2 rows, with memory on either side of the table that stays as it was."""
    cap, guard = 2 ** 31 - 2, 1 << 20
    buf = torch.full((guard + cap + guard,), 5, dtype=torch.int32, device="cuda:0")
    token = buf[guard:guard + cap]
    small = torch.full((16,), 9, dtype=torch.int32, device="cuda:0")  # expert | row_of | offsets, 16 bytes each
    small[0] = 0
    p = small.data_ptr()
    st = fp8q.load_library().fp8q_moe_sort(p, fp8q.INDEX_I32, 1, 1, 1, 0, 1, cap, cap, p + 32, token.data_ptr(), p + 16, None, 0,
                                           torch.cuda.current_stream().cuda_stream)
    assert st == fp8q.OK
    assert small[4].item() == 0 and small[8:10].tolist() == [0, cap]
    assert token[0].item() == 0
    assert all((token[max(a, 1):b] == -1).all().item() for a, b in chunks(cap))
    assert (buf[:guard] == 5).all().item() and (buf[guard + cap:] == 5).all().item()


def test_sort_of_the_most_pairs():
    """2^31 - 3 pairs of one expert (the last row is padding), and 2^31 - 5 that go to two hosted experts and a third in turn."""
    pairs = 2 ** 31 - 3
    experts = torch.zeros((pairs, 1), dtype=torch.int32, device="cuda:0")
    offsets, token, row_of = fp8q.moe_sort(experts, 1, align=2)
    assert offsets.tolist() == [0, pairs + 1] and token.numel() == pairs + 1 and token[pairs].item() == -1
    for a, b in chunks(pairs):
        assert torch.equal(row_of[a:b, 0], ar(a, b)) and torch.equal(token[a:b], ar(a, b)), a
    del token, row_of
    pairs -= 2
    for a, b in chunks(pairs):
        experts[a:b, 0] = ar(a, b) % 3
    offsets, token, row_of = fp8q.moe_sort(experts[:pairs], 2, align=2)
    n = [(pairs + 2 - e) // 3 for e in range(2)]
    start = [0, (n[0] + 1) // 2 * 2]
    end = start[1] + (n[1] + 1) // 2 * 2
    assert offsets.tolist() == start + [end]
    for a, b in chunks(pairs):
        p = ar(a, b)
        e = p % 3
        assert torch.equal(row_of[a:b, 0], torch.where(e == 2, -1, p // 3 + torch.where(e == 1, start[1], 0)).int()), a
    for g in range(2):
        for a, b in chunks(n[g]):
            assert torch.equal(token[start[g] + a:start[g] + b], 3 * ar(a, b) + g), (g, a)
    assert (token[n[0]:start[1]] == -1).all().item() and (token[start[1] + n[1]:end] == -1).all().item()
    assert all((token[max(a, end):b] == -1).all().item() for a, b in chunks(token.numel()) if b > end)


MOST = (1 << 30) - 1  # columns of a row
PAST = 7.0            # in every output before the call


def whole(shape, gen, low=-4, high=5):
    """Whole numbers as BF16: sums of a few million are exact in float32."""
    return torch.randint(low, high, shape, generator=gen, device="cuda:0", dtype=torch.int8).bfloat16()


def gen(seed):
    return torch.Generator(device="cuda:0").manual_seed(seed)


def test_combine_of_the_most_tokens():
    """2^24 - 1 tokens of one step each."""
    g, tokens, cap = gen(1), (1 << 24) - 1, 1000003
    y = whole((cap, 8), g)
    rows = (ar(0, tokens).long() * 7919 % (cap + 5)).int()[:, None].contiguous()  # (a few outside)
    want = torch.where(rows < cap, y[rows[:, 0].clamp(max=cap - 1).long()], 0)
    assert torch.equal(fp8q.moe_combine(y, rows, out=torch.full((tokens, 8), PAST, device="cuda:0")), want.float())
    assert torch.equal(fp8q.moe_combine(y, rows), want)


def test_combine_of_the_widest_rows():
    """One token, two rows of 2^30 - 1 columns; the second starts off a 16-byte boundary."""
    y = whole((2, MOST), gen(2))
    w = torch.tensor([[0.5, 2.0]], device="cuda:0")
    rows = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda:0")
    out = fp8q.moe_combine(y, rows, w, out=torch.full((1, MOST), PAST, device="cuda:0"))
    for a, b in chunks(MOST):
        assert torch.equal(out[0, a:b], 0.5 * y[1, a:b].float() + 2.0 * y[0, a:b].float()), a
    del out
    out = fp8q.moe_combine(y, rows, w)
    for a, b in chunks(MOST):
        assert torch.equal(out[0, a:b], (0.5 * y[1, a:b].float() + 2.0 * y[0, a:b].float()).bfloat16()), a


def test_combine_backward_of_the_most_pairs():
    """tokens * topk + rows_cap / 4 just below 2^24 - 1; every fifth pair without a row, its row cleared."""
    g, pairs = gen(3), 13421771
    p = ar(0, pairs)
    gone = p % 5 == 0
    rows = torch.where(gone, -1, pairs - 1 - p).int()[:, None].contiguous()
    token = torch.where(gone, -1, p).int().flip(0).contiguous()
    dout, y = whole((pairs, 8), g), whole((pairs, 8), g)
    w = torch.where(p % 2 == 0, 0.25, -2.0)[:, None].contiguous()
    dy, codes, scales, dw = fp8q.moe_combine_backward(dout, y, rows, w, token, quantize=True)
    want = torch.where(gone[:, None], 0.0, dout.float() * w).flip(0).bfloat16()
    assert torch.equal(dy, want)
    assert torch.equal(dw[:, 0], torch.where(gone, 0.0, (dout.float() * y.flip(0).float()).sum(1)))
    again, again_s = fp8q.quantize_act(want)
    assert torch.equal(codes, again) and torch.equal(scales, again_s)
    with pytest.raises(fp8q.Fp8qError):
        fp8q.moe_combine_backward(dout.expand(pairs, 8), y.new_empty((pairs + 16, 8)), rows, w)


def test_combine_backward_of_the_widest_rows():
    """Two pairs of 2^30 - 1 columns, to BF16 and E4M3."""
    g = gen(4)
    dout, y = whole((1, MOST), g), torch.zeros((2, MOST), dtype=torch.bfloat16, device="cuda:0")
    y[:, ::4096] = whole((2, -(-MOST // 4096)), g)
    y[:, -1] = 3.0
    rows = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda:0")
    w = torch.tensor([[0.3, -5.0]], device="cuda:0")
    dy, codes, scales, dw = fp8q.moe_combine_backward(dout, y, rows, w, quantize=True)
    at = torch.cat([torch.arange(0, MOST, 4096, device="cuda:0"), torch.tensor([MOST - 1], device="cuda:0")])
    for j in range(2):
        row = 1 - j
        assert dw[0, j].item() == (dout[0, at].float() * y[row, at].float()).sum(dtype=torch.float64).item()
        for a, b in chunks(MOST):
            assert torch.equal(dy[row, a:b], (w[0, j] * dout[0, a:b].float()).bfloat16()), (j, a)
        for a in (0, (1 << 29) - 128, MOST // 128 * 128 - 128):  # whole tiles, and the last one
            b = min(a + 384, MOST)
            oc, os_ = Q.quantize_rows(host_bf16_bits(dy[row:row + 1, a:b]))
            assert_codes_equal(host_codes(codes[row:row + 1, a:b]), oc, f"codes at {a}")
            assert_scales_equal(host(scales[row:row + 1, a // 128:-(-b // 128)]), os_, f"scales at {a}")


@pytest.mark.parametrize("rows,inter", [((1 << 28) - 17, 1), (1, MOST)])
def test_swiglu_backward_of_the_most_tiles(rows, inter):
    """rows * ceil(inter / 128) just below 2^28 - 16, and the widest row: inputs that repeat every 1000 elements of the long
    axis give outputs that do, and equal those of the first 1000 alone."""
    g, dim = gen(5), 1 if rows == 1 else 0
    period, n = 1000, max(rows, inter)
    small = [torch.randn((1, period) if dim else (period, 1), generator=g, device="cuda:0").bfloat16() for _ in range(3)]
    reps = -(-n // period)
    gate, up, dy = (v.repeat((1, reps) if dim else (reps, 1)).narrow(dim, 0, n) for v in small)
    x = torch.cat([gate, up], 1)
    del gate, up
    dx, y, _, _ = fp8q.swiglu_backward(x, dy.contiguous(), want_y=True)
    del x, dy
    sdx, sy, _, _ = fp8q.swiglu_backward(torch.cat(small[:2], 1), small[2], want_y=True)
    for long, short in ((dx[:, :inter], sdx[:, :sdx.shape[1] // 2]), (dx[:, inter:], sdx[:, sdx.shape[1] // 2:]), (y, sy)):
        long, short = long.reshape(-1), short.reshape(-1)
        full = n // period * period
        assert (long[:full].view(-1, period) == short).all().item() and torch.equal(long[full:], short[:n - full])


def codes_of(shape, g):
    """E4M3 codes of -1, 0 and 1."""
    return torch.tensor([0xB8, 0, 0x38], dtype=torch.uint8, device="cuda:0")[torch.randint(0, 3, shape, generator=g, device="cuda:0", dtype=torch.uint8).int()]


def value(codes):
    return codes.view(torch.float8_e4m3fn).float()


@pytest.mark.parametrize("acc", ["fp32", "fp32_pow2", "fp8_mfma", "fp8_mfma_scaled"])
def test_grouped_wgrad_of_the_longest_token_axis(acc):
    """2^24 - 128 tokens, both operands just below 2 GiB; sums of whole numbers below 2^24 are exact."""
    g, cap, n = gen(6), (1 << 24) - 128, 127
    dy, x = codes_of((n, cap), g), codes_of((n, cap), g)
    one = torch.ones((n, cap // 128), device="cuda:0")
    cut = 128 * 50000
    offsets = torch.tensor([0, cut, cut, cap], dtype=torch.int32, device="cuda:0")
    out = fp8q.grouped_wgrad(dy, one, x, one, offsets, acc=acc)
    for i, (a, b) in enumerate(((0, cut), (cut, cut), (cut, cap))):
        want = torch.zeros((n, n), dtype=torch.float64, device="cuda:0")
        for c in range(a, b, 1 << 20):
            want += (value(dy[:, c:min(c + (1 << 20), b)]) @ value(x[:, c:min(c + (1 << 20), b)]).t().contiguous()).double()
        assert torch.equal(out[i].double(), want), i


@pytest.mark.parametrize("acc", ["fp32", "fp32_pow2"])
def test_grouped_wgrad_of_the_largest_operands(acc):
    """16383 x 16383 outputs over 131072 tokens: operands just below 2 GiB on 128 x 128 and 256 x 256 tiles."""
    g, cap, n = gen(7), 1 << 17, 16383
    dy, x = codes_of((n, cap), g), codes_of((n, cap), g)
    one = torch.ones((n, cap // 128), device="cuda:0")
    offsets = torch.tensor([0, cap], dtype=torch.int32, device="cuda:0")
    out = fp8q.grouped_wgrad(dy, one, x, one, offsets, acc=acc)[0]
    pick = torch.tensor([0, 1, 127, 128, 255, 256, 8191, 8192, 16255, 16256, n - 2, n - 1], device="cuda:0")
    for a, b in ((0, n // 2), (n // 2, n)):
        assert torch.equal(out[pick, a:b], value(dy[pick]) @ value(x[a:b]).t().contiguous()), a
        assert torch.equal(out[a:b, pick], value(dy[a:b]) @ value(x[pick]).t().contiguous()), a


def test_grouped_wgrad_of_the_most_groups():
    """262143 groups of one output, every second without tokens."""
    g, groups = gen(8), (1 << 18) - 1
    cap = 128 * (groups // 2)
    dy, x = codes_of((1, cap), g), codes_of((1, cap), g)
    one = torch.ones((1, cap // 128), device="cuda:0")
    offsets = (128 * torch.div(torch.arange(groups + 1, device="cuda:0"), 2, rounding_mode="floor")).int()
    out = torch.full((groups, 1, 1), PAST, device="cuda:0")
    fp8q.grouped_wgrad(dy, one, x, one, offsets, out=out)
    sums = (value(dy) * value(x)).view(-1, 128).sum(1)
    assert torch.equal(out[1::2, 0, 0], sums) and not out[0::2].any().item()
    with pytest.raises(fp8q.Fp8qError):
        fp8q.grouped_wgrad(dy, one, x, one, torch.cat([offsets, offsets[-1:]]))
