"""The expert-layer operators at the largest sizes their entry points accept."""

import pytest
import torch

import fine_grained_fp8_fp8q_amd as fp8q
from tests.gpu_util import need_gpu, say

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
