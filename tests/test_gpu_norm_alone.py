"""A row's results do not depend on the other rows nor on their number: rows
whose 1 / rms, or whose mean in the gradient, lies so close to the border
between two float32 values that another order of the 64-bit sum would round it
the other way, alone and in batches of every size at which the kernels change."""

import numpy as np
import pytest
import torch

import fine_grained_fp8_fp8q_amd as fp8q
from tests.gpu_util import dev, need_gpu, say

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-6
ROWS = 300  # different ones; a batch repeats them


@pytest.fixture(autouse=True)
def _gpu(request):
    need_gpu()
    say(f"[norm alone] {request.node.name}")


def border_above(v):
    """The border between the float32 next below v and the one below that, in extended precision."""
    low = np.nextafter(np.float32(v), np.float32(0))
    return (np.longdouble(low) + np.longdouble(np.nextafter(low, np.float32(0)))) / 2


def rows_at_a_border(r, n):
    """float32 rows whose 1 / rms is within a few 64-bit steps of the sum of a border: two values of each make up what the sum lacks,
    the second what the first leaves."""
    x = r.normal(size=(ROWS, n)).astype(np.float32)
    at = r.integers(0, n, size=(ROWS, 2))
    at[:, 1] = (at[:, 0] + 1 + r.integers(0, n - 1, size=ROWS)) % n
    for t in range(ROWS):
        x[t, at[t]] = 0
        wide = x[t].astype(np.longdouble)
        rest = (wide * wide).sum()
        border = border_above(1 / np.sqrt(rest / n + EPS))
        lacks = n * (1 / (border * border) - np.longdouble(EPS)) - rest + np.longdouble(r.uniform(-3, 3) * 2.0 ** -52) * rest
        for i in at[t]:
            v = np.float32(np.sqrt(lacks))
            v = np.nextafter(v, np.float32(0)) if np.longdouble(v) ** 2 > lacks else v
            x[t, i] = v
            lacks -= np.longdouble(v) ** 2
    return x


@pytest.mark.parametrize("n,pad", [(1032, 0), (1030, 3), (1280, 0), (1536, 0), (1535, 1), (1544, 0), (2048, 0), (2048, 1), (4104, 0), (7168, 0), (7168, 5), (9000, 0), (16384, 0)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_of_a_row_is_that_of_the_row_alone(n, pad, residual):
    r = np.random.default_rng(n + pad)
    x = torch.zeros((ROWS, n + pad), device="cuda:0")[:, :n]
    x.copy_(dev(rows_at_a_border(r, n)))
    w = dev((1 + 0.2 * r.normal(size=n)).astype(np.float32))

    def norm(v):
        return fp8q.rmsnorm_quantize(v, w, residual=torch.zeros_like(v) if residual else None, eps=EPS, bf16=True)[:4]

    want = norm(x)
    alone = [norm(x[t:t + 1].clone()) for t in range(40)]
    for i, v in enumerate(want):
        assert torch.equal(v[:40], torch.cat([a[i] for a in alone])), i
    for rows in (2047, 2048, 4095, 4096, 5000):
        pick = torch.arange(rows, device="cuda:0") % ROWS
        many = torch.zeros((rows, n + pad), device="cuda:0")[:, :n]
        many.copy_(x[pick])
        for i, v in enumerate(norm(many)):
            bad = torch.nonzero((v != want[i][pick]).reshape(rows, -1).any(1)).flatten()
            assert bad.numel() == 0, (rows, i, bad.numel(), bad[0].item())


def gradients_at_a_border(r, n):
    """(dy, h), float32, of positive terms whose mean is within a few 64-bit steps of a border."""
    h, dy = np.abs(r.normal(size=(ROWS, n))).astype(np.float32), np.abs(r.normal(size=(ROWS, n))).astype(np.float32)
    first = r.integers(0, n - 1, size=ROWS)
    for t in range(ROWS):
        i = first[t]
        h[t, i], h[t, i + 1], dy[t, i], dy[t, i + 1] = 1, 2.0 ** -20, 0, 0
        rest = (dy[t].astype(np.longdouble) * h[t].astype(np.longdouble)).sum()
        border = (np.longdouble(np.float32(rest / n)) + np.longdouble(np.nextafter(np.float32(rest / n), np.float32(9)))) / 2
        lacks = border * n - rest + np.longdouble(r.uniform(-3, 3) * 2.0 ** -52) * rest
        dy[t, i] = np.float32(lacks)
        dy[t, i + 1] = np.float32((lacks - np.longdouble(dy[t, i])) * 2 ** 20)
    return dy, h


@pytest.mark.parametrize("n,pad", [(1030, 0), (1032, 0), (1536, 0), (1536, 1), (2048, 0), (7168, 0), (520, 0)])
@pytest.mark.parametrize("odt", [F32, BF])
def test_gradient_of_a_row_is_that_of_the_row_alone(n, pad, odt):
    r = np.random.default_rng(n + pad)
    values = gradients_at_a_border(r, n)
    w = torch.ones(n, device="cuda:0")

    def grad(pick):
        t = [torch.zeros((len(pick), n + pad), device="cuda:0")[:, :n].copy_(dev(v[pick])) for v in values]
        return fp8q.rmsnorm_backward(t[0], t[1], torch.ones(len(pick), device="cuda:0"), w, out_dtype=odt, quantize=True, want_dweight=False)[:3]

    want = grad(np.arange(ROWS))
    alone = [grad(np.array([t])) for t in range(20)]
    for i, v in enumerate(want):
        assert torch.equal(v[:20], torch.cat([a[i] for a in alone])), i
    for rows in (600, 1600, 2047, 2048, 4096):
        pick = np.arange(rows) % ROWS
        for i, v in enumerate(grad(pick)):
            bad = torch.nonzero((v != want[i][dev(pick)]).reshape(rows, -1).any(1)).flatten()
            assert bad.numel() == 0, (rows, i, bad.numel(), bad[0].item())
