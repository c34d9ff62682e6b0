"""What the header says of the 8-bit products' sums, where large products cancel and the
result is made of small ones.

Tolerance, u = 2^-24. Of eight products of consecutive k, the largest has a magnitude of
2^p or more with p the sum of its operands' exponents, and is a multiple of 2^(p - 6), as
E4M3 has 3 bits behind the point: it comes out whole. Each of the others loses less than
2^(p - 13): a group is off by less than 7 2^-13 of its largest product. The sums of the
groups meet in float32, cut to the next number: 2 u of what has been summed for each
group at most, and each block's scales and fma 3 u more. All of it in absolute terms,
since the signs here are not random.
"""

import pytest
import torch

from eight import F8, U, blocks, close, cpu64, gen, spread
from muon_newton_schulz_04_amd import layers as L

pytestmark = pytest.mark.gpu


def _bound(x, w):
    """Of float64 operands [n, k], [o, k]."""
    k = x.shape[1]
    pad = (0, -k % 8)
    gx, gw = (torch.nn.functional.pad(v.abs(), pad).view(v.shape[0], -1, 8) for v in (x, w))
    largest = torch.zeros(x.shape[0], w.shape[0], dtype=torch.float64)
    for j in range(gx.shape[1]):
        largest += (gx[:, None, j] * gw[None, :, j]).amax(2)
    return 7 * 2.0 ** -13 * largest + (2 * gx.shape[1] + 3 * blocks(k)) * U * (x.abs() @ w.abs().t())


def _scaled(q, s, tall):
    return cpu64(q.float()) * spread(s.double(), tall, *q.shape)


def _rows16(q):
    """The same on the GPU, in rows that start 16-byte aligned."""
    r, c = q.shape
    buf = torch.zeros(r, (c + 15) // 16 * 16, dtype=torch.uint8)
    buf[:, :c] = q.view(torch.uint8)
    return buf.cuda().view(q.dtype)[:, :c]


@pytest.mark.parametrize("n", [1, 30, 300, 2050])
@pytest.mark.parametrize("k", [128, 136, 700])
def test_large_products_that_cancel(n, k):
    """Every eight products hold two large ones of opposite sign; the others are smaller
    by 2^4 to 2^18."""
    g = gen(n + k)
    o, fmt = 72, F8["e4m3"]
    x = torch.randn(n, k, generator=g) * torch.exp2(torch.randint(-7, 0, (n, k), generator=g).float())
    w = torch.randn(o, k, generator=g) * torch.exp2(torch.randint(-7, 0, (o, k), generator=g).float())
    for j in range(0, k - 7, 8):
        a, b = torch.randperm(8, generator=g)[:2].tolist()
        x[:, j + a] = x[:, j + b] = 16 * (1 + torch.rand(n, generator=g))
        w[:, j + a] = 16 * (1 + torch.rand(o, generator=g))
        w[:, j + b] = -w[:, j + a]
    x, w = x.to(fmt), w.to(fmt)
    sx, sw = (torch.exp2(torch.randint(-3, 4, s, generator=g).float()) for s in ((blocks(k), n), (blocks(o), blocks(k))))
    y = L.linear_fp8_forward((_rows16(x), sx.cuda()), (_rows16(w), sw.cuda()), dtype=torch.float16)
    x64, w64 = _scaled(x, sx.t(), 1), _scaled(w, sw, 128)
    close(y, x64 @ w64.t(), _bound(x64, w64), torch.float16)


def test_groups_meet_in_float32():
    """A product 22 powers of two below two that cancel, in another eight of the block."""
    for n in (16, 64, 600):
        for k1, k2 in ((1, 9), (64, 33), (127, 8)):
            x, w = torch.zeros(n, 128), torch.zeros(16, 128)
            x[:, 0] = x[:, k1] = w[:, 0] = 2.0 ** 7
            w[:, k1] = -2.0 ** 7
            x[:, k2] = w[:, k2] = 2.0 ** -4
            y = L.linear_fp8_forward((x.to(F8["e4m3"]).cuda(), torch.ones(1, n, device="cuda")),
                                     (w.to(F8["e4m3"]).cuda(), torch.ones(1, 1, device="cuda")), dtype=torch.float16)
            assert (y.float() == 2.0 ** -8).all(), (n, k1, k2)
