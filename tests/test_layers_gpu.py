"""The layer operators on the GPU against plain float64 implementations of
their definitions.

Tolerances. Inputs are exact in their 16-bit type, so a product's terms are
exact in float32; sums are taken in float32. For a sum of K terms of magnitude
sum|t| in float32, any order of additions (and the matrix unit's) is off by at
most K 2^-24 sum|t|; in practice the errors are independent and the bound used
is (8 + 4 sqrt(K)) 2^-24 sum|t|. The stored result is then rounded once: half a
step, finfo.eps / 2 relative, or half the smallest subnormal.
"""

import math

import pytest
import torch

from muon_newton_schulz_04_amd import binding as B
from muon_newton_schulz_04_amd import layers as L

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ACTS = list(L.ACTIVATIONS)


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _rand(g, shape, dtype, std=1.0, mean=0.0, stride=None):
    """A [rows, cols] GPU tensor with the given row stride; the gap between
    rows holds NaN, which no result may pick up."""
    r, c = shape
    v = (torch.randn(r, c, generator=g) * std + mean).to(dtype)
    buf = torch.full((r, stride or c), float("nan"), dtype=dtype)
    buf[:, :c] = v
    return buf.cuda()[:, :c]


def act64(name, z):
    if name == "relu":
        return z.clamp(min=0)
    if name == "relu2":
        return z.clamp(min=0) ** 2
    if name == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    if name == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def slope64(name, z):
    if name == "relu":
        return (z > 0).double()
    if name == "relu2":
        return 2 * z.clamp(min=0)
    if name == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        k = 2 * math.sqrt(2 / math.pi)
        q = torch.sigmoid(k * (z + 0.044715 * z ** 3))
        return q + z * q * (1 - q) * k * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        q = torch.sigmoid(z)
        return q + z * q * (1 - q)
    return torch.ones_like(z)


def _sum_tol(a, b):
    """Bound on a float32 product's error, from the float64 operands."""
    k = a.shape[1]
    return (8 + 4 * math.sqrt(k)) * 2.0 ** -24 * (a.abs() @ b.abs())


def _half_step(want, dtype):
    f = torch.finfo(dtype)
    return want.abs() * f.eps / 2 + f.smallest_normal * f.eps / 2


def _close(got, want, tol, dtype):
    got = got.double().cpu()
    assert got.shape == want.shape
    # a result `tol` off may round a further half step away
    lim = tol + _half_step(want.abs() + tol, dtype)
    bad = ~((got - want).abs() <= lim)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} off, worst {float((got - want).abs().max())}, "
                           f"first at {bad.nonzero()[0].tolist()}")


def _cpu64(t):
    return t.double().cpu()


# tokens, in, out: one element, one token, edges around the tiles (32, 128,
# 256) and chunks (8), odd sizes (packed operands), K shorter than a slice,
# long K with few outputs (split), more than one 256 tile
SIZES = [(1, 1, 1), (1, 64, 48), (1, 1600, 400), (3, 8, 8), (5, 7, 9), (33, 40, 136), (127, 100, 129), (64, 333, 257),
         (130, 1000, 264), (257, 96, 520), (300, 2048, 72), (17, 4104, 65), (600, 200, 640), (16, 1608, 96), (24, 6400, 200),
         (32, 72, 1601)]


@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_linear_sizes(size, dtype, layout):
    n, i, o = size
    t = T[dtype]
    g = _gen(n * 7 + i)
    x = _rand(g, (n, i), t)
    w = _rand(g, (i, o) if layout == "in_out" else (o, i), t, std=i ** -0.5)
    dy = _rand(g, (n, o), t, std=0.1)
    w64 = _cpu64(w) if layout == "in_out" else _cpu64(w).t()
    y = L.linear_forward(x, w, weight_layout=layout)
    _close(y, _cpu64(x) @ w64, _sum_tol(_cpu64(x), w64), t)
    dx = L.linear_grad_input(dy, w, weight_layout=layout)
    _close(dx, _cpu64(dy) @ w64.t(), _sum_tol(_cpu64(dy), w64.t()), t)
    dw, db = L.linear_grad_weight(x, dy, dbias=True, weight_layout=layout)
    a, b = (_cpu64(x).t(), _cpu64(dy)) if layout == "in_out" else (_cpu64(dy).t(), _cpu64(x))
    _close(dw, a @ b, _sum_tol(a, b), torch.float32)
    ones = torch.ones(1, n, dtype=torch.float64)
    _close(db, _cpu64(dy).sum(0), _sum_tol(ones, _cpu64(dy))[0], torch.float32)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("size", [(70, 72, 136), (9, 50, 33), (20, 3000, 64)], ids=str)
def test_linear_epilogues(size, act, dtype):
    """Bias, activation, residual and the kept pre-activation together, in one
    launch and over K splits, and the activation's slope on the way back."""
    n, i, o = size
    t = T[dtype]
    g = _gen(i)
    x, w = _rand(g, (n, i), t), _rand(g, (i, o), t, std=2 * i ** -0.5)
    bias = torch.randn(o, generator=g).cuda()
    res = _rand(g, (n, o), t)
    z64 = _cpu64(x) @ _cpu64(w) + bias.double().cpu()
    ztol = _sum_tol(_cpu64(x), _cpu64(w)) + 2.0 ** -23 * z64.abs()
    y, z = L.linear_forward(x, w, bias=bias, residual=res, activation=act, save_preact=True)
    _close(z, z64, ztol, t)
    # the activations' slopes are at most 2 |z| (relu2) or 1.2, and each takes
    # about ten float32 steps; the last addition one more
    want = act64(act, z64)
    slope = 2 * z64.abs() + 1.2 if act == "relu2" else 1.2
    tol = slope * ztol + 16 * 2.0 ** -24 * (z64.abs() + want.abs()) + 2.0 ** -24 * (want + _cpu64(res)).abs()
    _close(y, want + _cpu64(res), tol, t)
    dy = _rand(g, (n, o), t, std=0.1)
    pre, add = _rand(g, (n, i), t, std=2.0), _rand(g, (n, i), t, std=0.1)
    dx = L.linear_grad_input(dy, w, preact=pre, activation=act, add=add)
    raw, s64 = _cpu64(dy) @ _cpu64(w).t(), slope64(act, _cpu64(pre))
    want = raw * s64 + _cpu64(add)
    tol = _sum_tol(_cpu64(dy), _cpu64(w).t()) * s64.abs() + 2.0 ** -24 * (
        16 * (raw.abs() * (1 + _cpu64(pre).abs())) + want.abs())
    _close(dx, want, tol, t)


@pytest.mark.parametrize("rows,cols", [(0, 8), (1, 1), (1, 1600), (3, 7), (5, 512), (6, 513), (130, 1003), (9, 2048),
                                       (2, 2049), (11, 4100), (3, 8192), (70, 8200), (2, 20001)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_layernorm_sizes(rows, cols, dtype):
    t = T[dtype]
    g = _gen(rows + cols)
    x = _rand(g, (rows, cols), t, std=1.5, mean=2.0, stride=cols + (8 if cols % 3 else 5))
    w, b = torch.randn(cols, generator=g).cuda(), torch.randn(cols, generator=g).cuda()
    y, mean, rstd = L.layernorm_forward(x, w, b)
    x64 = _cpu64(x)
    m64 = x64.mean(1)
    r64 = 1 / (((x64 - m64[:, None]) ** 2).mean(1) + 1e-5).sqrt()
    u = 2.0 ** -24
    # a row's sum is taken in strands of at most 32 terms and 12 joins, each
    # one rounding of a partial sum of |x|; the variance likewise, relative
    mtol = 44 * u * x64.abs().mean(1) + u * m64.abs()
    _close(mean, m64, mtol, torch.float32)
    rtol = r64 * (60 * u + mtol * r64)
    _close(rstd, r64, rtol, torch.float32)
    xh = (x64 - m64[:, None]) * r64[:, None]
    w64, b64 = w.double().cpu(), b.double().cpu()
    xhtol = (mtol * r64)[:, None] + xh.abs() * (rtol / r64 + 4 * u)[:, None] + u * (x64.abs() * r64[:, None])
    _close(y, xh * w64 + b64, xhtol * w64.abs() + 2 * u * ((xh * w64).abs() + b64.abs()), t)

    dy = _rand(g, (rows, cols), t, std=0.1)
    add = _rand(g, (rows, cols), t, std=0.1)
    dx, dw, db = L.layernorm_backward(dy, x, mean, rstd, weight=w, add=add, dweight=True, dbias=True)
    # from the statistics that the forward pass stored, as the call has them
    m, r = mean.double().cpu()[:, None], rstd.double().cpu()[:, None]
    xh = (x64 - m) * r
    gg = _cpu64(dy) * w64
    s0, s1 = gg.mean(1, keepdim=True), (gg * xh).mean(1, keepdim=True)
    want = r * (gg - s0 - xh * s1) + _cpu64(add)
    xht = 3 * u * xh.abs() + u * x64.abs() * r
    t0 = 46 * u * gg.abs().mean(1, keepdim=True)
    t1 = 48 * u * (gg * xh).abs().mean(1, keepdim=True) + (gg.abs() * xht).mean(1, keepdim=True)
    tol = r * (4 * u * (gg.abs() + s0.abs() + (xh * s1).abs()) + t0 + xh.abs() * t1 + xht * s1.abs())
    _close(dx, want, tol + 2 * u * want.abs(), t)
    d64 = _cpu64(dy)
    n = (8 + 4 * math.sqrt(max(rows, 1))) * u
    _close(dw, (d64 * xh).sum(0), n * (d64 * xh).abs().sum(0) + (d64.abs() * xht).sum(0), torch.float32)
    _close(db, d64.sum(0), n * d64.abs().sum(0), torch.float32)
