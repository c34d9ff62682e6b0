"""Root-mean-square norm with the residual's addition and an 8-bit output, its
backward pass, and the quantisation of matrices to 8 bits, on the GPU against
float64.

Tolerances, u = 2^-24. A row's squares are summed in strands of at most 32 terms
and 12 joins (for rows in registers; a longer row's strands are cols / 256 terms),
each an fma or an addition of positive terms: relative error at most (32 + 12) u,
half of it in rstd, whose root, division and mean take 3 u more. y takes two
roundings more before its own. An 8-bit value is off by half a step of its format
from y / scale, where scale is y's largest magnitude's error and one division off.
"""

import pytest
import torch

from eight import (F8, LARGEST, SMALLEST, T, U, amax64, blocks, close, cpu64, gen, half_step8, nearest8, rand, spread)
from muon_newton_schulz_04_amd import layers as L

pytestmark = pytest.mark.gpu

SIZES = [(0, 8), (1, 1), (1, 1600), (3, 7), (5, 512), (6, 513), (130, 1003), (9, 2048), (2, 2049), (11, 4100), (3, 8192),
         (70, 8200), (2, 20001), (17, 16), (8, 128), (4, 129), (5, 1000)]


def _strand(cols):
    return 44 if cols <= 8192 else cols / 256 + 12


def _check_eight(pair, want, tol, fmt):
    """An 8-bit output against float64 values that it may have seen `tol` off."""
    q, s = pair
    rows, cols = want.shape
    assert q.shape == want.shape and s.shape == (blocks(cols), rows) and q.stride(0) % 16 == 0
    top = amax64(want, 1)
    s64 = cpu64(s).t()
    s_want = top.clamp(min=SMALLEST) / LARGEST[fmt]
    worst = amax64(tol, 1) / LARGEST[fmt]
    assert ((s64 - s_want).abs() <= worst + U * s_want).all()
    v = want / spread(s64, 1, rows, cols)
    # the quotient's own error: tol, and three roundings (the reciprocal, twice, and the product)
    off = tol / spread(s64, 1, rows, cols) + 3 * U * v.abs()
    q64 = cpu64(q.float())
    assert ((q64 - v).abs() <= off + half_step8(v.abs() + off, fmt)).all()
    # the bytes up to the next multiple of 16 are zeros
    pad = q.stride(0) - cols if rows > 1 else 0
    if pad:
        b = torch.as_strided(q.view(torch.uint8), (rows, cols + pad), (q.stride(0), 1))
        assert not b[:, cols:(cols + 15) // 16 * 16].any()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_rmsnorm_sizes(rows, cols, dtype):
    t = T[dtype]
    g = gen(rows * 3 + cols)
    x = rand(g, (rows, cols), t, std=1.5, mean=0.5, stride=cols + (8 if cols % 3 else 5))
    res = rand(g, (rows, cols), t, std=2.0, stride=cols + 3)
    w = torch.randn(cols, generator=g).cuda()
    w64 = cpu64(w)

    def want_of(r):
        r64 = cpu64(r)
        rs = 1 / ((r64 ** 2).mean(1) + 1e-5).sqrt()
        rt = (_strand(cols) / 2 + 4) * U
        y = r64 * rs[:, None] * w64
        return rs, rt, y, (rt + 2 * U) * y.abs()

    # plain, no residual
    y, rstd = L.rmsnorm_forward(x, w)
    rs, rt, want, tol = want_of(x)
    close(rstd, rs, rt * rs, torch.float32)
    close(y, want, tol, t)
    # the residual first: the sum is rounded once, and the norm is of what is stored
    fmt = "e5m2" if cols % 2 else "e4m3"
    out = torch.empty(rows, cols, dtype=t, device="cuda")
    q, rstd2, r = L.rmsnorm_forward(x, w, residual=res, quantize=F8[fmt], out=out)
    if dtype == "fp32":
        assert torch.equal(r, x + res)
    else:
        assert torch.equal(r.cpu(), (x.float() + res.float()).to(t).cpu())
    rs, rt, want, tol = want_of(r)
    close(rstd2, rs, rt * rs, torch.float32)
    close(out, want, tol, t)
    _check_eight(q, want, tol, fmt)
    # 8 bits alone gives the same bits, and so does the sum in the residual's place
    other = res.clone()
    q2, _, r2 = L.rmsnorm_forward(x, w, residual=other, quantize=F8[fmt], residual_out=other)
    assert r2 is other and torch.equal(other, r)
    assert torch.equal(q2.data.view(torch.uint8), q.data.view(torch.uint8)) and torch.equal(q2.scale, q.scale)

    dy = rand(g, (rows, cols), t, std=0.1, stride=cols + 1)
    add = rand(g, (rows, cols), t, std=0.1)
    dx, dw = L.rmsnorm_backward(dy, r, rstd2, weight=w, add=add, dweight=True)
    xh = cpu64(r) * cpu64(rstd2)[:, None]
    gg = cpu64(dy) * w64
    s = (gg * xh).mean(1, keepdim=True)
    want = cpu64(rstd2)[:, None] * (gg - xh * s) + cpu64(add)
    # the sum's strands as above, on terms with three roundings of their own; then the terms' own
    st = (_strand(cols) + 4) * U * (gg * xh).abs().mean(1, keepdim=True)
    tol = cpu64(rstd2)[:, None] * (4 * U * (gg.abs() + (xh * s).abs()) + xh.abs() * st) + 2 * U * want.abs()
    close(dx, want, tol, t)
    # rows in any order, each term with two roundings
    d = cpu64(dy) * xh
    close(dw, d.sum(0), (10 + 4 * max(rows, 1) ** 0.5) * U * d.abs().sum(0), torch.float32)
    # without weight and add, accumulated, over the add
    dx2, none = L.rmsnorm_backward(dy, r, rstd2)
    assert none is None
    g1 = cpu64(dy)
    s = (g1 * xh).mean(1, keepdim=True)
    want = cpu64(rstd2)[:, None] * (g1 - xh * s)
    st = (_strand(cols) + 4) * U * (g1 * xh).abs().mean(1, keepdim=True)
    close(dx2, want, cpu64(rstd2)[:, None] * (4 * U * (g1.abs() + (xh * s).abs()) + xh.abs() * st), t)
    acc = dw.clone()
    over = add.clone()
    dx3, _ = L.rmsnorm_backward(dy, r, rstd2, weight=w, add=over, dweight=acc, accumulate=True, out=over)
    assert dx3 is over and torch.equal(over, dx) and torch.equal(acc, dw + dw)


def test_rmsnorm_gradient_against_differences():
    """The gradient against central differences of the float64 definition."""
    g = gen(5)
    x, dy = rand(g, (4, 24), torch.float32), rand(g, (4, 24), torch.float32)
    w = torch.randn(24, generator=g).cuda()
    _, rstd = L.rmsnorm_forward(x, w)
    dx, dw = L.rmsnorm_backward(dy, x, rstd, weight=w, dweight=True)

    def loss(a, b):
        return (a / ((a ** 2).mean(1, keepdim=True) + 1e-5).sqrt() * b * cpu64(dy)).sum()

    h = 1e-5
    for got, at in ((dx, 0), (dw, 1)):
        args = [cpu64(x), cpu64(w)]
        want = torch.zeros_like(args[at])
        flat = args[at].view(-1)
        for k in range(flat.numel()):
            old = float(flat[k])
            flat[k] = old + h
            up = loss(*args)
            flat[k] = old - h
            want.view(-1)[k] = (up - loss(*args)) / (2 * h)
            flat[k] = old
        # differences are off by h^2 times the third derivative and 2^-53 / h
        assert (cpu64(got) - want).abs().max() < 1e-5 * (1 + want.abs().max())


def test_rmsnorm_special_rows():
    """Rows of zeros, tiny and huge values, infinities and NaN: each stays in its
    row, and in 8 bits in its block."""
    x = torch.zeros(8, 300, device="cuda")
    x[1] = 1e-30
    x[2] = 1e15
    x[3, 5] = float("inf")
    x[4, 200] = float("nan")
    x[5] = torch.arange(300, device="cuda") - 150.0
    x[6] = 1e25  # squares overflow
    x[7, 299] = -3.0
    q, rstd, = L.rmsnorm_forward(x, quantize=torch.float8_e4m3fn)
    y, rstd2 = L.rmsnorm_forward(x)
    assert torch.equal(rstd.nan_to_num(-1), rstd2.nan_to_num(-1))
    assert not y[0].any() and not q.data.float()[0].any() and (q.scale[:, 0] > 0).all()
    assert torch.allclose(y[1], torch.full((300,), 1e-30 / 1e-5 ** 0.5, device="cuda"), rtol=1e-6)
    assert torch.allclose(y[2], torch.ones(300, device="cuda"), rtol=1e-6)
    assert (y[3] == 0)[:5].all() and y[3, 5].isnan()
    assert y[4].isnan().all()
    assert not y[6].any()
    v = q.data.float() * q.scale.t().repeat_interleave(128, 1)[:, :300]
    # the row of an infinity: its own block stands for nothing, the others for zeros
    assert v[3, :128].isnan().all() and not v[3, 128:].any()
    assert v[4].isnan().all()
    assert torch.allclose(v[5], y[5], rtol=2.0 ** -4, atol=float(y[5].abs().max()) * 2.0 ** -10 / 448)
    assert v[7, 299] == y[7, 299].clamp(-448, 448) or abs(v[7, 299] / y[7, 299] - 1) <= 2.0 ** -4
    # the way back: rows keep to themselves
    dx, dw = L.rmsnorm_backward(torch.ones_like(x), x, rstd2, dweight=True)
    good = [0, 1, 2, 5, 7]
    assert dx[good].isfinite().all() and dx[4].isnan().all()
    assert dw.isnan().any()  # a weight's gradient sums all rows


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(0, 8), (1, 1), (1, 127), (3, 128), (5, 129), (2, 511), (7, 513), (130, 1003),
                                       (9, 6400), (2051, 40)])
def test_quantize_rows(rows, cols, dtype, fmt):
    t = T[dtype]
    g = gen(rows + cols)
    x = rand(g, (rows, cols), t, std=0.01, stride=cols + 5)
    if rows > 2:
        x[1] = 0
        x[2, ::3] = 1.0  # exact ratios: ties
        x[2, 1::3] = -17 / 256
    q, s = L.quantize_fp8(x, dtype=F8[fmt])
    x64 = cpu64(x)
    want_s = (amax64(x64, 1).clamp(min=SMALLEST)).float() / LARGEST[fmt]
    assert torch.equal(s.cpu(), want_s.t().contiguous())  # one correctly rounded division
    v = x64 * LARGEST[fmt] / spread(amax64(x64, 1).clamp(min=SMALLEST), 1, rows, cols)
    got = cpu64(q.float())
    if dtype == "fp32":
        # 7/8 of a float32 value is itself rounded
        assert ((got - v).abs() <= 2 * U * v.abs() + half_step8(v.abs() * (1 + 2 * U), fmt)).all()
    else:
        # the quotient of two 16-bit values that is no border between 8-bit values is further from one than
        # its float32 rounding, so rounding it twice is rounding it once
        assert torch.equal(got, nearest8(v, fmt))


@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("fin,fout", [(1, 1), (128, 128), (127, 130), (300, 77), (16, 1000), (257, 640)])
def test_quantize_weight(fin, fout, dtype, layout):
    t = T[dtype]
    g = gen(fin + fout)
    shape = (fin, fout) if layout == "in_out" else (fout, fin)
    w = rand(g, shape, t, std=0.05, stride=shape[1] + 3)
    w8, w8_t = L.quantize_fp8_weight(w, weight_layout=layout, transpose=True)
    w64 = cpu64(w).t().contiguous() if layout == "in_out" else cpu64(w)
    top = amax64(w64, 128).clamp(min=SMALLEST)
    assert torch.equal(w8.scale.cpu(), top.float() / 448)
    assert torch.equal(w8_t.scale, w8.scale.t())
    v = w64 * 448 / spread(top, 128, fout, fin)
    got = cpu64(w8.data.float())
    if dtype == "fp32":
        assert ((got - v).abs() <= 2 * U * v.abs() + half_step8(v.abs() * (1 + 2 * U), "e4m3")).all()
    else:
        assert torch.equal(got, nearest8(v, "e4m3"))
    assert torch.equal(w8_t.data.view(torch.uint8), w8.data.view(torch.uint8).t())
    one, none = L.quantize_fp8_weight(w, weight_layout=layout)
    assert none is None and torch.equal(one.data.view(torch.uint8), w8.data.view(torch.uint8))
    for q, n in ((w8.data, fin), (w8_t.data, fout)):
        if q.shape[0] > 1 and q.stride(0) > n:
            b = torch.as_strided(q.view(torch.uint8), (q.shape[0], q.stride(0)), (q.stride(0), 1))
            assert not b[:, n:(n + 15) // 16 * 16].any()


def test_quantize_nothing_and_everything():
    """Blocks of zeros, of the smallest numbers, and with infinities and NaN."""
    x = torch.zeros(6, 256, device="cuda")
    x[1, :128] = 1e-42
    x[2, 3] = float("inf")
    x[3, 130] = float("nan")
    x[4] = 3.4e38
    x[5, 0] = 2.0 ** -109
    q, s = L.quantize_fp8(x)
    v = q.float() * s.t().repeat_interleave(128, 1)
    assert (s[:, 0] == torch.tensor(SMALLEST).div(448).item()).all() and not v[0].any() and not v[1].any()
    assert v[2, :128].isnan().all() and not v[2, 128:].any()
    assert v[3, 128:].isnan().all() and not v[3, :128].any()
    assert torch.allclose(v[4], x[4], rtol=2.0 ** -4) and v[5, 0] > 0
    w8, _ = L.quantize_fp8_weight(x.t().contiguous(), weight_layout="out_in")
    assert w8.scale[1, 0].isnan() and w8.scale[0, 0].isinf()
