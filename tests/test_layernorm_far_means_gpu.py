"""Layer norm of rows whose mean is far from 0 against their spread, forward and
backward, against float64.

Tolerances. u = 2^-24, half a float32 step. A row's sum is taken in strands (a
lane's own elements in turn: up to 32, beyond 8192 columns 8 of every 2048) and
at most 14 joins of lanes and waves, so `terms` = strand + 14 roundings of
partial sums.
"""

import pytest
import torch

from muon_newton_schulz_04_amd import layers as L

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = 2.0 ** -24


def _terms(cols):
    return (32 if cols <= 8192 else -(-cols // 2048) * 8) + 14


def _within(got, want, tol, dtype):
    f = torch.finfo(dtype)
    lim = tol + (want.abs() + tol) * (f.eps / 2) + f.smallest_normal * f.eps / 2
    got = got.double().cpu()
    bad = ~((got - want).abs() <= lim)
    assert not bad.any(), (int(bad.sum()), float(((got - want).abs() / lim).max()), bad.nonzero()[0].tolist())


@pytest.mark.parametrize("cols", [1, 5, 8, 520, 1003, 1600, 2049, 8192, 9001])
@pytest.mark.parametrize("dtype,mean,std", [("bf16", 2.0 ** 100, 1e15), ("bf16", -1e30, 1e12), ("fp32", 1e25, 1e15)])
def test_backward_where_the_mean_over_the_spread_overflows(cols, dtype, mean, std):
    """Constant rows for which (0 - mean) rstd would overflow float32, though no
    element of the row is 0. What lies past a row's end (lanes without a chunk,
    the rest of a chunk) must not come in as such a 0."""
    t = T[dtype]
    g = torch.Generator().manual_seed(cols)
    c = torch.tensor(mean).to(t).double()
    x = torch.full((3, cols), c.item(), dtype=t)
    dy = (torch.randn(3, cols, generator=g) * 2.0 ** -60).to(t)
    w = torch.randn(cols, generator=g)
    m, r = torch.full((3,), c.item()), torch.full((3,), std)
    dx, dw, db = L.layernorm_backward(dy.cuda(), x.cuda(), m.cuda(), r.cuda(), weight=w.cuda(), dweight=True,
                                      dbias=True)
    gg = dy.double() * w.double()
    s0 = gg.mean(1, keepdim=True)
    r64 = r.double()[:, None]
    # xhat is 0 exactly: dx = rstd (g - mean(g)), the product, difference and
    # scaling one rounding each
    tol = r64 * (4 * U * (gg.abs() + s0.abs()) + _terms(cols) * U * gg.abs().mean(1, keepdim=True))
    _within(dx, r64 * (gg - s0), tol, t)
    assert (dw == 0).all()
    _within(db, dy.double().sum(0), 3 * U * dy.double().abs().sum(0), torch.float32)


@pytest.mark.parametrize("cols", [1, 7, 200, 1003, 1600, 2049, 8192, 9001, 20001])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_forward_of_nearly_constant_rows(cols, dtype):
    """Rows of one large value, and of a few neighbouring ones: what the float32
    mean is off by must not come out as a deviation."""
    t = T[dtype]
    g = torch.Generator().manual_seed(cols + 1)
    base = torch.tensor([1e5, 12345.678, -777.77, 3.3e4, 0.1, 1.0, 6e4, -4.1e4]).clamp(max=6e4 if dtype == "fp16" else 1e9)
    x = base[:, None].expand(-1, cols).to(t).clone()
    # in the last rows some elements a step or two of the type away
    step = x[4:, :1].double().abs() * torch.finfo(t).eps
    x[4:] = (x[4:].double() + step * torch.randint(-2, 3, (4, cols), generator=g).double()).to(t)
    w, b = torch.randn(cols, generator=g), torch.randn(cols, generator=g)
    y, mean, rstd = L.layernorm_forward(x.cuda(), w.cuda(), b.cuda(), eps=1e-5)
    x64 = x.double()
    m = x64.mean(1, keepdim=True)
    v = ((x64 - m) ** 2).mean(1, keepdim=True) + 1e-5
    n = _terms(cols)
    # the first mean is off by at most D; from there on deviations d count: their
    # mean, which corrects it, is off by er, and their mean square, less the
    # square of that correction, by ev
    D = (n + 2) * U * x64.abs().mean(1, keepdim=True)
    d = (x64 - m).abs() + D
    er = (n + 2) * U * d.mean(1, keepdim=True)
    ev = (n + 4) * U * (d * d).mean(1, keepdim=True) + 2 * D * er + 4 * U * D * D
    assert (ev < v).all()
    rel = (1 - ev / v) ** -0.5 - 1 + 4 * U
    r = v ** -0.5
    _within(mean, m[:, 0], er[:, 0] + U * m.abs()[:, 0], torch.float32)
    _within(rstd, r[:, 0], (r * rel)[:, 0], torch.float32)
    xh = (x64 - m) * r
    tol = (1 + rel) * r * (er + 3 * U * d) + xh.abs() * rel
    w64, b64 = w.double(), b.double()
    _within(y, xh * w64 + b64, tol * w64.abs() + 2 * U * ((xh * w64).abs() + b64.abs()), t)


@pytest.mark.parametrize("cols", [8, 200, 1003, 1600, 4100, 8192, 9001])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_rows_that_are_not_finite_stay_alone(cols, dtype):
    """A NaN or an infinity makes its row NaN (and an infinite row's mean
    infinite), forward and backward, and leaves the rows around it as they are."""
    t = T[dtype]
    g = torch.Generator().manual_seed(cols)
    x = (torch.randn(9, cols, generator=g) + 30).to(t)
    dy = torch.randn(9, cols, generator=g).to(t)
    ref = L.layernorm_forward(x.cuda())
    want = L.layernorm_backward(dy.cuda(), x.cuda(), *ref[1:])[0]
    bad, good = [1, 4, 5, 8], [0, 2, 3, 6, 7]
    x[1, 0], x[4, cols - 1], x[5, cols // 2], x[8, 3] = float("nan"), float("inf"), -float("inf"), float("nan")
    y, mean, rstd = L.layernorm_forward(x.cuda())
    for a, b in zip((y, mean, rstd), ref):
        assert torch.equal(a[good], b[good])
    assert y[bad].isnan().all() and rstd[bad].isnan().all()
    assert mean[4].item() == float("inf") and mean[5].item() == -float("inf") and mean[[1, 8]].isnan().all()
    dx = L.layernorm_backward(dy.cuda(), x.cuda(), mean, rstd)[0]
    assert torch.equal(dx[good], want[good]) and dx[bad].isnan().all()
