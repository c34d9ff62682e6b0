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
