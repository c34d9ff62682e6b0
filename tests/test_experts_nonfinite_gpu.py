"""Infinities and NaN in one expert's rows, weight, bias, residual and kept
pre-activation, and in rows of no expert: the other experts' results are the same bits
as without them, on every kind of tile, with whole rows and rows off 16-byte borders.
"""

import pytest
import torch

from eight import gen, rand
from muon_newton_schulz_04_amd import layers as L
from test_scaled_tiles_gpu import GROUPED

pytestmark = pytest.mark.gpu

# experts' rows, in, out, layout
ODD = [(op, counts, i, o, lay, "raw") for op in ("forward", "grad input", "grad weight") for lay in (0, 1)
       for counts, i, o in (([1, 0, 2], 9, 11), ([100, 0, 333, 77], 101, 203), ([9000, 77, 5000], 73, 137))]


def _poison(t, at):
    """A copy with infinities and NaN in the rows `at`."""
    v = t.clone()
    for r in at:
        v[r] = float("nan")
        v[r].view(-1, v.shape[-1])[:, ::3] = float("inf")
        v[r].view(-1, v.shape[-1])[:, 1::3] = float("-inf")
    return v


@pytest.mark.parametrize("case", GROUPED + ODD, ids=lambda c: f"{c[0]}-{c[-1]}-{c[4]}-{c[2]}".replace(" ", "_"))
def test_other_experts_are_untouched(case):
    op, counts, i, o, lay, _ = case
    t = torch.bfloat16
    g = gen(i + o)
    before, behind = 3, 5
    e, n = len(counts), sum(counts) + before + behind
    at = [before + sum(counts[:k]) for k in range(e + 1)]
    off = torch.tensor(at, dtype=torch.int32).cuda()
    layout = ("in_out", "out_in")[lay]
    shape = (e, o, i) if lay else (e, i, o)
    w = (torch.randn(*shape, generator=g) * i ** -0.5).to(t).cuda()
    x, dy = rand(g, (n, i), t), rand(g, (n, o), t, std=0.1)
    bias, res = torch.randn(e, o, generator=g).cuda(), rand(g, (n, o), t)
    pre, add = rand(g, (n, i), t, std=2.0), rand(g, (n, i), t, std=0.1)
    bad = next(k for k in range(e) if counts[k])  # with other experts' rows behind it
    lost = [slice(0, before), slice(at[bad], at[bad + 1]), slice(at[-1], n)]
    rows = torch.ones(n, dtype=torch.bool)
    for r in lost:
        rows[r] = False
    others = [k for k in range(e) if k != bad]
    rows, others = rows.cuda(), torch.tensor(others).cuda()
    assert rows.any()
    p = {k: _poison(v, lost) for k, v in (("x", x), ("dy", dy), ("res", res), ("pre", pre), ("add", add))}
    pw, pb = _poison(w, [slice(bad, bad + 1)]), _poison(bias, [slice(bad, bad + 1)])
    if op == "forward":
        kw = dict(activation="gelu", weight_layout=layout, save_preact=True)
        want = L.grouped_linear_forward(x, w, off, bias=bias, residual=res, **kw)
        got = L.grouped_linear_forward(p["x"], pw, off, bias=pb, residual=p["res"], **kw)
        for a, b in zip(got, want):
            assert torch.equal(a[rows], b[rows]) and b[rows].isfinite().all()
            assert not a[lost[1]].isfinite().any()
    elif op == "grad input":
        kw = dict(activation="silu", weight_layout=layout)
        want = L.grouped_linear_grad_input(dy, w, off, preact=pre, add=add, **kw)
        got = L.grouped_linear_grad_input(p["dy"], pw, off, preact=p["pre"], add=p["add"], **kw)
        assert torch.equal(got[rows], want[rows]) and want[rows].isfinite().all()
        assert not got[lost[1]].isfinite().any()
    else:
        want = L.grouped_linear_grad_weight(x, dy, off, dbias=True, weight_layout=layout)
        got = L.grouped_linear_grad_weight(p["x"], p["dy"], off, dbias=True, weight_layout=layout)
        for a, b in zip(got, want):
            assert torch.equal(a[others], b[others]) and b.isfinite().all()
            assert not a[bad].isfinite().any()
