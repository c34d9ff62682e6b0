"""The experts' operators on features and strides off 16-byte borders at sizes of many
tiles, against float64. Tolerances are test_grouped_linear_gpu.py's.
"""

import pytest
import torch

from eight import T, U, act64, act_tol, close, cpu64, gen, rand, sum_tol
from muon_newton_schulz_04_amd import layers as L

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("i,o", [(1601, 1003), (1000, 1601), (1601, 1000)])
def test_many_tiles(i, o, layout, dtype):
    counts, t = [1500, 0, 1, 900, 63, 65, 1570], T[dtype]
    g = gen(i + o)
    e, n = len(counts), sum(counts)
    at = [sum(counts[:k]) for k in range(e + 1)]
    off = torch.tensor(at, dtype=torch.int32).cuda()
    w = (torch.randn(e, *((i, o) if layout == "in_out" else (o, i)), generator=g) * i ** -0.5).to(t).cuda()
    x, dy = rand(g, (n, i), t, stride=i + 2), rand(g, (n, o), t, std=0.1)
    bias = torch.randn(e, o, generator=g).cuda()
    y = L.grouped_linear_forward(x, w, off, bias=bias, activation="gelu", weight_layout=layout)
    dx = L.grouped_linear_grad_input(dy, w, off, weight_layout=layout)
    dw, db = L.grouped_linear_grad_weight(x, dy, off, dbias=True, weight_layout=layout)
    for k in range(e):
        r = slice(at[k], at[k + 1])
        w64 = cpu64(w[k]) if layout == "in_out" else cpu64(w[k]).t()
        x64, d64 = cpu64(x[r]), cpu64(dy[r])
        z64 = x64 @ w64 + cpu64(bias[k])
        ztol = sum_tol(x64, w64) + 2 * U * z64.abs()
        close(y[r], act64("gelu", z64), act_tol("gelu", z64, ztol), t)
        close(dx[r], d64 @ w64.t(), sum_tol(d64, w64.t()), t)
        a, b = (x64.t(), d64) if layout == "in_out" else (d64.t(), x64)
        close(dw[k], a @ b, sum_tol(a, b), torch.float32)
        ones = torch.ones(1, counts[k], dtype=torch.float64)
        close(db[k], d64.sum(0), sum_tol(ones, d64)[0], torch.float32)
