"""The 8-bit and the grouped products on every kind of tile: sizes that take it (checked
on the CPU against the plans), each against float64 with the epilogues that the kernels
fetch ahead. Tolerances are test_linear_fp8_gpu.py's and test_grouped_linear_gpu.py's.
"""

import pytest
import torch

from eight import U, act64, act_tol, close, cpu64, eight, gen, rand, slope64, sum_tol, values
from muon_newton_schulz_04_amd import layers as L

# rows, in, out: rows and columns end inside a tile, K inside a block of 128
EIGHT = [
    ("eight", 13, 1000, 200, "few 16"),
    ("eight", 31, 300, 333, "few 32"),
    ("eight", 70, 1500, 500, "few 32"),
    ("eight", 300, 400, 1001, "small"),
    ("eight", 301, 6401, 1003, "small groups"),
    ("eight", 2049, 1000, 1601, "square groups"),
    ("eight", 4097, 700, 1601, "square"),
    ("eight", 4000, 1601, 2090, "tall"),
]
# K past 64 blocks of 128 (the scales of so many are fetched at once) on each tile, and
# past the scales that the kernel for few rows holds
EIGHT += [
    ("eight", 3, 66001, 40, "few 16"),
    ("eight", 31, 33001, 40, "few 32"),
    ("eight", 1100, 8323, 1003, "small"),
    ("eight", 301, 16521, 1003, "small groups"),
    ("eight", 2049, 8323, 1601, "square groups"),
    ("eight", 4097, 8323, 1601, "square"),
    ("eight", 4000, 8323, 2090, "tall"),
]
# experts' rows, in, out, layout (0: [in, out])
GROUPED = [
    ("forward", [1, 0, 2], 1600, 72, 0, "few 16"),
    ("forward", [20, 41, 0, 30], 1608, 200, 1, "few 32"),
    ("forward", [60, 0, 90, 11], 96, 808, 0, "small"),
    ("forward", [60, 0, 90, 11], 1608, 808, 1, "small groups"),
    ("forward", [300, 0, 650, 50], 1608, 2056, 1, "square groups"),
    ("forward", [1500, 0, 2000, 600], 264, 1608, 0, "square"),
    ("forward", [3000, 41, 0, 5200], 264, 3208, 1, "tall"),
    ("grad input", [1, 0, 2], 72, 1600, 1, "few 16"),
    ("grad input", [20, 41, 0, 30], 200, 1608, 0, "few 32"),
    ("grad input", [60, 0, 90, 11], 808, 96, 1, "small"),
    ("grad input", [60, 0, 90, 11], 808, 1608, 0, "small groups"),
    ("grad input", [300, 0, 650, 50], 2056, 1608, 0, "square groups"),
    ("grad input", [1500, 0, 2000, 600], 1608, 264, 1, "square"),
    ("grad input", [3000, 41, 0, 5200], 3208, 264, 0, "tall"),
    ("grad weight", [60, 0, 90, 11], 200, 136, 0, "small"),
    ("grad weight", [60, 0, 90, 11], 136, 200, 1, "small"),
    ("grad weight", [9000, 0, 5000], 200, 136, 0, "small in 8"),
    ("grad weight", [9000, 77, 5000], 136, 200, 1, "small in 8"),
    ("grad weight", [1500] * 45 + [0, 7, 70] + [1500] * 30, 24, 16, 0, "small in 4"),
    ("grad weight", [18000, 6000], 1032, 520, 0, "square in 4"),
    ("grad weight", [18000, 6000], 520, 1032, 1, "square in 4"),
    ("grad weight", [0, 16000, 9000], 1544, 808, 0, "tall in 2"),
    ("grad weight", [0, 16000, 9000], 808, 1544, 1, "tall in 2"),
    ("grad weight", [500, 0, 90, 311], 808, 1032, 0, "square"),
    ("grad weight", [500, 0, 90, 311], 1032, 808, 1, "square"),
    ("grad weight", [1500, 0, 890, 3011, 700], 1608, 1544, 0, "tall"),
    ("grad weight", [1500, 0, 890, 3011, 700], 1544, 1608, 1, "tall"),
]
OPS = {"eight": 0, "forward": 1, "grad input": 2, "grad weight": 3}


def line_of(c):
    """The case for tests/native/scaled_plan.cpp."""
    if c[0] == "eight":
        return (0, c[1], c[2], c[3], 0, 0)
    op, counts, i, o, lay, _ = c
    return (OPS[op], sum(counts), len(counts), i, o, lay)


@pytest.mark.gpu
@pytest.mark.parametrize("case", EIGHT, ids=lambda c: f"{c[-1].replace(' ', '_')}-{c[1]}x{c[2]}x{c[3]}")
def test_eight(case):
    from test_linear_fp8_gpu import _near, _tol
    _, n, i, o, _ = case
    g = gen(n)
    t = torch.bfloat16
    x, w = eight(g, n, i), eight(g, o, i, std=i ** -0.5, weight=True)
    a, b = values(x), values(w, True).t()
    raw, tol = a @ b, _tol(a, b)
    y = L.linear_fp8_forward(x, w)
    close(y, raw, tol, t)
    _near(y, raw, t)
    bias, res = torch.randn(o, generator=g).cuda(), rand(g, (n, o), t, stride=o + 3)
    y, z = L.linear_fp8_forward(x, w, bias=bias, residual=res, activation="silu", save_preact=True)
    z64 = raw + cpu64(bias)
    ztol = tol + 2 * U * z64.abs()
    close(z, z64, ztol, t)
    want = act64("silu", z64) + cpu64(res)
    close(y, want, act_tol("silu", z64, ztol) + U * want.abs(), t)
    pre = rand(g, (n, o), t, std=2.0, stride=o + 1)
    dx = L.linear_fp8_grad_input(x, w, preact=pre, activation="gelu", add=res, dtype=t)
    s64 = slope64("gelu", cpu64(pre))
    want = raw * s64 + cpu64(res)
    close(dx, want, tol * s64.abs() + U * (16 * raw.abs() * (1 + cpu64(pre).abs()) + want.abs()), t)
    again = L.linear_fp8_grad_input(x, w, preact=pre, activation="gelu", add=res, dtype=t)
    assert torch.equal(again, dx)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", GROUPED, ids=lambda c: f"{c[0]}-{c[-1]}-{c[4]}".replace(" ", "_"))
def test_grouped(case, dtype):
    op, counts, i, o, lay, _ = case
    t = torch.bfloat16 if dtype == "bf16" else torch.float16
    g = gen(i + o)
    e, n = len(counts), sum(counts)
    at = [sum(counts[:k]) for k in range(e + 1)]
    off = torch.tensor(at, dtype=torch.int32).cuda()
    layout = ("in_out", "out_in")[lay]
    shape = (e, o, i) if lay else (e, i, o)
    w = (torch.randn(*shape, generator=g) * i ** -0.5).to(t).cuda()
    x, dy = rand(g, (n, i), t, stride=i + 8), rand(g, (n, o), t, std=0.1, stride=o + 16)
    rows = [slice(at[k], at[k + 1]) for k in range(e)]

    def weight(k):
        return cpu64(w[k]).t() if lay else cpu64(w[k])

    if op == "forward":
        bias, res = torch.randn(e, o, generator=g).cuda(), rand(g, (n, o), t)
        plain = L.grouped_linear_forward(x, w, off, weight_layout=layout)
        y, z = L.grouped_linear_forward(x, w, off, bias=bias, residual=res, activation="gelu_tanh",
                                        weight_layout=layout, save_preact=True)
        for k, r in enumerate(rows):
            a, b = cpu64(x[r]), weight(k)
            raw, tol = a @ b, sum_tol(a, b)
            close(plain[r], raw, tol, t)
            z64 = raw + cpu64(bias[k])
            ztol = tol + 2 * U * z64.abs()
            close(z[r], z64, ztol, t)
            want = act64("gelu_tanh", z64) + cpu64(res[r])
            close(y[r], want, act_tol("gelu_tanh", z64, ztol) + U * want.abs(), t)
    elif op == "grad input":
        pre, add = rand(g, (n, i), t, std=2.0), rand(g, (n, i), t, std=0.1)
        plain = L.grouped_linear_grad_input(dy, w, off, weight_layout=layout)
        dx = L.grouped_linear_grad_input(dy, w, off, preact=pre, activation="silu", add=add, weight_layout=layout)
        for k, r in enumerate(rows):
            a, b = cpu64(dy[r]), weight(k).t()
            raw, tol = a @ b, sum_tol(a, b)
            close(plain[r], raw, tol, t)
            s64 = slope64("silu", cpu64(pre[r]))
            want = raw * s64 + cpu64(add[r])
            close(dx[r], want, tol * s64.abs() + U * (16 * raw.abs() * (1 + cpu64(pre[r]).abs()) + want.abs()), t)
    else:
        dw, db = L.grouped_linear_grad_weight(x, dy, off, dbias=True, weight_layout=layout)
        bare, none = L.grouped_linear_grad_weight(x, dy, off, weight_layout=layout)
        assert none is None and torch.equal(bare, dw)
        for k, r in enumerate(rows):
            a, b = (cpu64(dy[r]).t(), cpu64(x[r])) if lay else (cpu64(x[r]).t(), cpu64(dy[r]))
            close(dw[k], a @ b, sum_tol(a, b), torch.float32)
            ones = torch.ones(1, counts[k], dtype=torch.float64)
            close(db[k], cpu64(dy[r]).sum(0), sum_tol(ones, cpu64(dy[r]))[0], torch.float32)
        dw2, db2 = L.grouped_linear_grad_weight(x, dy, off, dw=dw.clone(), dbias=db.clone(), accumulate=True,
                                                weight_layout=layout)
        assert torch.equal(dw2, dw + dw) and torch.equal(db2, db + db)
