"""The linear layers of a mixture of experts on the GPU against float64 products of
each expert's rows. Tolerances are the linear layer's: float32 sums of K terms within
(8 + 4 sqrt(K)) 2^-24 sum|t|, then the epilogue's roundings and one to the output's
type.
"""

import pytest
import torch

from eight import T, U, act64, act_tol, close, cpu64, gen, rand, slope64, sum_tol
from muon_newton_schulz_04_amd import binding as B
from muon_newton_schulz_04_amd import layers as L

pytestmark = pytest.mark.gpu


def _weights(g, n, shape, dtype, std, pad=0, gap=0):
    """[n, *shape] weights with gaps of NaN between rows and experts."""
    r, c = shape
    step = r * (c + pad) + gap
    buf = torch.full((n * step,), float("nan"), dtype=dtype)
    v = torch.as_strided(buf, (n, r, c), (step, c + pad, 1))
    v.copy_((torch.randn(n, r, c, generator=g) * std).to(dtype))
    return torch.as_strided(buf.cuda(), (n, r, c), (step, c + pad, 1))


def _offsets(counts, first=0):
    o = [first]
    for c in counts:
        o.append(o[-1] + c)
    return torch.tensor(o, dtype=torch.int32).cuda(), o


# rows of each expert (empty ones among them), rows before the first and behind the
# last one, in, out: single tokens, few rows (blocks of 16 and 32), each tile, more
# than 64 experts, odd sizes and strides (operands through registers)
CASES = [
    ([1], 0, 0, 8, 8),
    ([0, 0, 0], 0, 5, 16, 24),
    ([1, 0, 0, 1], 0, 0, 1600, 640),
    ([3, 0, 9, 2, 0], 2, 3, 104, 72),
    ([0, 17, 5, 0, 30, 1], 0, 7, 256, 136),
    ([20] * 3 + [1] * 90, 0, 0, 72, 48),
    ([65, 0, 190, 33], 1, 2, 96, 200),
    ([300, 2, 0, 511], 0, 40, 136, 264),
    ([1500, 900, 40, 2100], 0, 0, 264, 2056),
    ([5000, 0, 6700, 300], 3, 100, 72, 1544),
    ([1] * 130 + [700], 0, 0, 64, 72),
    ([9, 0, 4], 0, 0, 9, 11),
    ([100, 0, 333, 77], 2, 1, 101, 203),
]
_ids = [f"{len(c[0])}x{sum(c[0])}-{c[3]}-{c[4]}" for c in CASES]


@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", CASES, ids=_ids)
def test_sizes(case, dtype, layout):
    counts, before, behind, i, o = case
    t = T[dtype]
    g = gen(i + o + sum(counts))
    e, n = len(counts), before + sum(counts) + behind
    off, at = _offsets(counts, before)
    odd = i % 8 != 0
    w = _weights(g, e, (i, o) if layout == "in_out" else (o, i), t, i ** -0.5, pad=3 if odd else 8, gap=1 if odd else 16)
    x = rand(g, (n, i), t, stride=i + (5 if odd else 8))
    dy = rand(g, (n, o), t, std=0.1, stride=o + (1 if odd else 8))
    mark = torch.randn(n, max(i, o), generator=g).to(t).cuda()
    out = mark[:, :o].clone()
    y = L.grouped_linear_forward(x, w, off, weight_layout=layout, out=out)
    dx = L.grouped_linear_grad_input(dy, w, off, weight_layout=layout, out=mark[:, :i].clone())
    dw, db = L.grouped_linear_grad_weight(x, dy, off, dbias=True, weight_layout=layout)
    assert y is out
    for k in range(e):
        r = slice(at[k], at[k + 1])
        w64 = cpu64(w[k]) if layout == "in_out" else cpu64(w[k]).t()
        x64, d64 = cpu64(x[r]), cpu64(dy[r])
        close(y[r], x64 @ w64, sum_tol(x64, w64), t)
        close(dx[r], d64 @ w64.t(), sum_tol(d64, w64.t()), t)
        a, b = (x64.t(), d64) if layout == "in_out" else (d64.t(), x64)
        close(dw[k], a @ b, sum_tol(a, b), torch.float32)
        ones = torch.ones(1, at[k + 1] - at[k], dtype=torch.float64)
        close(db[k], d64.sum(0), sum_tol(ones, d64)[0], torch.float32)
    # rows of no expert are as they were
    for got, width in ((y, o), (dx, i)):
        assert torch.equal(got[:before], mark[:before, :width]) and torch.equal(got[at[-1]:], mark[at[-1]:, :width])
    # accumulated: one more addition
    dw2, db2 = L.grouped_linear_grad_weight(x, dy, off, dw=dw.clone(), dbias=db.clone(), accumulate=True,
                                            weight_layout=layout)
    assert torch.equal(dw2, dw + dw) and torch.equal(db2, db + db)


@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("act", list(L.ACTIVATIONS))
@pytest.mark.parametrize("counts,i,o", [([3, 0, 8], 72, 136), ([70, 0, 200, 5], 64, 264), ([9, 40], 25, 33),
                                        ([900, 1200, 0, 300], 136, 1544)], ids=str)
def test_epilogues(counts, i, o, act, layout):
    t = torch.bfloat16
    g = gen(i + o)
    e, n = len(counts), sum(counts) + 3
    off, at = _offsets(counts, 1)
    shape = (i, o) if layout == "in_out" else (o, i)
    x, w = rand(g, (n, i), t), _weights(g, e, shape, t, 2 * i ** -0.5)
    bias = torch.randn(e, o, generator=g).cuda()
    res = rand(g, (n, o), t, stride=o + 3)
    y, z = L.grouped_linear_forward(x, w, off, bias=bias, residual=res, activation=act, weight_layout=layout,
                                    save_preact=True)
    dy = rand(g, (n, o), t, std=0.1)
    pre, add = rand(g, (n, i), t, std=2.0), rand(g, (n, i), t, std=0.1)
    dx = L.grouped_linear_grad_input(dy, w, off, preact=pre, activation=act, add=add, weight_layout=layout)
    for k in range(e):
        r = slice(at[k], at[k + 1])
        x64, w64 = cpu64(x[r]), cpu64(w[k]) if layout == "in_out" else cpu64(w[k]).t()
        z64 = x64 @ w64 + cpu64(bias[k])
        ztol = sum_tol(x64, w64) + 2 * U * z64.abs()
        close(z[r], z64, ztol, t)
        want = act64(act, z64) + cpu64(res[r])
        close(y[r], want, act_tol(act, z64, ztol) + U * want.abs(), t)
        d64, s64 = cpu64(dy[r]), slope64(act, cpu64(pre[r]))
        raw = d64 @ w64.t()
        want = raw * s64 + cpu64(add[r])
        tol = sum_tol(d64, w64.t()) * s64.abs() + U * (16 * raw.abs() * (1 + cpu64(pre[r]).abs()) + want.abs())
        close(dx[r], want, tol, t)


def test_offsets_of_any_value_stay_inside():
    """Offsets that go beyond the rows, below 0 or down: nothing outside the tensors is
    written, and experts whose rows are in order have their products."""
    g = gen(2)
    t = torch.bfloat16
    n, i, o, e = 40, 64, 72, 5
    x, dy = rand(g, (n, i), t), rand(g, (n, o), t)
    w = _weights(g, e, (i, o), t, 0.1)
    for values in ([0, 10, 20, 30, 40, 1000], [-50, 10, 20, 30, 40, 40], [0, 10, 5, 30, 40, 40],
                   [2 ** 31 - 1, -2 ** 31, 7, 3, 2 ** 31 - 1, 0]):
        off = torch.tensor(values, dtype=torch.int32).cuda()
        buf = torch.full((n + 16, o), 7.0, dtype=t, device="cuda")
        y = L.grouped_linear_forward(x, w, off, out=buf[8:8 + n])
        assert (buf[:8] == 7).all() and (buf[8 + n:] == 7).all()
        dbuf = torch.full((e + 2, i, o), 7.0, device="cuda")
        L.grouped_linear_grad_weight(x, dy, off, dw=dbuf[1:-1])
        assert (dbuf[0] == 7).all() and (dbuf[-1] == 7).all()
        L.grouped_linear_grad_input(dy, w, off)
        if values[1:5] == [10, 20, 30, 40]:
            a, b = cpu64(x[10:20]), cpu64(w[1])
            close(y[10:20], a @ b, sum_tol(a, b), t)


def test_offsets_that_repeat_all_rows():
    """Every other of 65536 experts claims all 2^20 rows: blocks of 16 rows for them
    number 2^31, more than 32 bits hold, and the grid has workgroups for 2^17. Nothing
    beside the tensors is written, and the call ends."""
    t = torch.bfloat16
    e, n, i, o = 65536, 1 << 20, 8, 8
    off = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
    off[1::2] = n
    x = torch.ones(n, i, dtype=t, device="cuda")
    w = torch.ones(e, i, o, dtype=t, device="cuda")
    buf = torch.full((n + 16, o), 7.0, dtype=t, device="cuda")
    L.grouped_linear_forward(x, w, off, out=buf[8:8 + n])
    assert (buf[:8] == 7).all() and (buf[8 + n:] == 7).all()
    assert ((buf[8:8 + n] == 8) | (buf[8:8 + n] == 7)).all() and (buf[8] == 8).all()


@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("at", [0, 1])
def test_pieces_of_many_rows(at, layout):
    """Few experts of few features whose rows are summed in pieces: the C call on a
    workspace full of NaN with guard bytes behind it, rows 16-byte aligned or not, experts
    with fewer slices of rows than pieces or none, a gradient with gaps, adding to it."""
    g = gen(at)
    t, i, o = torch.bfloat16, 72, 136
    counts = [9001, 0, 100, 3000]
    n, e = 12200, len(counts)  # 99 rows behind the last expert's
    x, dy = rand(g, (n, i + 8), t)[:, at:at + i], rand(g, (n, o + 8), t, std=0.1)[:, at:at + o]
    off = torch.tensor([0] + counts).cumsum(0).int().cuda()
    r, c = (i, o) if layout == "in_out" else (o, i)
    lay = B.MUON_WEIGHT_IN_OUT if layout == "in_out" else B.MUON_WEIGHT_OUT_IN
    step = (r + 1) * (c + 5)
    d = B.muon_grouped(n, e, i, o, i + 8, c + 5, o + 8, step, 0, lay)
    s, need = B.muon_grouped_linear_workspace_bytes(d, x.data_ptr(), dy.data_ptr())
    assert s == 0 and need >= 2 * e * r * c * 4
    want, dbias = [], []
    for k in range(e):
        rows = slice(int(off[k]), int(off[k + 1]))
        a, b = (cpu64(x[rows]).t(), cpu64(dy[rows])) if layout == "in_out" else (cpu64(dy[rows]).t(), cpu64(x[rows]))
        want.append((a @ b, sum_tol(a, b)))
        ones = torch.ones(1, counts[k], dtype=torch.float64)
        dbias.append((cpu64(dy[rows]).sum(0), sum_tol(ones, cpu64(dy[rows]))[0]))
    results = []
    for accumulate in (0, 1):
        buf = torch.full((e * step,), 3.0, device="cuda")
        db = torch.full((e * o,), 5.0, device="cuda")
        ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
        assert ws.data_ptr() % 256 == 0
        s = B.muon_grouped_linear_grad_weight(d, x.data_ptr(), dy.data_ptr(), off.data_ptr(), buf.data_ptr(),
                                              db.data_ptr(), accumulate, ws.data_ptr(), need,
                                              torch.cuda.current_stream().cuda_stream)
        assert s == 0, B.muon_op_last_error()
        assert (ws[need:] == 0xFF).all()
        full = buf.view(e, r + 1, c + 5)
        assert (full[:, r] == 3).all() and (full[:, :, c:] == 3).all()
        for k in range(e):
            more = accumulate * U * (want[k][0].abs() + 3)
            close(full[k, :r, :c], want[k][0] + 3 * accumulate, want[k][1] + more, torch.float32)
            more = accumulate * U * (dbias[k][0].abs() + 5)
            close(db[k * o:k * o + o], dbias[k][0] + 5 * accumulate, dbias[k][1] + more, torch.float32)
        results.append((full.clone(), db.clone()))
    dw, db = L.grouped_linear_grad_weight(x, dy, off, dbias=True, weight_layout=layout)
    assert torch.equal(dw, results[0][0][:, :r, :c]) and torch.equal(db.flatten(), results[0][1])


def test_no_rows():
    w = torch.zeros(3, 16, 24, dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    x, dy = w.new_zeros(0, 16), w.new_zeros(0, 24)
    assert L.grouped_linear_forward(x, w, off).shape == (0, 24)
    assert L.grouped_linear_grad_input(dy, w, off).shape == (0, 16)
    dw, db = L.grouped_linear_grad_weight(x, dy, off, dbias=True)
    assert not dw.any() and not db.any() and dw.shape == (3, 16, 24)
    keep = torch.ones(3, 16, 24, device="cuda")
    L.grouped_linear_grad_weight(x, dy, off, dw=keep, accumulate=True)
    assert (keep == 1).all()


def test_refusals():
    x = torch.zeros(12, 16, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(3, 16, 24, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, 4, 8, 12], dtype=torch.int32, device="cuda")
    for args, kw, what in [
        ((x, w, off.long()), {}, "offsets: dtype"),
        ((x, w, off.cpu()), {}, "offsets: on"),
        ((x, w, off[:3]), {}, "offsets: shape"),
        ((x, w, off.repeat(2)[::2]), {}, "contiguous"),
        ((x, w[0], off), {}, "w: shape"),
        ((x, w.half(), off), {}, "w: dtype"),
        ((x, w.transpose(1, 2), off), {"weight_layout": "out_in"}, "contiguous"),
        ((x[:, :8], w, off), {}, "x: shape"),
        ((x, w, off), {"bias": torch.zeros(24, device="cuda")}, "bias: shape"),
        ((x, w, off), {"activation": "swish"}, "activation"),
    ]:
        with pytest.raises(ValueError, match=what):
            L.grouped_linear_forward(*args, **kw)
    with pytest.raises(ValueError, match="accumulate"):
        L.grouped_linear_grad_weight(x, x, off, accumulate=True)
    with pytest.raises(Exception, match="features"):
        L.grouped_linear_forward(x[:, :4], w[:, :4], off)
    with pytest.raises(Exception, match="overlaps"):
        L.grouped_linear_forward(x, torch.zeros(3, 16, 16, dtype=x.dtype, device="cuda"), off, out=x)
