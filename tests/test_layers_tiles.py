"""The linear layer's kernel for each tile and each way a product is cut, over
all three products. On the CPU: the sizes below take the tile and the cut that
they stand for, so that another choice of plan cannot leave a kernel untested.
On the GPU: each against float64, every element, with the epilogues that the
kernels fetch ahead.

Tolerances are test_layers_gpu.py's: float32 sums of K terms within
(8 + 4 sqrt(K)) 2^-24 sum|t|, then one rounding to the output's type.
"""

import math
import os
import subprocess

import pytest
import torch

from muon_newton_schulz_04_amd import layers as L
from test_abi_sanitize import CSRC, NATIVE, ROCM, ROOT, _have_toolchain

FWD, GI, GW = 0, 1, 2
T = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = 2.0 ** -24

# operation, tokens, in, out: rows of the tile, the cut (whole tiles, all of them
# in K pieces, or whole ones with pieces beside them; 8 pieces or more are added
# by four lanes a chunk), operands copied to aligned rows first. Rows and columns
# end inside a tile, K inside a slice; 1, 2, 3 and more slices, odd and even.
CASES = [
    (FWD, 1797, 40, 2248, 256, "whole", False),
    (FWD, 12000, 72, 1608, 256, "whole", False),
    (FWD, 9001, 136, 2056, 256, "whole", False),
    (FWD, 5003, 1032, 3080, 256, "whole", False),
    (FWD, 4099, 1001, 3081, 256, "whole", True),
    (FWD, 13280, 736, 584, 256, "beside", False),
    (FWD, 1458, 1120, 5456, 256, "beside8", False),
    (FWD, 2522, 4928, 1624, 256, "pieces", False),
    (FWD, 12067, 40, 136, 128, "whole", False),
    (FWD, 2051, 1608, 1544, 128, "whole", False),
    (FWD, 2051, 777, 1609, 128, "whole", True),
    (FWD, 8443, 5056, 80, 128, "pieces", False),
    (FWD, 414, 1744, 72, 64, "pieces", False),
    (FWD, 301, 1448, 40, 64, "pieces8", False),
    (GI, 9753, 392, 40, 256, "whole", False),
    (GI, 4099, 1544, 1032, 256, "whole", False),
    (GI, 4099, 1001, 3081, 256, "whole", True),
    (GI, 3416, 2424, 976, 256, "beside", False),
    (GI, 3257, 2456, 3200, 256, "beside8", False),
    (GI, 13243, 280, 5528, 256, "pieces", False),
    (GI, 9041, 200, 40, 128, "whole", False),
    (GI, 2051, 1608, 1544, 128, "whole", False),
    (GI, 8630, 72, 5136, 128, "pieces", False),
    (GI, 287, 40, 1456, 64, "pieces8", False),
    (GW, 258, 872, 4736, 256, "whole", False),
    (GW, 711, 3240, 2544, 256, "beside", False),
    (GW, 1238, 1504, 5424, 256, "beside8", False),
    (GW, 9355, 144, 5648, 256, "pieces", False),
    (GW, 265, 2336, 872, 128, "whole", False),
    (GW, 2051, 1608, 1544, 128, "whole", False),
    (GW, 4099, 1001, 3081, 128, "whole", True),
    (GW, 7257, 72, 4432, 128, "pieces", False),
    (GW, 11274, 72, 2664, 128, "pieces8", False),
    (GW, 1305, 40, 40, 64, "pieces8", False),
]


def _id(c):
    return f"{'fwd gi gw'.split()[c[0]]}-{c[1]}x{c[2]}x{c[3]}-{c[4]}{c[5]}{'-packed' if c[6] else ''}"


def _sizes(case, layout):
    """Tokens, in and out: those of an [out, in] weight's gradient change places,
    so that the product and its cut are the same."""
    n, i, o = case[1:4]
    return (n, o, i) if case[0] == GW and layout == "out_in" else (n, i, o)


def plans(tmp_path, lines):
    """What layers.cpp makes of products (tests/native/layer_plan.cpp)."""
    exe = str(tmp_path / "layer_plan")
    subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include", f"-I{ROOT}/include",
                    f"-I{CSRC}", os.path.join(NATIVE, "layer_plan.cpp"), os.path.join(NATIVE, "layer_stubs.cpp"), "-o",
                    exe, f"-L{ROCM}/lib", "-lamdhip64", f"-Wl,-rpath,{ROCM}/lib"], check=True)
    r = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, timeout=60, check=True)
    return [[int(v) for v in row.split()] for row in r.stdout.splitlines()]


@pytest.mark.skipif(not _have_toolchain(), reason="g++ / ROCm HIP runtime not available")
def test_cases_take_the_tiles_they_stand_for(tmp_path):
    keys = [(c, lay) for c in CASES for lay in (0, 1)]
    got = plans(tmp_path, ["%d %d %d %d %d 0 0 0 0 0" % (c[0], *_sizes(c, ("in_out", "out_in")[lay]), lay)
                           for c, lay in keys])
    assert len(got) == len(keys)
    for (c, lay), (status, tile, tiles, whole, splits, slices, raw, pack_a, pack_b) in zip(keys, got):
        cut = "whole" if whole == tiles else ("beside" if whole else "pieces") + ("8" if splits >= 8 else "")
        assert (status, tile, cut, raw) == (0, c[4], c[5], 0), (_id(c), lay)
        assert (pack_a or pack_b) == c[6], (_id(c), lay)
    kinds = {(c[0], c[4], c[5].rstrip("8")) for c in CASES}
    for op in (FWD, GI, GW):
        assert {(op, 256, "whole"), (op, 256, "beside"), (op, 256, "pieces"), (op, 128, "whole"),
                (op, 128, "pieces"), (op, 64, "pieces")} <= kinds


def _rand(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _product(a, b):
    """a b and the bound on a float32 sum's error, in 64 bits."""
    a, b = a.double().contiguous(), b.double().contiguous()
    return a @ b, (8 + 4 * math.sqrt(a.shape[1])) * U * (a.abs() @ b.abs())


def _close(got, want, tol, dtype):
    f = torch.finfo(dtype)
    lim = tol + (want.abs() + tol) * (f.eps / 2) + f.smallest_normal * f.eps / 2
    assert got.shape == want.shape and got.dtype is dtype
    bad = ~((got.double() - want).abs() <= lim)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(), float(((got.double() - want).abs() / lim).max()))


def _gate(z):
    return torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))


def _gapped(t, pad, first=1):
    """The tensor in rows `pad` elements longer, `first` elements into their
    allocation, and the buffer of its rows; the gaps hold NaN."""
    r, c = t.shape
    buf = torch.full((first + r * (c + pad),), float("nan"), dtype=t.dtype, device="cuda")[first:].view(r, c + pad)
    buf[:, :c] = t
    return buf[:, :c], buf


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("case", CASES, ids=_id)
def test_each_tile_and_cut(case, layout):
    op, (n, i, o) = case[0], _sizes(case, layout)
    dtype = T["fp16" if (n + (layout == "in_out")) % 2 else "bf16"]
    g = torch.Generator(device="cuda").manual_seed(n + i)
    w = _rand(g, (i, o) if layout == "in_out" else (o, i), dtype, i ** -0.5)
    w64 = w if layout == "in_out" else w.t()
    kw = {"weight_layout": layout}
    if op == FWD:
        x, res, bias = _rand(g, (n, i), dtype), _rand(g, (n, o), dtype), torch.randn(o, generator=g, device="cuda")
        p, tol = _product(x, w64)
        plain = L.linear_forward(x, w, **kw)
        _close(plain, p, tol, dtype)
        y, z = L.linear_forward(x, w, bias=bias, residual=res, activation="gelu_tanh", save_preact=True, **kw)
        p, tol = p + bias.double(), tol + 2 * U * (p.abs() + bias.double().abs())
        _close(z, p, tol, dtype)
        act = p * _gate(p)
        # the slope is at most 1.2; about ten float32 steps, and the last addition
        _close(y, act + res.double(), 1.2 * tol + 16 * U * (p.abs() + act.abs()) + U * (act + res.double()).abs(), dtype)
        # the same bits into rows off 16-byte borders, whose gaps stay as they are, and in place over the residual
        (ys, yb), (zs, zb), (rs, rb) = _gapped(torch.zeros_like(y), 3), _gapped(torch.zeros_like(z), 5), _gapped(res, 1)
        L.linear_forward(x, w, bias=bias, residual=rs, activation="gelu_tanh", out=ys, preact_out=zs, **kw)
        assert torch.equal(ys, y) and torch.equal(zs, z)
        assert yb[:, o:].isnan().all() and zb[:, o:].isnan().all()
        L.linear_forward(x, w, bias=bias, residual=rs, activation="gelu_tanh", out=rs, **kw)
        assert torch.equal(rs, y) and rb[:, o:].isnan().all()
    elif op == GI:
        dy, add, pre = _rand(g, (n, o), dtype, 0.1), _rand(g, (n, i), dtype, 0.1), _rand(g, (n, i), dtype, 2.0)
        p, tol = _product(dy, w64.t())
        _close(L.linear_grad_input(dy, w, **kw), p, tol, dtype)
        _close(L.linear_grad_input(dy, w, add=add, **kw), p + add.double(), tol + U * (p + add.double()).abs(), dtype)
        z = pre.double()
        q = _gate(z)
        slope = q + z * q * (1 - q) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
        want = p * slope + add.double()
        tol = tol * slope.abs() + U * (16 * p.abs() * (1 + z.abs()) + want.abs())
        dx = L.linear_grad_input(dy, w, preact=pre, activation="gelu_tanh", add=add, **kw)
        _close(dx, want, tol, dtype)
        (ds, db), (ps, _), (adds, _) = _gapped(torch.zeros_like(dx), 3), _gapped(pre, 5), _gapped(add, 1)
        L.linear_grad_input(dy, w, preact=ps, activation="gelu_tanh", add=adds, out=ds, **kw)
        assert torch.equal(ds, dx) and db[:, i:].isnan().all()
        L.linear_grad_input(dy, w, preact=ps, activation="gelu_tanh", add=adds, out=adds, **kw)
        assert torch.equal(adds, dx)
    else:
        x, dy = _rand(g, (n, i), dtype), _rand(g, (n, o), dtype, 0.1)
        a, b = (x.t(), dy) if layout == "in_out" else (dy.t(), x)
        p, tol = _product(a, b)
        dw, db = L.linear_grad_weight(x, dy, dbias=True, **kw)
        _close(dw, p, tol, torch.float32)
        s, stol = _product(torch.ones(1, n, device="cuda"), dy)
        _close(db, s[0], stol[0], torch.float32)
        assert torch.equal(L.linear_grad_weight(x, dy, **kw)[0], dw)
        ws, wb = _gapped(torch.zeros_like(dw), 3)
        bs = torch.full((o + 2,), float("nan"), device="cuda")
        L.linear_grad_weight(x, dy, dw=ws, dbias=bs[1:-1], **kw)
        assert torch.equal(ws, dw) and torch.equal(bs[1:-1], db)
        L.linear_grad_weight(x, dy, dw=ws, dbias=bs[1:-1], accumulate=True, **kw)
        assert torch.equal(ws, 2 * dw) and torch.equal(bs[1:-1], 2 * db)
        assert wb[:, dw.shape[1]:].isnan().all() and bs[0].isnan() and bs[-1].isnan()


@pytest.mark.gpu
def test_pieces_in_two_graphs_at_once():
    """Products in K pieces captured into two graphs, replayed on two streams at
    the same time, with eager calls between the replays: each has a workspace of
    its own."""
    g = torch.Generator(device="cuda").manual_seed(3)
    sets = []
    for _ in range(2):
        x, dy = _rand(g, (1238, 1504), torch.bfloat16), _rand(g, (1238, 5424), torch.bfloat16, 0.1)
        sets.append({"x": x, "dy": dy, "dw": torch.zeros(1504, 5424, device="cuda"),
                     "db": torch.zeros(5424, device="cuda"), "graph": torch.cuda.CUDAGraph(),
                     "stream": torch.cuda.Stream()})
    for s in sets:
        L.linear_grad_weight(s["x"], s["dy"], dw=s["dw"], dbias=s["db"])
        torch.cuda.synchronize()
        with torch.cuda.graph(s["graph"], stream=s["stream"]):
            L.linear_grad_weight(s["x"], s["dy"], dw=s["dw"], dbias=s["db"])
    for k in range(3):
        for s in sets:
            s["x"].copy_(_rand(g, s["x"].shape, torch.bfloat16))
            s["dw"].zero_()
            s["db"].zero_()
        torch.cuda.synchronize()
        for s in sets:
            with torch.cuda.stream(s["stream"]):
                s["graph"].replay()
        torch.cuda.synchronize()
        for s in sets:
            dw, db = L.linear_grad_weight(s["x"], s["dy"], dbias=True)
            assert torch.equal(s["dw"], dw) and torch.equal(s["db"], db), k
