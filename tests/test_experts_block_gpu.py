"""The RMS norm, the 8-bit and the grouped operators as a block of a mixture of experts
uses them, on the GPU: norm of a residual sum with an 8-bit output for a layer that all
tokens pass, experts on rows grouped by expert, the way back through both, and the Muon
step that reads the experts' gradients. Then the same block captured, and on two
streams at once; offsets past 32 bits; ranges of one buffer.
"""

import pytest
import torch

from eight import U, act64, act_tol, close, cpu64, eight, gen, rand, slope64, sum_tol, values
from muon_newton_schulz_04_amd import binding as B
from muon_newton_schulz_04_amd import layers as L
from test_linear_fp8_gpu import _tol

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
D, H, E = 128, 256, 4


def _block(seed, counts, n=70):
    """The block's tensors, and a call that runs it forward and backward."""
    g = gen(seed)

    def mk(*shape, std=1.0, dtype=BF):
        return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()

    at = torch.tensor([0] + counts).cumsum(0)
    assert len(counts) == E and at[-1] == n
    s = {"x": mk(n, D), "res": mk(n, D), "dout": mk(n, D, std=0.1), "off": at.int().cuda(),
         "lw": 1 + mk(D, std=0.1, dtype=torch.float32), "ws": mk(D, D, std=0.06), "bs": mk(D, dtype=torch.float32),
         "w1": mk(E, D, H, std=0.06), "b1": mk(E, H, std=0.3, dtype=torch.float32), "w2": mk(E, H, D, std=0.04)}
    s["grads"] = torch.zeros(2 * E * D * H, device="cuda")
    s["small"] = torch.zeros(D * D, device="cuda")

    def run():
        o = {}
        o["h"] = torch.empty(n, D, dtype=BF, device="cuda")
        (q, qs), o["rstd"], o["r"] = L.rmsnorm_forward(s["x"], s["lw"], residual=s["res"], out=o["h"],
                                                       quantize=torch.float8_e4m3fn)
        w8, w8t = L.quantize_fp8_weight(s["ws"], transpose=True)
        o["shared"] = L.linear_fp8_forward((q, qs), w8, bias=s["bs"], residual=o["r"])
        o["a"], o["z"] = L.grouped_linear_forward(o["h"], s["w1"], s["off"], bias=s["b1"], activation="silu",
                                                  save_preact=True)
        o["out"] = L.grouped_linear_forward(o["a"], s["w2"], s["off"], residual=o["shared"])
        g1, g2 = s["grads"][:E * D * H].view(E, D, H), s["grads"][E * D * H:].view(E, H, D)
        o["g2"], _ = L.grouped_linear_grad_weight(o["a"], s["dout"], s["off"], dw=g2)
        o["dz"] = L.grouped_linear_grad_input(s["dout"], s["w2"], s["off"], preact=o["z"], activation="silu")
        o["g1"], o["db1"] = L.grouped_linear_grad_weight(o["h"], o["dz"], s["off"], dw=g1, dbias=True)
        o["dh"] = L.grouped_linear_grad_input(o["dz"], s["w1"], s["off"])
        d8 = L.quantize_fp8(s["dout"], torch.float8_e5m2)
        o["dh2"] = L.linear_fp8_grad_input(d8, w8t, add=o["dh"])
        o["gs"], o["dbs"] = L.linear_grad_weight(o["h"], s["dout"], dw=s["small"].view(D, D), dbias=True)
        o["dr"], o["dlw"] = L.rmsnorm_backward(o["dh2"], o["r"], o["rstd"], s["lw"], add=s["dout"], dweight=True)
        for name, (data, scale) in (("q", (q, qs)), ("w8", w8), ("w8t", w8t), ("d8", d8)):
            o[name], o[name + "s"] = data.view(torch.uint8), scale
        return o

    return s, run


def _eight_of(o, name, f8):
    return o[name].view(f8), o[name + "s"]


def test_block_with_a_muon_step():
    """Each result against the formula on what the call before it stored, the gradients
    against differences of the block's loss in 64 bits, and the step that reads them."""
    counts = [31, 0, 38, 1]
    s, run = _block(3, counts)
    raw = run()
    o = {k: cpu64(v) for k, v in raw.items() if v.dtype != torch.uint8}
    e4, e5 = torch.float8_e4m3fn, torch.float8_e5m2
    q, w8 = values(_eight_of(raw, "q", e4)), values(_eight_of(raw, "w8", e4), True)
    w8t, d8 = values(_eight_of(raw, "w8t", e4), True), values(_eight_of(raw, "d8", e5))
    assert torch.equal(w8t, w8.t())
    x, res, dout, lw, ws, bs, w1, b1, w2 = (cpu64(s[k]) for k in
                                            ("x", "res", "dout", "lw", "ws", "bs", "w1", "b1", "w2"))
    at = s["off"].tolist()
    rows = [(e, slice(at[e], at[e + 1])) for e in range(E)]

    def norm(r):
        return r / (r.square().mean(1, keepdim=True) + 1e-5).sqrt()

    close(raw["r"], x + res, U * (x + res).abs(), BF)
    xh = norm(o["r"])
    close(raw["h"], xh * lw, 100 * U * (1 + xh.abs()) * lw.abs(), BF)
    # 8-bit values of what h is rounded from: half a step of each format's largest binade
    top = (xh * lw).abs().amax(1, keepdim=True)
    assert ((q - xh * lw).abs() <= 2.0 ** -4 * (1 + 2.0 ** -10) * (xh * lw).abs() + 2.0 ** -10 * top / 448).all()
    z = q @ w8.t() + bs
    want = z + o["r"]
    close(raw["shared"], want, _tol(q, w8.t()) + U * (2 * z.abs() + want.abs()), BF)
    for e, r in rows:
        z = o["h"][r] @ w1[e] + b1[e]
        zt = sum_tol(o["h"][r], w1[e]) + 2 * U * z.abs()
        close(raw["z"][r], z, zt, BF)
        close(raw["a"][r], act64("silu", z), act_tol("silu", z, zt), BF)
        want = o["a"][r] @ w2[e] + o["shared"][r]
        close(raw["out"][r], want, sum_tol(o["a"][r], w2[e]) + U * want.abs(), BF)
        pre, sl = dout[r] @ w2[e].t(), slope64("silu", o["z"][r])
        close(raw["dz"][r], pre * sl,
              sum_tol(dout[r], w2[e].t()) * sl.abs() + 16 * U * pre.abs() * (1 + o["z"][r].abs()), BF)
        close(raw["dh"][r], o["dz"][r] @ w1[e].t(), sum_tol(o["dz"][r], w1[e].t()), BF)
        close(raw["g2"][e], o["a"][r].t() @ dout[r], sum_tol(o["a"][r].t(), dout[r]), torch.float32)
        close(raw["g1"][e], o["h"][r].t() @ o["dz"][r], sum_tol(o["h"][r].t(), o["dz"][r]), torch.float32)
        ones = torch.ones(1, counts[e], dtype=torch.float64)
        close(raw["db1"][e], o["dz"][r].sum(0), sum_tol(ones, o["dz"][r])[0], torch.float32)
    want = d8 @ w8t.t() + o["dh"]
    close(raw["dh2"], want, _tol(d8, w8t.t()) + U * want.abs(), BF)

    def parts(x, ws, w1, b1, w2, lw):
        h = norm(x + res) * lw
        shared = h @ ws
        out = shared + x + res
        mixed = torch.cat([act64("silu", h[r] @ w1[e] + b1[e]) @ w2[e] for e, r in rows])
        return shared, ((out + mixed) * dout).sum()

    # As for the dense block: 2^-6 of |gradient| |direction| is four times what the bf16
    # roundings can add up to in one sign. The gradient that goes back through the 8-bit
    # layer is besides of 8-bit operands: dout off by 2^-3 of each element at most, so the
    # loss along a direction by 2^-3 |dout| |what the layer's output changes along it|;
    # the loss takes the weight's own 8-bit values.
    g = gen(5)
    at64 = [x, w8.t(), w1, b1, w2, lw]
    grads = [o["dr"], o["gs"], o["g1"], o["db1"], o["g2"], o["dlw"]]
    for k in range(6):
        v = [torch.zeros_like(t) for t in at64]
        v[k] = grads[k] / grads[k].norm() + 0.5 * torch.randn(at64[k].shape, generator=g).double() / at64[k].numel() ** 0.5
        h = 1e-4
        up, down = (parts(*[a + f * h * b for a, b in zip(at64, v)]) for f in (1, -1))
        diff, moved = (up[1] - down[1]) / (2 * h), (up[0] - down[0]) / (2 * h)
        tol = 2.0 ** -6 * grads[k].norm() * v[k].norm()
        if k in (0, 5):
            tol = tol + 2.0 ** -3 * dout.norm() * moved.norm()
        got = (grads[k] * v[k]).sum()
        assert abs(got - diff) <= tol, (k, got, diff, tol)

    table = [B.muon_matrix(D, H, E, 0, 1.0, 1.0, 0, 0), B.muon_matrix(H, D, E, E * D * H, 1.0, 1.0, 0, 0)]
    params = torch.cat([s["w1"].float().flatten(), s["w2"].float().flatten()])
    after = []
    for grad in (s["grads"], s["grads"].clone()):
        handle = B.MuonHandle(table, B.make_hparams())
        p, m = params.clone(), torch.zeros_like(params)
        handle.step(p, grad, m, lr=0.02)
        torch.cuda.synchronize()
        assert (handle.view(B.MUON_VIEW_STATUS, torch.int32) == 0).all()
        handle.close()
        after.append(p)
    assert torch.equal(after[0], after[1]) and after[0].isfinite().all() and not torch.equal(after[0], params)
    # the expert without rows has a gradient of zeros and stays
    p, before = after[0][:E * D * H].view(E, D, H), params[:E * D * H].view(E, D, H)
    assert torch.equal(p[1], before[1]) and not torch.equal(p[0], before[0])


def test_graph_replays_match_eager_calls():
    """One graph for any choice of the router: the offsets are read where they lie."""
    s, run = _block(12, [20, 10, 30, 10])
    run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for k, counts in enumerate(([70, 0, 0, 0], [0, 1, 0, 69], [17, 18, 16, 19], [0, 0, 64, 6])):
        fresh, fresh_run = _block(20 + k, counts)
        for name in ("x", "res", "dout", "off", "lw", "ws", "bs", "w1", "b1", "w2"):
            s[name].copy_(fresh[name])
        graph.replay()
        torch.cuda.synchronize()
        got = {n: v.clone() for n, v in held.items()}
        want = fresh_run()  # the program's own eager work between replays
        for n in got:
            assert torch.equal(got[n], want[n]), (k, n)


def test_two_graphs_and_two_streams_at_once():
    pairs = [_block(31, [40, 10, 0, 20]), _block(32, [3, 3, 60, 4])]
    want = []
    for s, run in pairs:
        want.append({k: v.clone() for k, v in run().items()})
        s["grads"].zero_()
        s["small"].zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(3):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[k] = pairs[k][1]()
    torch.cuda.synchronize()
    for k in range(2):
        for n in want[k]:
            assert torch.equal(got[k][n], want[k][n]), (k, n)
    graphs, held = [], []
    for s, run in pairs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(run())
        graphs.append(g)
        s["grads"].zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for k in range(2):
            for n in want[k]:
                assert torch.equal(held[k][n], want[k][n]), (k, n)


def test_offsets_past_32_bits():
    """Rows 2^21 elements apart, 2100 of them, and experts' weights 2^31 apart: elements
    (and bytes) past 2^32 from a tensor's start."""
    g = gen(9)
    n, i, o, ld = 2100, 96, 40, 1 << 21
    flat = torch.empty(n * ld, dtype=BF, device="cuda")
    far = flat.view(n, ld)

    def put(at, v):
        far[:, at:at + v.shape[1]] = v
        return far[:, at:at + v.shape[1]]

    near = {k: rand(g, (n, i), BF) for k in ("x", "res", "dy")}
    at = {k: put(j * 128, near[k]) for j, k in enumerate(near)}
    y, rstd, r = L.rmsnorm_forward(near["x"], residual=near["res"])
    out, sums = put(1024, y * 0), put(1152, y * 0)
    y2, rstd2, r2 = L.rmsnorm_forward(at["x"], residual=at["res"], out=out, residual_out=sums)
    assert torch.equal(y, y2) and torch.equal(r, r2) and torch.equal(rstd, rstd2)
    dx, _ = L.rmsnorm_backward(near["dy"], r, rstd)
    dx2, _ = L.rmsnorm_backward(at["dy"], r2, rstd, out=put(1280, y * 0))
    assert torch.equal(dx, dx2)
    q, q2 = L.quantize_fp8(near["x"]), L.quantize_fp8(at["x"])
    assert torch.equal(q.data.view(torch.uint8), q2.data.view(torch.uint8)) and torch.equal(q.scale, q2.scale)
    w8, _ = L.quantize_fp8_weight(near["x"][:, :o].contiguous())
    w8b, _ = L.quantize_fp8_weight(at["x"][:, :o])
    assert torch.equal(w8.data.view(torch.uint8), w8b.data.view(torch.uint8))
    # 8-bit rows 2^21 bytes apart
    w = eight(g, o, i, weight=True)
    far8 = flat.view(torch.uint8).view(-1)[:n * ld].view(n, ld)
    want = L.linear_fp8_forward(q, w)
    far8[:, 256 * 64:256 * 64 + i] = q.data.view(torch.uint8)
    x8 = far8[:, 256 * 64:256 * 64 + i].view(torch.float8_e4m3fn)
    assert torch.equal(L.linear_fp8_forward((x8, q.scale), w), want)
    assert torch.equal(L.linear_fp8_forward(q, w, out=put(2048, want * 0)), want)
    off = torch.tensor([0, 900, 2100], dtype=torch.int32).cuda()
    we = (torch.randn(2, i, o, generator=g) * 0.1).to(BF).cuda()
    spare = torch.empty((1 << 31) + i * o, dtype=BF, device="cuda")
    wide = spare.as_strided((2, i, o), (1 << 31, o, 1))
    wide.copy_(we)
    want = L.grouped_linear_forward(near["x"], we, off)
    assert torch.equal(L.grouped_linear_forward(at["x"], wide, off, out=put(4096, want * 0)), want)
    want = L.grouped_linear_grad_input(want, we, off)
    dy = L.grouped_linear_forward(near["x"], we, off)
    assert torch.equal(L.grouped_linear_grad_input(put(8192, dy), wide, off, out=put(12288, want * 0)), want)
    dw, _ = L.grouped_linear_grad_weight(near["x"], dy, off)
    fw = torch.empty((1 << 30) + i * o, device="cuda").as_strided((2, i, o), (1 << 30, o, 1))
    dw2, _ = L.grouped_linear_grad_weight(at["x"], far[:, 8192:8192 + o], off, dw=fw)
    assert torch.equal(dw, dw2)


def test_sums_in_place_of_either_operand():
    g = gen(4)
    for cols in (72, 1003, 9001):
        x, res = rand(g, (9, cols), BF, stride=cols + 5), rand(g, (9, cols), BF, stride=cols + 5)
        y, rstd, r = L.rmsnorm_forward(x, residual=res)
        for into in (0, 1):
            pair = [x.clone(), res.clone()]
            y2, rstd2, r2 = L.rmsnorm_forward(pair[0], residual=pair[1], residual_out=pair[into])
            assert r2 is pair[into]
            assert torch.equal(y2, y) and torch.equal(rstd2, rstd) and torch.equal(r2, r)


@pytest.mark.parametrize("at", [0, 1, 8])
def test_column_ranges_of_one_buffer(at):
    """Operands and results side by side in the rows of one buffer, aligned to 16 bytes
    or to 2; what lies between stays."""
    g = gen(at)
    n, i, o = 150, 72, 136
    x, res = rand(g, (n, i), BF), rand(g, (n, o), BF)
    off = torch.tensor([0, 90, 90, 131], dtype=torch.int32).cuda()
    w = (torch.randn(3, i, o, generator=g) * 0.1).to(BF).cuda()
    want = L.grouped_linear_forward(x, w, off, residual=res)
    y, rstd = L.rmsnorm_forward(x)
    buf = torch.full((n, 600), 3.0, dtype=BF, device="cuda")
    buf[:, at:at + i], buf[:, 80 + at:80 + at + o] = x, res
    before = buf.clone()
    got = L.grouped_linear_forward(buf[:, at:at + i], w, off, residual=buf[:, 80 + at:80 + at + o],
                                   out=buf[:, 80 + at:80 + at + o])
    assert torch.equal(got[:131], want[:131])
    assert torch.equal(got[131:], res[131:])  # rows of no expert
    got2, _ = L.rmsnorm_forward(buf[:, at:at + i], out=buf[:, 320 + at:320 + at + i])
    assert torch.equal(got2, y)
    before[:, 80 + at:80 + at + o], before[:, 320 + at:320 + at + i] = got, got2
    assert torch.equal(buf, before)
    q, q2 = L.quantize_fp8(x), L.quantize_fp8(buf[:, at:at + i])
    assert torch.equal(q.data.view(torch.uint8), q2.data.view(torch.uint8)) and torch.equal(q.scale, q2.scale)
