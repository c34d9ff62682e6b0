"""The layer operators of libmuon on torch tensors: the linear layer (matrix
product with bias, activation and residual in its epilogue) with its two
gradients, and layer norm with its backward pass. They make the gradients
that a Muon step reads: `dw` may be a view of the flat gradient buffer.

Each function checks its tensors, allocates the outputs that are not given and
the workspace through torch's caching allocator, and makes one C call
(include/libmuon.h) on the tensors' device and that device's current stream.
It never synchronises, and may be captured into a graph. They are plain
functions, not autograd ones: gradients are what the `*_grad_*` and
`*_backward` calls return.

Matrices are [rows, features] with any row stride (the last dimension
contiguous); leading dimensions of x, dy and the like are flattened only by
the caller. Weights are [in, out] ("in_out", as the body's c_fc [d, 4d]) or
[out, in] ("out_in").
"""

from __future__ import annotations

import torch

from . import binding as B

_TYPES = {torch.bfloat16: B.MUON_TYPE_BF16, torch.float16: B.MUON_TYPE_FP16, torch.float32: B.MUON_TYPE_FP32}
_LAYOUTS = {"in_out": B.MUON_WEIGHT_IN_OUT, "out_in": B.MUON_WEIGHT_OUT_IN}
ACTIVATIONS = {"none": B.MUON_ACT_NONE, "relu": B.MUON_ACT_RELU, "relu2": B.MUON_ACT_RELU2, "gelu": B.MUON_ACT_GELU,
               "gelu_tanh": B.MUON_ACT_GELU_TANH, "silu": B.MUON_ACT_SILU}


def _matrix(name, t, dtype, device, rows=None, cols=None):
    """Row stride of a matrix argument, after its checks."""
    if t.dim() != 2 or (rows is not None and t.shape[0] != rows) or (cols is not None and t.shape[1] != cols):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [{'*' if rows is None else rows}, "
                         f"{'*' if cols is None else cols}]")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    r, c = t.shape
    s0, s1 = t.stride()
    if c > 1 and s1 != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    if r <= 1:
        return c
    if s0 < c:
        raise ValueError(f"{name}: rows overlap (stride {s0}, length {c})")
    return s0


def _vector(name, t, n, device):
    if t.dim() != 1 or t.shape[0] != n:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [{n}]")
    if t.dtype != torch.float32:
        raise ValueError(f"{name}: dtype {t.dtype}, expected torch.float32")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if n > 1 and t.stride(0) != 1:
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr()


def _first(name, t):
    """Type and device of a call's first tensor."""
    if not t.is_cuda:
        raise ValueError(f"{name}: on {t.device}, expected a GPU tensor")
    return t.dtype, t.device


def _check(status, what):
    if status != B.MUON_OK:
        raise B.MuonError(f"{what}: {B.muon_status_string(status)} ({B.muon_op_last_error()})")


def _call(device, fn):
    """fn(stream pointer) with `device` current."""
    if device.index == torch.cuda.current_device():
        return fn(torch.cuda.current_stream().cuda_stream)
    with torch.cuda.device(device):
        return fn(torch.cuda.current_stream().cuda_stream)


def _workspace(nbytes, device):
    """A workspace of its own for one call, from the current stream's pool."""
    if nbytes == 0:
        return None, 0
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return ws, ws.data_ptr()


def _choice(table, value, what):
    try:
        return table[value]
    except (KeyError, TypeError):
        raise ValueError(f"{what} {value!r}: expected one of {', '.join(table)}") from None


def _linear(x_name, x, w, layout, dtype):
    if dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"{x_name}: dtype {dtype}, expected torch.bfloat16 or torch.float16")
    return _choice(_LAYOUTS, layout, "weight_layout")


def _run_linear(op, call, what, a, w, act, bias, add, z, out, layout, device, dtype):
    """forward (a = x) and grad input (a = dy)."""
    lay = _linear("x" if op == B.MUON_LINEAR_FORWARD else "dy", a, w, layout, dtype)
    fwd = op == B.MUON_LINEAR_FORWARD
    if w.dim() != 2:
        raise ValueError(f"w: shape {tuple(w.shape)}, expected a matrix")
    fin, fout = w.shape if lay == B.MUON_WEIGHT_IN_OUT else (w.shape[1], w.shape[0])
    ld_a = _matrix("x" if fwd else "dy", a, dtype, device, None, fin if fwd else fout)
    ld_w = _matrix("w", w, dtype, device)
    rows, cols = a.shape[0], fout if fwd else fin
    if out is None:
        out = torch.empty((rows, cols), dtype=dtype, device=device)
        ld_o = cols
    else:
        ld_o = _matrix("out", out, dtype, device, rows, cols)
    d = B.muon_linear(rows, fin, fout, ld_a if fwd else ld_o, ld_w, ld_o if fwd else ld_a, _TYPES[dtype], lay)
    e = None
    if act or bias is not None or add is not None or z is not None:
        e = B.muon_epilogue(act, 0)
        if bias is not None:
            e.bias = _vector("bias", bias, fout, device)
        if add is not None:
            e.ld_add = _matrix("residual" if fwd else "add", add, dtype, device, rows, cols)
            e.add = add.data_ptr()
        if z is not None:
            e.ld_z = _matrix("preact", z, dtype, device, rows, cols)
            e.z = z.data_ptr()
    pa, pw, po = a.data_ptr(), w.data_ptr(), out.data_ptr()
    s, nbytes = B.muon_linear_workspace_bytes(d, op, pa, pw, e, po)
    _check(s, what)
    ws, pws = _workspace(nbytes, device)
    _check(_call(device, lambda st: call(d, pa, pw, e, po, pws, nbytes, st)), what)
    return out


def linear_forward(x, w, bias=None, residual=None, activation="none", weight_layout="in_out", save_preact=False,
                   out=None, preact_out=None):
    """y = act(x w + bias) + residual; with save_preact (or preact_out) also
    z = x w + bias rounded to x's type, for linear_grad_input of the next
    layer: returns y, or (y, z). `out` may be `residual` itself."""
    dtype, device = _first("x", x)
    act = _choice(ACTIVATIONS, activation, "activation")
    z = preact_out
    if z is None and save_preact:
        lay = _choice(_LAYOUTS, weight_layout, "weight_layout")
        z = torch.empty((x.shape[0], w.shape[1 if lay == B.MUON_WEIGHT_IN_OUT else 0]), dtype=dtype, device=device)
    y = _run_linear(B.MUON_LINEAR_FORWARD, B.muon_linear_forward, "linear_forward", x, w, act, bias, residual, z, out,
                    weight_layout, device, dtype)
    return y if z is None else (y, z)


def linear_grad_input(dy, w, preact=None, activation="none", add=None, weight_layout="in_out", out=None):
    """dx = (dy w^T) * act'(preact) + add. With an activation, `preact` is the
    pre-activation that made this layer's x (x = act(preact)), and dx is its
    gradient. `out` may be `add` itself."""
    dtype, device = _first("dy", dy)
    act = _choice(ACTIVATIONS, activation, "activation")
    return _run_linear(B.MUON_LINEAR_GRAD_INPUT, B.muon_linear_grad_input, "linear_grad_input", dy, w, act, None, add,
                       preact if act else None, out, weight_layout, device, dtype)


def linear_grad_weight(x, dy, dw=None, dbias=None, accumulate=False, weight_layout="in_out"):
    """(dw, dbias): the float32 gradients of a linear layer's weight and bias,
    written to (or with accumulate added to) the tensors given. dbias=True
    allocates one; None leaves the bias gradient out."""
    dtype, device = _first("x", x)
    lay = _linear("x", x, None, weight_layout, dtype)
    ld_x = _matrix("x", x, dtype, device)
    ld_y = _matrix("dy", dy, dtype, device, x.shape[0])
    fin, fout = x.shape[1], dy.shape[1]
    shape = (fin, fout) if lay == B.MUON_WEIGHT_IN_OUT else (fout, fin)
    if accumulate and (dw is None or dbias is True):
        raise ValueError("accumulate needs the tensors to add to")
    if dw is None:
        dw = torch.empty(shape, dtype=torch.float32, device=device)
    ld_w = _matrix("dw", dw, torch.float32, device, *shape)
    if dbias is True:
        dbias = torch.empty(fout, dtype=torch.float32, device=device)
    pb = 0 if dbias is None else _vector("dbias", dbias, fout, device)
    d = B.muon_linear(x.shape[0], fin, fout, ld_x, ld_w, ld_y, _TYPES[dtype], lay)
    px, py, pd = x.data_ptr(), dy.data_ptr(), dw.data_ptr()
    s, nbytes = B.muon_linear_workspace_bytes(d, B.MUON_LINEAR_GRAD_WEIGHT, px, py, None, pd)
    _check(s, "linear_grad_weight")
    ws, pws = _workspace(nbytes, device)
    _check(_call(device, lambda st: B.muon_linear_grad_weight(d, px, py, pd, pb, int(accumulate),
                                                                      pws, nbytes, st)), "linear_grad_weight")
    return dw, dbias


def layernorm_forward(x, weight=None, bias=None, eps=1e-5, out=None):
    """(y, mean, rstd) of layer norm over the rows of x (bf16, fp16 or fp32);
    weight, bias, mean and rstd are float32."""
    dtype, device = _first("x", x)
    if dtype not in _TYPES:
        raise ValueError(f"x: dtype {dtype}, expected torch.bfloat16, torch.float16 or torch.float32")
    ld_x = _matrix("x", x, dtype, device)
    rows, cols = x.shape
    if out is None:
        out = torch.empty((rows, cols), dtype=dtype, device=device)
    ld_y = _matrix("out", out, dtype, device, rows, cols)
    stats = torch.empty((2, rows), dtype=torch.float32, device=device)
    mean, rstd = stats[0], stats[1]
    d = B.muon_layernorm(rows, cols, ld_x, ld_y, 0, 0, _TYPES[dtype], eps)
    pw = 0 if weight is None else _vector("weight", weight, cols, device)
    pb = 0 if bias is None else _vector("bias", bias, cols, device)
    pm = stats.data_ptr()
    _check(_call(device, lambda st: B.muon_layernorm_forward(d, x.data_ptr(), pw, pb, out.data_ptr(), pm,
                                                                     pm + 4 * rows, st)), "layernorm_forward")
    return out, mean, rstd


def layernorm_backward(dy, x, mean, rstd, weight=None, add=None, dweight=None, dbias=None, accumulate=False, out=None):
    """(dx, dweight, dbias): the gradient of x, plus `add`, and the float32
    gradients of weight and bias, written to (or with accumulate added to) the
    tensors given; True allocates one, None leaves it out. `out` may be `add`."""
    dtype, device = _first("dy", dy)
    if dtype not in _TYPES:
        raise ValueError(f"dy: dtype {dtype}, expected torch.bfloat16, torch.float16 or torch.float32")
    ld_y = _matrix("dy", dy, dtype, device)
    rows, cols = dy.shape
    ld_x = _matrix("x", x, dtype, device, rows, cols)
    pm, pr = _vector("mean", mean, rows, device), _vector("rstd", rstd, rows, device)
    pw = 0 if weight is None else _vector("weight", weight, cols, device)
    ld_a, pa = (0, 0) if add is None else (_matrix("add", add, dtype, device, rows, cols), add.data_ptr())
    if accumulate and (dweight is True or dbias is True):
        raise ValueError("accumulate needs the tensors to add to")
    if dweight is True:
        dweight = torch.empty(cols, dtype=torch.float32, device=device)
    if dbias is True:
        dbias = torch.empty(cols, dtype=torch.float32, device=device)
    pdw = 0 if dweight is None else _vector("dweight", dweight, cols, device)
    pdb = 0 if dbias is None else _vector("dbias", dbias, cols, device)
    if out is None:
        out = torch.empty((rows, cols), dtype=dtype, device=device)
    ld_o = _matrix("out", out, dtype, device, rows, cols)
    d = B.muon_layernorm(rows, cols, ld_x, ld_y, ld_o, ld_a, _TYPES[dtype], 0.0)
    nbytes = 0
    if pdw or pdb:
        s, nbytes = B.muon_layernorm_workspace_bytes(d)
        _check(s, "layernorm_backward")
    ws, pws = _workspace(nbytes, device)
    _check(_call(device, lambda st: B.muon_layernorm_backward(
        d, dy.data_ptr(), x.data_ptr(), pw, pm, pr, pa, out.data_ptr(), pdw, pdb, int(accumulate), pws, nbytes, st)),
        "layernorm_backward")
    return out, dweight, dbias
