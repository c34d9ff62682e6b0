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


def _matrix(name, t, dtype, dev, rows=-1, cols=-1):
    """Row stride of a matrix argument (rows, cols: what they have to be, -1
    any), after its checks."""
    if t.dim() == 2 and t.dtype is dtype and t.get_device() == dev:
        r, c = t.shape
        if (r == rows or rows < 0) and (c == cols or cols < 0):
            s0, s1 = t.stride()
            if s1 == 1 or c <= 1:
                if r <= 1:
                    return c
                if s0 >= c:
                    return s0
                raise ValueError(f"{name}: rows overlap (stride {s0}, length {c})")
            raise ValueError(f"{name}: the last dimension must be contiguous")
    _same(name, t, dtype, dev)
    raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [{'*' if rows < 0 else rows}, "
                     f"{'*' if cols < 0 else cols}]")


def _vector(name, t, n, dev):
    """Address of a contiguous float32 vector argument, after its checks."""
    if t.dtype is torch.float32 and t.get_device() == dev and t.shape == (n,):
        if n <= 1 or t.stride(0) == 1:
            return t.data_ptr()
        raise ValueError(f"{name}: must be contiguous")
    _same(name, t, torch.float32, dev)
    raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [{n}]")


def _same(name, t, dtype, dev):
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, expected cuda:{dev}")


def _first(name, t):
    """Type, device and device index of a call's first tensor."""
    if not t.is_cuda:
        raise ValueError(f"{name}: on {t.device}, expected a GPU tensor")
    return t.dtype, t.device, t.get_device()


def _check(status, what):
    if status != B.MUON_OK:
        raise B.MuonError(f"{what}: {B.muon_status_string(status)} ({B.muon_op_last_error()})")


# the current stream's handle, without a Stream object around it where torch
# offers that (1 us of a call's 10)
_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _on(dev, fn, *args):
    """fn(*args, stream) on device `dev`'s current stream, with `dev` current."""
    if dev == torch.cuda.current_device():
        return fn(*args, _stream(dev))
    with torch.cuda.device(dev):
        return fn(*args, _stream(dev))


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


def _linear_type(name, dtype):
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise ValueError(f"{name}: dtype {dtype}, expected torch.bfloat16 or torch.float16")
    return _TYPES[dtype]


def _weight(w, layout):
    """(layout code, in features, out features) of a weight."""
    lay = _choice(_LAYOUTS, layout, "weight_layout")
    if w.dim() != 2:
        raise ValueError(f"w: shape {tuple(w.shape)}, expected a matrix")
    a, b = w.shape
    return (lay, a, b) if lay == B.MUON_WEIGHT_IN_OUT else (lay, b, a)


def linear_forward(x, w, bias=None, residual=None, activation="none", weight_layout="in_out", save_preact=False,
                   out=None, preact_out=None):
    """y = act(x w + bias) + residual; with save_preact (or preact_out) also
    z = x w + bias rounded to x's type, for linear_grad_input of the next
    layer: returns y, or (y, z). `out` may be `residual` itself, unless that
    is x or w too."""
    dtype, device, dev = _first("x", x)
    code = _linear_type("x", dtype)
    act = _choice(ACTIVATIONS, activation, "activation")
    lay, fin, fout = _weight(w, weight_layout)
    ld_x = _matrix("x", x, dtype, dev, -1, fin)
    ld_w = _matrix("w", w, dtype, dev)
    n = x.shape[0]
    z = preact_out
    if z is None and save_preact:
        z = x.new_empty((n, fout))
    if out is None:
        out = x.new_empty((n, fout))
        ld_y = fout
    else:
        ld_y = _matrix("out", out, dtype, dev, n, fout)
    e = None
    if act or bias is not None or residual is not None or z is not None:
        e = B.muon_epilogue(act, 0, None if bias is None else _vector("bias", bias, fout, dev))
        if residual is not None:
            e.ld_add = _matrix("residual", residual, dtype, dev, n, fout)
            e.add = residual.data_ptr()
        if z is not None:
            e.ld_z = _matrix("preact_out", z, dtype, dev, n, fout)
            e.z = z.data_ptr()
    d = B.muon_linear(n, fin, fout, ld_x, ld_w, ld_y, code, lay)
    _run_linear(B.MUON_LINEAR_FORWARD, B.muon_linear_forward, "linear_forward", d, x, w, e, out, device, dev)
    return out if z is None else (out, z)


def linear_grad_input(dy, w, preact=None, activation="none", add=None, weight_layout="in_out", out=None):
    """dx = (dy w^T) * act'(preact) + add. With an activation, `preact` is the
    pre-activation that made this layer's x (x = act(preact)), and dx is its
    gradient. `out` may be `add` itself, unless that is another input too."""
    dtype, device, dev = _first("dy", dy)
    code = _linear_type("dy", dtype)
    act = _choice(ACTIVATIONS, activation, "activation")
    lay, fin, fout = _weight(w, weight_layout)
    ld_y = _matrix("dy", dy, dtype, dev, -1, fout)
    ld_w = _matrix("w", w, dtype, dev)
    n = dy.shape[0]
    if out is None:
        out = dy.new_empty((n, fin))
        ld_x = fin
    else:
        ld_x = _matrix("out", out, dtype, dev, n, fin)
    e = None
    if act or add is not None:
        e = B.muon_epilogue(act, 0)
        if add is not None:
            e.ld_add = _matrix("add", add, dtype, dev, n, fin)
            e.add = add.data_ptr()
        if act:
            if preact is None:
                raise ValueError("linear_grad_input: an activation needs its preact")
            e.ld_z = _matrix("preact", preact, dtype, dev, n, fin)
            e.z = preact.data_ptr()
    d = B.muon_linear(n, fin, fout, ld_x, ld_w, ld_y, code, lay)
    _run_linear(B.MUON_LINEAR_GRAD_INPUT, B.muon_linear_grad_input, "linear_grad_input", d, dy, w, e, out, device, dev)
    return out


def _run_linear(op, call, what, d, a, w, e, out, device, dev):
    pa, pw, po = a.data_ptr(), w.data_ptr(), out.data_ptr()
    # most calls need no workspace
    s = _on(dev, call, d, pa, pw, e, po, 0, 0)
    if s == B.MUON_E_WORKSPACE:
        s, nbytes = B.muon_linear_workspace_bytes(d, op, pa, pw)
        _check(s, what)
        ws, pws = _workspace(nbytes, device)
        s = _on(dev, call, d, pa, pw, e, po, pws, nbytes)
    if s:
        _check(s, what)


def linear_grad_weight(x, dy, dw=None, dbias=None, accumulate=False, weight_layout="in_out"):
    """(dw, dbias): the float32 gradients of a linear layer's weight and bias,
    written to (or with accumulate added to) the tensors given. dbias=True
    allocates one; None leaves the bias gradient out."""
    dtype, device, dev = _first("x", x)
    code = _linear_type("x", dtype)
    lay = _choice(_LAYOUTS, weight_layout, "weight_layout")
    ld_x = _matrix("x", x, dtype, dev)
    n, fin = x.shape
    ld_y = _matrix("dy", dy, dtype, dev, n)
    fout = dy.shape[1]
    r, c = (fin, fout) if lay == B.MUON_WEIGHT_IN_OUT else (fout, fin)
    if accumulate and (dw is None or dbias is True):
        raise ValueError("accumulate needs the tensors to add to")
    if dw is None:
        dw = torch.empty((r, c), dtype=torch.float32, device=device)
    ld_w = _matrix("dw", dw, torch.float32, dev, r, c)
    if dbias is True:
        dbias = torch.empty(fout, dtype=torch.float32, device=device)
    pb = 0 if dbias is None else _vector("dbias", dbias, fout, dev)
    d = B.muon_linear(n, fin, fout, ld_x, ld_w, ld_y, code, lay)
    px, py, pd = x.data_ptr(), dy.data_ptr(), dw.data_ptr()
    s = _on(dev, B.muon_linear_grad_weight, d, px, py, pd, pb, int(accumulate), 0, 0)
    if s == B.MUON_E_WORKSPACE:
        s, nbytes = B.muon_linear_workspace_bytes(d, B.MUON_LINEAR_GRAD_WEIGHT, px, py)
        _check(s, "linear_grad_weight")
        ws, pws = _workspace(nbytes, device)
        s = _on(dev, B.muon_linear_grad_weight, d, px, py, pd, pb, int(accumulate), pws, nbytes)
    if s:
        _check(s, "linear_grad_weight")
    return dw, dbias


def _norm_type(name, dtype):
    if dtype not in _TYPES:
        raise ValueError(f"{name}: dtype {dtype}, expected torch.bfloat16, torch.float16 or torch.float32")
    return _TYPES[dtype]


def layernorm_forward(x, weight=None, bias=None, eps=1e-5, out=None):
    """(y, mean, rstd) of layer norm over the rows of x (bf16, fp16 or fp32);
    weight, bias, mean and rstd are float32."""
    dtype, device, dev = _first("x", x)
    code = _norm_type("x", dtype)
    ld_x = _matrix("x", x, dtype, dev)
    rows, cols = x.shape
    if out is None:
        out = x.new_empty((rows, cols))
        ld_y = cols
    else:
        ld_y = _matrix("out", out, dtype, dev, rows, cols)
    mean = torch.empty(rows, dtype=torch.float32, device=device)
    rstd = torch.empty(rows, dtype=torch.float32, device=device)
    d = B.muon_layernorm(rows, cols, ld_x, ld_y, 0, 0, code, eps)
    s = _on(dev, B.muon_layernorm_forward, d, x.data_ptr(), 0 if weight is None else _vector("weight", weight, cols, dev),
            0 if bias is None else _vector("bias", bias, cols, dev), out.data_ptr(), mean.data_ptr(), rstd.data_ptr())
    if s:
        _check(s, "layernorm_forward")
    return out, mean, rstd


def layernorm_backward(dy, x, mean, rstd, weight=None, add=None, dweight=None, dbias=None, accumulate=False, out=None):
    """(dx, dweight, dbias): the gradient of x, plus `add`, and the float32
    gradients of weight and bias, written to (or with accumulate added to) the
    tensors given; True allocates one, None leaves it out. `out` may be `add`
    itself, unless that is dy or x too."""
    dtype, device, dev = _first("dy", dy)
    code = _norm_type("dy", dtype)
    ld_y = _matrix("dy", dy, dtype, dev)
    rows, cols = dy.shape
    ld_x = _matrix("x", x, dtype, dev, rows, cols)
    pm, pr = _vector("mean", mean, rows, dev), _vector("rstd", rstd, rows, dev)
    pw = 0 if weight is None else _vector("weight", weight, cols, dev)
    ld_a, pa = (0, 0) if add is None else (_matrix("add", add, dtype, dev, rows, cols), add.data_ptr())
    if accumulate and (dweight is True or dbias is True):
        raise ValueError("accumulate needs the tensors to add to")
    if dweight is True:
        dweight = torch.empty(cols, dtype=torch.float32, device=device)
    if dbias is True:
        dbias = torch.empty(cols, dtype=torch.float32, device=device)
    pdw = 0 if dweight is None else _vector("dweight", dweight, cols, dev)
    pdb = 0 if dbias is None else _vector("dbias", dbias, cols, dev)
    if out is None:
        out = dy.new_empty((rows, cols))
        ld_o = cols
    else:
        ld_o = _matrix("out", out, dtype, dev, rows, cols)
    d = B.muon_layernorm(rows, cols, ld_x, ld_y, ld_o, ld_a, code, 0.0)
    nbytes = 0
    if dweight is not None or dbias is not None:
        s, nbytes = B.muon_layernorm_workspace_bytes(d)
        if s:
            _check(s, "layernorm_backward")
    ws, pws = _workspace(nbytes, device)
    s = _on(dev, B.muon_layernorm_backward, d, dy.data_ptr(), x.data_ptr(), pw, pm, pr, pa, out.data_ptr(), pdw, pdb,
            int(accumulate), pws, nbytes)
    if s:
        _check(s, "layernorm_backward")
    return out, dweight, dbias
