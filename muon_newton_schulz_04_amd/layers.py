"""The layer operators of libmuon on torch tensors: the linear layer (matrix
product with bias, activation and residual in its epilogue) with its two
gradients, on 16-bit tensors, on 8-bit ones and for the experts of a mixture,
and layer norm and root-mean-square norm with their backward passes. They make
the gradients that a Muon step reads: `dw` may be a view of the flat gradient
buffer.

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

8-bit matrices are `Fp8` pairs (or any pair) of a torch.float8_e4m3fn or
float8_e5m2 matrix whose rows start 16-byte aligned and float32 scales, one for
each block of 128: [ceil(cols / 128), rows] for activations and gradients,
[ceil(rows / 128), ceil(cols / 128)] for weights.
"""

from __future__ import annotations

from typing import NamedTuple

import torch

from . import binding as B

_TYPES = {torch.bfloat16: B.MUON_TYPE_BF16, torch.float16: B.MUON_TYPE_FP16, torch.float32: B.MUON_TYPE_FP32}
_LAYOUTS = {"in_out": B.MUON_WEIGHT_IN_OUT, "out_in": B.MUON_WEIGHT_OUT_IN}
_EIGHT = {torch.float8_e4m3fn: B.MUON_EIGHT_E4M3, torch.float8_e5m2: B.MUON_EIGHT_E5M2}
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


class Fp8(NamedTuple):
    """An 8-bit matrix and its scales."""
    data: torch.Tensor
    scale: torch.Tensor


def _blocks(n):
    return (n + 127) // 128


def _new_eight(rows, cols, dtype, scale_shape, device):
    """A new 8-bit matrix and its descriptor. Rows start 16-byte aligned; those of many
    rows on whole cache lines, which the large products read best (16384 x 1664 x 6400
    204 us, 1600 with rows of 1600 bytes 220)."""
    ld = (cols + 15) // 16 * 16
    if rows >= 256 and cols > 128:
        ld = (cols + 127) // 128 * 128
    if cols % 16:
        # the last row too goes on to the next multiple of 16
        data = torch.empty(rows, ld, dtype=dtype, device=device)[:, :cols]
    elif ld == cols:
        data = torch.empty(rows, cols, dtype=dtype, device=device)
    else:
        data = torch.empty_strided((rows, cols), (ld, 1), dtype=dtype, device=device)
    scale = torch.empty(*scale_shape, dtype=torch.float32, device=device)
    return Fp8(data, scale), B.muon_eight(data.data_ptr(), scale.data_ptr(), ld, _EIGHT[dtype], 0)


def _eight(name, pair, dev, weight):
    """(descriptor, rows, cols) of an 8-bit matrix argument."""
    try:
        t, scale = pair
    except (TypeError, ValueError):
        raise ValueError(f"{name}: expected a pair of an 8-bit matrix and its scales") from None
    code = _EIGHT.get(t.dtype, -1)
    if code < 0 or weight and code != B.MUON_EIGHT_E4M3:
        raise ValueError(f"{name}: dtype {t.dtype}, expected torch.float8_e4m3fn" +
                         ("" if weight else " or torch.float8_e5m2"))
    ld = _matrix(name, t, t.dtype, dev)
    rows, cols = t.shape
    if rows <= 1:
        ld = (cols + 15) // 16 * 16
    p = t.data_ptr()
    if ld % 16 or p % 16:
        raise ValueError(f"{name}: rows must start 16-byte aligned (stride {ld})")
    end = t.storage_offset() + (rows - 1) * ld + (cols + 15) // 16 * 16
    if cols % 16 and rows and t.untyped_storage().nbytes() < end:
        raise ValueError(f"{name}: the last row's bytes up to the next multiple of 16 are read too, and lie outside")
    shape = (_blocks(rows), _blocks(cols)) if weight else (_blocks(cols), rows)
    if scale.dtype is not torch.float32 or scale.get_device() != dev:
        _same(f"{name}'s scales", scale, torch.float32, dev)
    if scale.shape != shape or not scale.is_contiguous():
        raise ValueError(f"{name}: scales {tuple(scale.shape)}, expected {list(shape)}, contiguous")
    return B.muon_eight(p, scale.data_ptr(), ld, code), rows, cols


def _eight_type(dtype):
    if dtype not in _EIGHT:
        raise ValueError(f"8-bit type {dtype}, expected torch.float8_e4m3fn or torch.float8_e5m2")
    return dtype


def rmsnorm_forward(x, weight=None, residual=None, eps=1e-5, quantize=None, out=None, residual_out=None):
    """(y, rstd) of root-mean-square norm over the rows of x (bf16, fp16 or fp32),
    or with a residual (y, rstd, r) of r = x + residual, rounded to x's type: the
    new residual stream, in `residual_out` if given (x or residual itself, for
    one). weight and rstd are float32. With quantize (torch.float8_e4m3fn or
    float8_e5m2) y is an Fp8 of the unrounded values, and x's type's y is written
    too if `out` is given."""
    dtype, device, dev = _first("x", x)
    code = _norm_type("x", dtype)
    ld_x = _matrix("x", x, dtype, dev)
    rows, cols = x.shape
    ld_a = ld_r = pa = pr = ld_y = py = 0
    if residual is not None:
        ld_a, pa = _matrix("residual", residual, dtype, dev, rows, cols), residual.data_ptr()
        if residual_out is None:
            residual_out = torch.empty(rows, cols, dtype=dtype, device=device)
            ld_r = cols
        else:
            ld_r = _matrix("residual_out", residual_out, dtype, dev, rows, cols)
        pr = residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    y = q = None
    if quantize is not None:
        y, q = _new_eight(rows, cols, _eight_type(quantize), (_blocks(cols), rows), device)
    elif out is None:
        out = torch.empty(rows, cols, dtype=dtype, device=device)
    if out is not None:
        ld_y, py = _matrix("out", out, dtype, dev, rows, cols), out.data_ptr()
    if y is None:
        y = out
    rstd = torch.empty(rows, dtype=torch.float32, device=device)
    d = B.muon_rmsnorm(rows, cols, ld_x, ld_a, ld_r, ld_y, 0, code, eps)
    pw = 0 if weight is None else _vector("weight", weight, cols, dev)
    s = _on(dev, B.muon_rmsnorm_forward, d, x.data_ptr(), pa, pw, pr, py, q, rstd.data_ptr())
    if s:
        _check(s, "rmsnorm_forward")
    return (y, rstd) if residual is None else (y, rstd, residual_out)


def rmsnorm_backward(dy, x, rstd, weight=None, add=None, dweight=None, accumulate=False, out=None):
    """(dx, dweight): the gradient of x (what the norm was taken of: with a
    residual, the r that the forward pass returned), plus `add`, and the float32
    gradient of weight, written to (or with accumulate added to) the tensor given;
    True allocates one, None leaves it out. `out` may be `add` itself, unless that
    is dy or x too."""
    dtype, device, dev = _first("dy", dy)
    code = _norm_type("dy", dtype)
    ld_y = _matrix("dy", dy, dtype, dev)
    rows, cols = dy.shape
    ld_x = _matrix("x", x, dtype, dev, rows, cols)
    pr = _vector("rstd", rstd, rows, dev)
    pw = 0 if weight is None else _vector("weight", weight, cols, dev)
    ld_a, pa = (0, 0) if add is None else (_matrix("add", add, dtype, dev, rows, cols), add.data_ptr())
    if dweight is True:
        if accumulate:
            raise ValueError("accumulate needs the tensor to add to")
        dweight = torch.empty(cols, dtype=torch.float32, device=device)
    pdw = 0 if dweight is None else _vector("dweight", dweight, cols, dev)
    if out is None:
        out = torch.empty(rows, cols, dtype=dtype, device=device)
        ld_o = cols
    else:
        ld_o = _matrix("out", out, dtype, dev, rows, cols)
    d = B.muon_rmsnorm(rows, cols, ld_x, ld_a, 0, ld_y, ld_o, code, 0.0)
    nbytes = 0
    if dweight is not None:
        s, nbytes = B.muon_rmsnorm_workspace_bytes(d)
        if s:
            _check(s, "rmsnorm_backward")
    ws, pws = _workspace(nbytes, device)
    s = _on(dev, B.muon_rmsnorm_backward, d, dy.data_ptr(), x.data_ptr(), pw, pr, pa, out.data_ptr(), pdw,
            int(accumulate), pws, nbytes)
    if s:
        _check(s, "rmsnorm_backward")
    return out, dweight


def quantize_fp8(x, dtype=torch.float8_e4m3fn):
    """x [rows, cols] (bf16, fp16 or fp32; an activation or a gradient) as Fp8, a
    scale for each 128 columns of a row."""
    kind, device, dev = _first("x", x)
    code = _norm_type("x", kind)
    ld = _matrix("x", x, kind, dev)
    rows, cols = x.shape
    y, q = _new_eight(rows, cols, _eight_type(dtype), (_blocks(cols), rows), device)
    s = _on(dev, B.muon_quantize, rows, cols, ld, code, x.data_ptr(), q)
    if s:
        _check(s, "quantize_fp8")
    return y


def quantize_fp8_weight(w, weight_layout="in_out", transpose=False):
    """(w8, w8_t) of a weight (bf16, fp16 or fp32: a view of the flat parameters as
    it is) in float8_e4m3fn, a scale for each 128 x 128: w8 [out, in] for
    linear_fp8_forward and, with transpose, w8_t [in, out] for
    linear_fp8_grad_input, else None."""
    kind, device, dev = _first("w", w)
    code = _norm_type("w", kind)
    lay, fin, fout = _weight(w, weight_layout)
    ld = _matrix("w", w, kind, dev)
    rows, cols = w.shape
    w8, q = _new_eight(fout, fin, torch.float8_e4m3fn, (_blocks(fout), _blocks(fin)), device)
    w8_t = q_t = None
    if transpose:
        w8_t, q_t = _new_eight(fin, fout, torch.float8_e4m3fn, (_blocks(fin), _blocks(fout)), device)
    if lay == B.MUON_WEIGHT_IN_OUT:
        q, q_t = q_t, q
    s = _on(dev, B.muon_quantize_weight, rows, cols, ld, code, w.data_ptr(), q, q_t)
    if s:
        _check(s, "quantize_fp8_weight")
    return w8, w8_t


def linear_fp8_forward(x, w, bias=None, residual=None, activation="none", save_preact=False, dtype=torch.bfloat16,
                       out=None, preact_out=None):
    """y = act(x w^T + bias) + residual in `dtype` (bf16 or fp16) of 8-bit x [tokens,
    in] and w [out, in]; with save_preact (or preact_out) also z = x w^T + bias
    rounded to it: returns y, or (y, z). `out` may be `residual` itself. Each 8
    products of consecutive k are summed to 13 bits below the largest of them, the
    rest in float32."""
    _, device, dev = _first("x", x[0])
    code = _linear_type("dtype", dtype)
    act = _choice(ACTIVATIONS, activation, "activation")
    a, n, fin = _eight("x", x, dev, False)
    b, fout, k = _eight("w", w, dev, True)
    if k != fin:
        raise ValueError(f"w: {k} in features, expected {fin}")
    z = preact_out
    if z is None and save_preact:
        z = torch.empty(n, fout, dtype=dtype, device=device)
    if out is None:
        out = torch.empty(n, fout, dtype=dtype, device=device)
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
    d = B.muon_linear(n, fin, fout, 0, 0, ld_y, code, B.MUON_WEIGHT_OUT_IN)
    s = _on(dev, B.muon_linear_scaled_forward, d, a, b, e, out.data_ptr())
    if s:
        _check(s, "linear_fp8_forward")
    return out if z is None else (out, z)


def linear_fp8_grad_input(dy, w, preact=None, activation="none", add=None, dtype=torch.bfloat16, out=None):
    """dx = (dy w^T) * act'(preact) + add in `dtype` (bf16 or fp16) of 8-bit dy
    [tokens, out] and w [in, out], as linear_grad_input. `out` may be `add`
    itself."""
    _, device, dev = _first("dy", dy[0])
    code = _linear_type("dtype", dtype)
    act = _choice(ACTIVATIONS, activation, "activation")
    a, n, fout = _eight("dy", dy, dev, False)
    b, fin, k = _eight("w", w, dev, True)
    if k != fout:
        raise ValueError(f"w: {k} out features, expected {fout}")
    if out is None:
        out = torch.empty(n, fin, dtype=dtype, device=device)
        ld_x = fin
    else:
        ld_x = _matrix("out", out, dtype, dev, n, fin)
    e = _grad_epilogue("linear_fp8_grad_input", act, preact, add, dtype, dev, n, fin)
    d = B.muon_linear(n, fin, fout, ld_x, 0, 0, code, B.MUON_WEIGHT_IN_OUT)
    s = _on(dev, B.muon_linear_scaled_grad_input, d, a, b, e, out.data_ptr())
    if s:
        _check(s, "linear_fp8_grad_input")
    return out


def _grad_epilogue(what, act, preact, add, dtype, dev, n, fin):
    """The epilogue of an input gradient, or None."""
    if not act and add is None:
        return None
    e = B.muon_epilogue(act, 0)
    if add is not None:
        e.ld_add = _matrix("add", add, dtype, dev, n, fin)
        e.add = add.data_ptr()
    if act:
        if preact is None:
            raise ValueError(f"{what}: an activation needs its preact")
        e.ld_z = _matrix("preact", preact, dtype, dev, n, fin)
        e.z = preact.data_ptr()
    return e


def _experts(name, w, dtype, dev, layout, shape=None):
    """(layout code, experts, in, out, row stride, expert stride) of the experts'
    weights, [experts, in, out] or [experts, out, in]."""
    lay = _choice(_LAYOUTS, layout, "weight_layout")
    if w.dim() != 3 or shape is not None and tuple(w.shape) != shape:
        raise ValueError(f"{name}: shape {tuple(w.shape)}, expected " +
                         ("[experts, rows, cols]" if shape is None else str(list(shape))))
    _same(name, w, dtype, dev)
    n, a, b = w.shape
    s0, s1, s2 = w.stride()
    if s2 != 1 and b > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    if a <= 1:
        s1 = b
    if n <= 1:
        s0 = a * s1
    if s1 < b or s0 < (a - 1) * s1 + b:
        raise ValueError(f"{name}: rows overlap (strides {s0}, {s1}, length {b})")
    return (lay, n, a, b, s1, s0) if lay == B.MUON_WEIGHT_IN_OUT else (lay, n, b, a, s1, s0)


def _offsets(offsets, experts, dev):
    """Address of the experts' row offsets, after their checks."""
    _same("offsets", offsets, torch.int32, dev)
    if experts >= 0 and offsets.shape != (experts + 1,) or offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError(f"offsets: shape {tuple(offsets.shape)}, expected "
                         f"[{'experts + 1' if experts < 0 else experts + 1}]")
    if offsets.stride(0) != 1:
        raise ValueError("offsets: must be contiguous")
    return offsets.data_ptr()


def _expert_vectors(name, t, experts, n, dev):
    """Address of contiguous float32 vectors, one an expert."""
    _same(name, t, torch.float32, dev)
    if t.shape != (experts, n) or not t.is_contiguous():
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [{experts}, {n}], contiguous")
    return t.data_ptr()


def grouped_linear_forward(x, w, offsets, bias=None, residual=None, activation="none", weight_layout="in_out",
                           save_preact=False, out=None, preact_out=None):
    """linear_forward of a mixture's experts on rows grouped by expert: rows
    offsets[e] .. offsets[e + 1] - 1 of x [rows, in] go through w[e] and bias[e].
    w: [experts, in, out] or [experts, out, in], bias [experts, out], offsets int32
    [experts + 1], ascending, on the device, where they are read. Rows of no expert
    (a padded batch's) are left as they are: unset, in an `out` that the call
    allocates."""
    dtype, device, dev = _first("x", x)
    code = _linear_type("x", dtype)
    act = _choice(ACTIVATIONS, activation, "activation")
    lay, n_e, fin, fout, ld_w, step = _experts("w", w, dtype, dev, weight_layout)
    po = _offsets(offsets, n_e, dev)
    ld_x = _matrix("x", x, dtype, dev, -1, fin)
    n = x.shape[0]
    z = preact_out
    if z is None and save_preact:
        z = torch.empty(n, fout, dtype=dtype, device=device)
    if out is None:
        out = torch.empty(n, fout, dtype=dtype, device=device)
        ld_y = fout
    else:
        ld_y = _matrix("out", out, dtype, dev, n, fout)
    e = None
    if act or bias is not None or residual is not None or z is not None:
        e = B.muon_epilogue(act, 0, None if bias is None else _expert_vectors("bias", bias, n_e, fout, dev))
        if residual is not None:
            e.ld_add = _matrix("residual", residual, dtype, dev, n, fout)
            e.add = residual.data_ptr()
        if z is not None:
            e.ld_z = _matrix("preact_out", z, dtype, dev, n, fout)
            e.z = z.data_ptr()
    d = B.muon_grouped(n, n_e, fin, fout, ld_x, ld_w, ld_y, step, code, lay)
    s = _on(dev, B.muon_grouped_linear_forward, d, x.data_ptr(), w.data_ptr(), po, e, out.data_ptr())
    if s:
        _check(s, "grouped_linear_forward")
    return out if z is None else (out, z)


def grouped_linear_grad_input(dy, w, offsets, preact=None, activation="none", add=None, weight_layout="in_out",
                              out=None):
    """linear_grad_input of a mixture's experts, rows as grouped_linear_forward's."""
    dtype, device, dev = _first("dy", dy)
    code = _linear_type("dy", dtype)
    act = _choice(ACTIVATIONS, activation, "activation")
    lay, n_e, fin, fout, ld_w, step = _experts("w", w, dtype, dev, weight_layout)
    po = _offsets(offsets, n_e, dev)
    ld_y = _matrix("dy", dy, dtype, dev, -1, fout)
    n = dy.shape[0]
    if out is None:
        out = torch.empty(n, fin, dtype=dtype, device=device)
        ld_x = fin
    else:
        ld_x = _matrix("out", out, dtype, dev, n, fin)
    e = _grad_epilogue("grouped_linear_grad_input", act, preact, add, dtype, dev, n, fin)
    d = B.muon_grouped(n, n_e, fin, fout, ld_x, ld_w, ld_y, step, code, lay)
    s = _on(dev, B.muon_grouped_linear_grad_input, d, dy.data_ptr(), w.data_ptr(), po, e, out.data_ptr())
    if s:
        _check(s, "grouped_linear_grad_input")
    return out


def grouped_linear_grad_weight(x, dy, offsets, dw=None, dbias=None, accumulate=False, weight_layout="in_out"):
    """(dw, dbias): the float32 gradients of the experts' weights [experts, in, out]
    (or [experts, out, in]; `count` matrices of a Muon table's entry, where dw is a
    view of the flat gradient buffer) and biases [experts, out], written to (or with
    accumulate added to) the tensors given. dbias=True allocates one; None leaves it
    out. Zeros (or unchanged) for experts without rows."""
    dtype, device, dev = _first("x", x)
    code = _linear_type("x", dtype)
    lay = _choice(_LAYOUTS, weight_layout, "weight_layout")
    po = _offsets(offsets, -1, dev)
    n_e = offsets.shape[0] - 1
    ld_x = _matrix("x", x, dtype, dev)
    n, fin = x.shape
    ld_y = _matrix("dy", dy, dtype, dev, n)
    fout = dy.shape[1]
    shape = (n_e, fin, fout) if lay == B.MUON_WEIGHT_IN_OUT else (n_e, fout, fin)
    if accumulate and (dw is None or dbias is True):
        raise ValueError("accumulate needs the tensors to add to")
    if dw is None:
        dw = torch.empty(shape, dtype=torch.float32, device=device)
    ld_w, step = _experts("dw", dw, torch.float32, dev, weight_layout, shape)[4:]
    if dbias is True:
        dbias = torch.empty((n_e, fout), dtype=torch.float32, device=device)
    pb = 0 if dbias is None else _expert_vectors("dbias", dbias, n_e, fout, dev)
    d = B.muon_grouped(n, n_e, fin, fout, ld_x, ld_w, ld_y, step, code, lay)
    px, py, pd = x.data_ptr(), dy.data_ptr(), dw.data_ptr()
    s = _on(dev, B.muon_grouped_linear_grad_weight, d, px, py, po, pd, pb, int(accumulate), 0, 0)
    if s == B.MUON_E_WORKSPACE:
        s, nbytes = B.muon_grouped_linear_workspace_bytes(d, px, py)
        _check(s, "grouped_linear_grad_weight")
        ws, pws = _workspace(nbytes, device)
        s = _on(dev, B.muon_grouped_linear_grad_weight, d, px, py, po, pd, pb, int(accumulate), pws, nbytes)
    if s:
        _check(s, "grouped_linear_grad_weight")
    return dw, dbias
