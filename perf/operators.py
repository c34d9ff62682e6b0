"""The layer operators' measured cases: the linear layer (matrix product with
bias, activation and residual in its epilogue) with its two gradients, and
layer norm with its backward pass, the weight's gradients reduced over rows.

`run` computes a case in its plain form, elementary torch operations in 32
bits rounded once at the end, or, where `own` is set, through
muon_newton_schulz_04_amd.layers. `exact` computes it in 64 bits.
"""

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-5


def _lin(name, op, tokens, fin, fout, dtype, layout, act="none", bias=False, residual=False, save=False,
         accumulate=False):
    return {"name": name, "op": op, "tokens": tokens, "fin": fin, "fout": fout, "dtype": dtype, "layout": layout,
            "act": act, "bias": bias, "residual": residual, "save": save, "accumulate": accumulate}


def _ln(name, op, rows, cols, dtype, residual=False, accumulate=False):
    return {"name": name, "op": op, "rows": rows, "cols": cols, "dtype": dtype, "residual": residual,
            "accumulate": accumulate}


def listed():
    return [
        # serving, one sequence: c_fc of the d = 1600 body for a single token
        _lin("linear_token", "linear", 1, 1600, 6400, "bf16", "in_out", act="gelu_tanh", bias=True),
        # serving, a small batch of sequences: c_proj with the residual stream, torch's [out, in] weights
        _lin("linear_tokens", "linear", 24, 6400, 1600, "fp16", "out_in", bias=True, residual=True),
        # training: c_fc of the d = 1600 body over 16 sequences of 1024, the pre-activation kept for the way back
        _lin("linear_train", "linear", 16384, 1600, 6400, "bf16", "in_out", act="gelu_tanh", bias=True, save=True),
        # a user's own layer of odd sizes on a ragged batch: rows that start on no 16-byte border
        _lin("linear_odd", "linear", 999, 1001, 777, "bf16", "out_in", act="relu2"),
        # training, the way back through c_proj: the gradient of c_fc's pre-activation
        _lin("grad_input_train", "grad_input", 16384, 6400, 1600, "bf16", "in_out", act="gelu_tanh"),
        # the way back through an attention projection of the 124M body on a ragged batch, joined to the residual's gradient
        _lin("grad_input_ragged", "grad_input", 2051, 768, 768, "fp16", "out_in", residual=True),
        # training: c_fc's weight and bias gradient into the flat gradient buffer
        _lin("grad_weight_train", "grad_weight", 16384, 1600, 6400, "bf16", "in_out", bias=True),
        # a later micro-batch of ragged length: an attention projection's gradient added to what is there
        _lin("grad_weight_accumulate", "grad_weight", 1027, 768, 768, "fp16", "out_in", bias=True, accumulate=True),
        # serving: one token's norm
        _ln("layernorm_token", "layernorm", 1, 1600, "bf16"),
        # training: a norm of the d = 1600 body
        _ln("layernorm_train", "layernorm", 16384, 1600, "bf16"),
        # training, its way back, joined to the residual's gradient
        _ln("layernorm_grad_train", "layernorm_grad", 16384, 1600, "bf16", residual=True),
        # fp32 on odd sizes, a later micro-batch
        _ln("layernorm_grad_odd", "layernorm_grad", 4099, 1003, "fp32", accumulate=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _features(rng):
    n = _log(rng, 64, 6400)
    step = rng.choice((64, 64, 8, 8, 1))
    return max(step, n // step * step)


def draw(rng):
    op = rng.choice(("linear", "linear", "grad_input", "grad_weight", "layernorm", "layernorm_grad"))
    flip = lambda: rng.random() < 0.5  # noqa: E731
    if op.startswith("layernorm"):
        cols = _features(rng)
        rows = min(_log(rng, 1, 16384), 16384 * 1600 // cols)
        dtype = rng.choice(("bf16", "fp16", "fp32")) if rows * cols <= 16384 * 800 else rng.choice(("bf16", "fp16"))
        c = _ln("", op, rows, cols, dtype, residual=op == "layernorm_grad" and flip(),
                accumulate=op == "layernorm_grad" and flip())
    else:
        fin, fout = _features(rng), _features(rng)
        tokens = min(_log(rng, 1, 16384), 16384 * 1600 * 6400 // (fin * fout))
        act = rng.choice(("none", "relu", "relu2", "gelu", "gelu_tanh", "silu")) if op != "grad_weight" else "none"
        c = _lin("", op, tokens, fin, fout, rng.choice(("bf16", "fp16")), rng.choice(("in_out", "out_in")), act=act,
                 bias=op != "grad_input" and flip(), residual=op != "grad_weight" and flip(),
                 save=op == "linear" and act != "none" and flip(), accumulate=op == "grad_weight" and flip())
    del c["name"]
    return c


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = TYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=t):
        return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)

    s = {"case": case}
    if case["op"].startswith("layernorm"):
        r, c = case["rows"], case["cols"]
        # a residual stream: channels of unlike sizes around means that are not zero
        scale = torch.rand(c, generator=g, device="cuda") * 2 + 0.2
        s["x"] = (torch.randn(r, c, generator=g, device="cuda") * scale + 0.3 * scale).to(t)
        s["weight"] = normal(c, std=0.2, mean=1.0, dtype=torch.float32)
        s["bias"] = normal(c, std=0.1, dtype=torch.float32)
        if case["op"] == "layernorm_grad":
            x = s["x"].float()
            s["mean"] = x.mean(1)
            s["rstd"] = 1 / ((x - s["mean"][:, None]).square().mean(1) + EPS).sqrt()
            s["dy"] = normal(r, c, std=0.01)
            s["add"] = normal(r, c, std=0.01) if case["residual"] else None
            # the norm's two gradients in the user's flat fp32 buffer
            s["grads"] = normal(2, c, std=0.01, dtype=torch.float32)
        return s
    n, i, o = case["tokens"], case["fin"], case["fout"]
    shape = (i, o) if case["layout"] == "in_out" else (o, i)
    if case["op"] != "grad_weight":
        s["w"] = normal(*shape, std=i ** -0.5)
    if case["op"] == "linear":
        s["x"] = normal(n, i)
        s["bias"] = normal(o, std=0.1, dtype=torch.float32) if case["bias"] else None
        s["residual"] = normal(n, o) if case["residual"] else None
    else:
        s["dy"] = normal(n, o, std=0.01)
    if case["op"] == "grad_input":
        s["preact"] = normal(n, i) if case["act"] != "none" else None
        s["add"] = normal(n, i, std=0.01) if case["residual"] else None
    if case["op"] == "grad_weight":
        s["x"] = normal(n, i)
        s["grads"] = normal(*shape, std=0.01, dtype=torch.float32)
        s["dbias"] = normal(o, std=0.01, dtype=torch.float32) if case["bias"] else None
    return s


def _act(name, z):
    if name == "relu":
        return z.clamp(min=0)
    if name == "relu2":
        return z.clamp(min=0).square()
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "relu2":
        return 2 * z.clamp(min=0)
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        q = 1 / (1 + torch.exp(-z))
        return q * (1 + z * (1 - q))
    return torch.ones_like(z)


def _run_plain(s):
    c = s["case"]
    t = TYPES[c["dtype"]]
    if c["op"] == "linear":
        w = s["w"].float() if c["layout"] == "in_out" else s["w"].float().t()
        z = s["x"].float() @ w
        if c["bias"]:
            z = z + s["bias"]
        y = _act(c["act"], z)
        if c["residual"]:
            y = y + s["residual"].float()
        return (y.to(t), z.to(t)) if c["save"] else y.to(t)
    if c["op"] == "grad_input":
        w = s["w"].float() if c["layout"] == "out_in" else s["w"].float().t()
        dx = s["dy"].float() @ w
        if c["act"] != "none":
            dx = dx * _act_grad(c["act"], s["preact"].float())
        if c["residual"]:
            dx = dx + s["add"].float()
        return dx.to(t)
    if c["op"] == "grad_weight":
        x, dy = s["x"].float(), s["dy"].float()
        dw = x.t() @ dy if c["layout"] == "in_out" else dy.t() @ x
        dw = s["grads"].add_(dw) if c["accumulate"] else s["grads"].copy_(dw)
        if not c["bias"]:
            return dw
        db = dy.sum(0)
        return dw, (s["dbias"].add_(db) if c["accumulate"] else s["dbias"].copy_(db))
    x = s["x"].float()
    if c["op"] == "layernorm":
        mean = x.mean(1)
        d = x - mean[:, None]
        rstd = 1 / (d.square().mean(1) + EPS).sqrt()
        return (d * rstd[:, None] * s["weight"] + s["bias"]).to(t), mean, rstd
    dy = s["dy"].float()
    xh = (x - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["weight"]
    dx = s["rstd"][:, None] * (g - g.mean(1)[:, None] - xh * (g * xh).mean(1)[:, None])
    if c["residual"]:
        dx = dx + s["add"].float()
    d = torch.stack(((dy * xh).sum(0), dy.sum(0)))
    d = s["grads"].add_(d) if c["accumulate"] else s["grads"].copy_(d)
    return dx.to(t), d


def _run_own(s):
    from muon_newton_schulz_04_amd import layers as L

    c = s["case"]
    if c["op"] == "linear":
        return L.linear_forward(s["x"], s["w"], bias=s["bias"], residual=s["residual"], activation=c["act"],
                                weight_layout=c["layout"], save_preact=c["save"])
    if c["op"] == "grad_input":
        return L.linear_grad_input(s["dy"], s["w"], preact=s["preact"], activation=c["act"], add=s["add"],
                                   weight_layout=c["layout"])
    if c["op"] == "grad_weight":
        dw, db = L.linear_grad_weight(s["x"], s["dy"], dw=s["grads"], dbias=s["dbias"], accumulate=c["accumulate"],
                                      weight_layout=c["layout"])
        return (dw, db) if c["bias"] else dw
    if c["op"] == "layernorm":
        return L.layernorm_forward(s["x"], weight=s["weight"], bias=s["bias"], eps=EPS)
    dx, _dw, _db = L.layernorm_backward(s["dy"], s["x"], s["mean"], s["rstd"], weight=s["weight"], add=s["add"],
                                        dweight=s["grads"][0], dbias=s["grads"][1], accumulate=c["accumulate"])
    return dx, s["grads"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    e = 4 if case["dtype"] == "fp32" else 2
    if case["op"].startswith("layernorm"):
        r, c = case["rows"], case["cols"]
        if case["op"] == "layernorm":
            return {"bytes": 2 * e * r * c + 8 * c + 8 * r, "flops": 8 * r * c}
        n = 3 + case["residual"]
        return {"bytes": n * e * r * c + 8 * r + 4 * c * (3 + 2 * case["accumulate"]), "flops": 14 * r * c}
    n, i, o = case["tokens"], case["fin"], case["fout"]
    if case["op"] == "linear":
        b = e * (n * i + i * o + n * o * (1 + case["residual"] + case["save"])) + 4 * o * case["bias"]
    elif case["op"] == "grad_input":
        b = e * (n * o + i * o + n * i * (1 + (case["act"] != "none") + case["residual"]))
    else:
        b = e * n * (i + o) + 4 * (i * o + o * case["bias"]) * (1 + case["accumulate"])
    return {"bytes": b, "flops": 2 * n * i * o}


def exact(case, seed):
    s = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in prepare(case, seed).items()}
    act, op = case["act"] if "act" in case else "none", case["op"]

    def cdf(v):  # the normal distribution's, without cancellation in its tail
        return torch.special.erfc(v * -math.sqrt(0.5)) * 0.5

    def value(z):
        if act == "gelu":
            return z * cdf(z)
        if act == "gelu_tanh":
            return z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))
        if act == "silu":
            return z * torch.sigmoid(z)
        if act in ("relu", "relu2"):
            return torch.where(z > 0, z if act == "relu" else z * z, torch.zeros_like(z))
        return z

    def slope(z):
        if act == "gelu":
            return cdf(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        if act == "gelu_tanh":
            u = math.sqrt(8 / math.pi)
            q = torch.sigmoid(u * (z + 0.044715 * z ** 3))
            return q + z * q * torch.sigmoid(-u * (z + 0.044715 * z ** 3)) * u * (1 + 0.134145 * z * z)
        if act == "silu":
            return torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z)
        return torch.where(z > 0, torch.ones_like(z) if act == "relu" else 2 * z, torch.zeros_like(z))

    def product(a, b):
        return torch.mm(a.contiguous(), b.contiguous())

    if op == "linear":
        z = product(s["x"], s["w"] if case["layout"] == "in_out" else s["w"].T)
        z = z + s["bias"] if case["bias"] else z
        y = value(z) + (s["residual"] if case["residual"] else 0)
        return (y, z) if case["save"] else y
    if op == "grad_input":
        dx = product(s["dy"], s["w"].T if case["layout"] == "in_out" else s["w"])
        dx = dx * slope(s["preact"]) if act != "none" else dx
        return dx + s["add"] if case["residual"] else dx
    if op == "grad_weight":
        dw = product(s["x"].T, s["dy"])
        dw = dw if case["layout"] == "in_out" else dw.T
        dw = dw.contiguous() + (s["grads"] if case["accumulate"] else 0)
        if not case["bias"]:
            return dw
        return dw, s["dy"].sum(0) + (s["dbias"] if case["accumulate"] else 0)
    if op == "layernorm":
        var, mean = torch.var_mean(s["x"], dim=1, correction=0)
        rstd = torch.rsqrt(var + EPS)
        return (s["x"] - mean[:, None]) * (rstd[:, None] * s["weight"]) + s["bias"], mean, rstd
    # dx from the projection of dy w off the row's constant and its normalised values
    n = s["x"].shape[1]
    xh = (s["x"] - s["mean"][:, None]) * s["rstd"][:, None]
    v = s["dy"] * s["weight"]
    dx = (v - v.sum(1, keepdim=True) / n - xh * ((v * xh).sum(1, keepdim=True) / n)) * s["rstd"][:, None]
    dx = dx + s["add"] if case["residual"] else dx
    d = torch.stack(((s["dy"] * xh).sum(0), s["dy"].sum(0)))
    return dx, d + s["grads"] if case["accumulate"] else d
