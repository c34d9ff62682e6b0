"""Helpers of the tests of the 8-bit and grouped layer operators: 8-bit floating
point from its definition in 64 bits, inputs, and comparisons."""

import math

import torch

T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
BITS = {"e4m3": (3, -6), "e5m2": (2, -14)}  # stored bits of the significand, lowest exponent
SMALLEST = 2.0 ** -110
U = 2.0 ** -24


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rand(g, shape, dtype, std=1.0, stride=None, mean=0.0):
    """A [rows, cols] GPU tensor with the given row stride; the gap between rows
    holds NaN, which no result may pick up."""
    r, c = shape
    v = (torch.randn(r, c, generator=g) * std + mean).to(dtype)
    buf = torch.full((r, stride or c), float("nan"), dtype=dtype)
    buf[:, :c] = v
    return buf.cuda()[:, :c]


def cpu64(t):
    return t.double().cpu()


def nearest8(v, fmt):
    """The 8-bit value nearest to each of v (float64), ties to even."""
    bits, low = BITS[fmt]
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=low) - bits)
    return (v / step).round() * step


def half_step8(v, fmt):
    """Half the distance between neighbouring 8-bit values around v."""
    bits, low = BITS[fmt]
    _, e = torch.frexp(v.abs() * (1 + 2.0 ** -20))
    return torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=low) - bits) / 2


def blocks(n):
    return -(-n // 128)


def amax64(v, tall):
    """Largest magnitudes of blocks of `tall` x 128, [row blocks, column blocks]."""
    r, c = v.shape
    p = torch.zeros(-(-r // tall) * tall, blocks(c) * 128, dtype=v.dtype)
    p[:r, :c] = v
    return p.view(p.shape[0] // tall, tall, blocks(c), 128).abs().amax(3).amax(1)


def spread(s, tall, rows, cols):
    """Blocks' values as one for each element."""
    return s.repeat_interleave(tall, 0)[:rows].repeat_interleave(128, 1)[:, :cols]


def values(pair, weight=False):
    """What an 8-bit matrix stands for, in float64."""
    q, s = pair
    s = cpu64(s) if weight else cpu64(s).t()
    return cpu64(q.float()) * spread(s, 128 if weight else 1, *q.shape)


def eight(g, rows, cols, fmt="e4m3", std=1.0, weight=False, stride=None):
    """An 8-bit matrix made without the library: random values, scales that differ
    from block to block, rows off into NaN past their end."""
    ld = stride or (cols + 15) // 16 * 16
    buf = torch.full((rows, ld), 0x7F, dtype=torch.uint8)  # NaN in both formats
    v = (torch.randn(rows, cols, generator=g) * LARGEST[fmt] / 16).clamp(-LARGEST[fmt], LARGEST[fmt])
    buf[:, :cols] = v.to(F8[fmt]).view(torch.uint8)
    shape = (blocks(rows), blocks(cols)) if weight else (blocks(cols), rows)
    scale = std * 16 / LARGEST[fmt] * torch.exp(torch.randn(shape, generator=g))
    return buf.cuda().view(F8[fmt])[:, :cols], scale.cuda()


def half_step(want, dtype):
    f = torch.finfo(dtype)
    return want.abs() * f.eps / 2 + f.smallest_normal * f.eps / 2


def close(got, want, tol, dtype):
    """|got - want| within tol and the half step a result tol off may round to."""
    got = got.double().cpu()
    assert got.shape == want.shape
    lim = tol + half_step(want.abs() + tol, dtype)
    # what is half a step or more beyond the type's largest number rounds to infinity
    beyond = (got == want.sign() * math.inf) & (want.abs() + tol >= torch.finfo(dtype).max * (1 + torch.finfo(dtype).eps / 4))
    bad = ~(((got - want).abs() <= lim) | beyond)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} off, worst {float((got - want).abs().max())}, "
                           f"first at {bad.nonzero()[0].tolist()}")


def sum_tol(a, b):
    """Bound on a float32 product's error, from the float64 operands: K terms, exact
    each, in any order of additions, errors independent."""
    k = a.shape[1]
    return (8 + 4 * math.sqrt(k)) * U * (a.abs() @ b.abs())


def act64(name, z):
    if name == "relu":
        return z.clamp(min=0)
    if name == "relu2":
        return z.clamp(min=0) ** 2
    if name == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    if name == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def slope64(name, z):
    if name == "relu":
        return (z > 0).double()
    if name == "relu2":
        return 2 * z.clamp(min=0)
    if name == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        k = 2 * math.sqrt(2 / math.pi)
        q = torch.sigmoid(k * (z + 0.044715 * z ** 3))
        return q + z * q * (1 - q) * k * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        q = torch.sigmoid(z)
        return q + z * q * (1 - q)
    return torch.ones_like(z)


def act_tol(act, z64, ztol):
    """Error of act(z) where z is ztol off: the activations' slopes are at most
    2 |z| (relu2) or 1.2, and each takes about ten float32 steps."""
    slope = 2 * z64.abs() + 1.2 if act == "relu2" else 1.2
    return slope * ztol + 16 * U * (z64.abs() + act64(act, z64).abs())
