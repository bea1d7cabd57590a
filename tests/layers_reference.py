"""The definitions of libgemm_layers.h in 64 bits (torch on the CPU), with the
bounds of what fp32 arithmetic may add to them."""
import math

import torch

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}  # half a step, relative
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
TINY = 2.0 ** -24  # below fp16's smallest normal value a step is 2^-24


def below(z):
    """The normal distribution function, to full relative precision in the lower tail (torch.special.ndtr is 0 there)."""
    return 0.5 * torch.special.erfc(-z / math.sqrt(2))


def act(z, a):
    if a == "relu":
        return torch.where(z > 0, z, 0.0)
    if a == "gelu":
        return z * below(z)
    if a == "silu":
        return z * torch.sigmoid(z)
    return z


def slope(z, a):
    if a == "relu":
        return (z > 0).double()
    if a == "gelu":
        return below(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if a == "silu":
        p = torch.sigmoid(z)
        return p * (1 + z * (1 - p))
    return torch.ones_like(z)


def act_error(z, a):
    """What evaluating the activation in fp32 may add: a relative error of 2^-20 (the polynomial's 5e-7, the
    reciprocal's and three products' roundings) and the exponential's, whose argument is rounded (2^-23 of it)."""
    if a in ("none", "relu"):
        return torch.zeros_like(z)
    arg = z * z / 2 if a == "gelu" else z.abs()
    return act(z, a).abs() * (2.0 ** -20 + 2.0 ** -22 * arg) + 2.0 ** -126


def slope_error(z, a):
    """The same of the slope's two terms; for SiLU 1 - p adds 2^-23 times z p."""
    if a in ("none", "relu"):
        return torch.zeros_like(z)
    if a == "gelu":
        terms = below(z) + (z * torch.exp(-z * z / 2)).abs()
        return terms * (2.0 ** -20 + 2.0 ** -22 * z * z / 2)
    p = torch.sigmoid(z)
    return p * (1 + z.abs()) * (2.0 ** -20 + 2.0 ** -22 * z.abs())


def product(a, b, alpha):
    """(alpha * a b, what fp32 sums in any order may be off by).  16-bit products are exact in fp32; each of K sums and
    the scaling round by 2^-23 of the magnitudes at most."""
    a, b = a.double(), b.double()
    size = abs(alpha) * torch.matmul(a.abs(), b.abs())
    return alpha * torch.matmul(a, b), (a.shape[-1] + 8) * 2.0 ** -23 * size


def rounded(value, error, out):
    """The bound on a stored value: `error` before it is rounded to `out`, and that rounding."""
    return error * (1 + HALF[out]) + HALF[out] * value.abs() + (TINY if out == "f16" else 2.0 ** -126)


def linear(a, b, bias, alpha, activation, beta, residual, out, kept):
    """({"out": value, "z": value}, the same of bounds); z is kept in type `kept`."""
    z, e = product(a, b, alpha)
    if bias is not None:
        z = z + bias.double()
    e = e + 2.0 ** -23 * z.abs()
    y = act(z, activation)
    # no activation's slope passes 1.13
    ey = 1.13 * e + act_error(z, activation)
    if beta:
        y = y + beta * residual.double()
        ey = ey + 2.0 ** -23 * (y.abs() + (beta * residual.double()).abs())
    return {"out": y, "z": z}, {"out": rounded(y, ey, out), "z": rounded(z, e, kept)}


def through(d, e, z, activation, d_bias, beta, out):
    """The gradient d, off by e, taken to the activation's input, and its column sums."""
    s = slope(z.double(), activation)
    y = d * s
    ey = e * s.abs() + d.abs() * slope_error(z.double(), activation) + 2.0 ** -23 * y.abs()
    total = y.sum(0)
    et = ey.sum(0) + (y.shape[0] + 8) * 2.0 ** -23 * y.abs().sum(0)
    if beta:
        total = total + beta * d_bias.double()
        et = et + 2.0 ** -22 * (beta * d_bias.double()).abs()
    return {"out": y, "d_bias": total}, {"out": rounded(y, ey, out), "d_bias": et + 2.0 ** -22 * total.abs() + 2.0 ** -126}


def experts_layer(x, ids, gates, up, down, activation, beta, before, out, kind):
    """up: [experts] of 2H x D, down: of D x H values, 64-bit.  kind: the activations' type."""
    T, D = x.shape
    H = down[0].shape[1]
    pieces = 2.0 ** -16 if kind == "bf16" else 2.0 ** -21  # what two pieces of h leave out
    y, e = torch.zeros(T, D, dtype=torch.float64), torch.zeros(T, D, dtype=torch.float64)
    for t in range(T):
        for j, expert in enumerate(ids[t].tolist()):
            if not 0 <= expert < len(up):
                continue
            h, eh = product(x[t:t + 1], up[expert].t(), 1.0)
            # codes' blocks are scaled, and the eight waves' sums added: two more roundings
            g, eg, m, em = h[:, :H], 1.25 * eh[:, :H], h[:, H:], 1.25 * eh[:, H:]
            ga = act(g, activation)
            ega = 1.13 * eg + act_error(g, activation)
            v = ga * m
            ev = ega * m.abs() + (ga.abs() + ega) * em + 2.0 ** -22 * v.abs()
            w = abs(gates[t, j].item())
            size = torch.matmul(v.abs(), down[expert].abs().t())
            y[t] += gates[t, j].double() * torch.matmul(v, down[expert].t())[0]
            e[t] += w * (torch.matmul(ev, down[expert].abs().t())[0] +
                         (pieces + (H + 64 + ids.shape[1]) * 2.0 ** -22) * size[0])
            # pieces of fp16 below its normal range: steps of 2^-24
            if kind == "f16":
                e[t] += 2.0 ** -24 * down[expert].abs().sum(1)
    if beta:
        y = y + beta * before.double()
        e = e + 2.0 ** -22 * (y.abs() + (beta * before.double()).abs())
    return y, rounded(y, e, out)


USUAL = (3.4445, -4.7750, 2.0315)


def newton_schulz(g, steps, coefficients=None, eps=0.0, rounding=False):
    """The steps in 64 bits, or with the roundings that the header names: X in two fp16 pieces, the products' operands
    (X, A less its mean eigenvalue, and its polynomial) in one, scaled to use fp16's range."""
    x = g.double()
    norm = torch.linalg.matrix_norm(x).item()
    turned = x.shape[0] > x.shape[1]
    x = x.t() if turned else x
    if norm == 0:
        return torch.zeros_like(g.double())
    x = x / max(norm, eps)
    half = (lambda v, s: (v * 2.0 ** s).half().double() * 2.0 ** -s) if rounding else (lambda v, s: v)
    for i in range(steps):
        a, b, c = USUAL if coefficients is None else coefficients[i]
        hi = half(x, 12)
        gram = hi @ hi.t()
        if rounding:
            s = ((x * x).sum() / x.shape[0]).item()
            gram = half(gram - s * torch.eye(x.shape[0], dtype=torch.float64), 12)
            a, b = a + s * (b + s * c), b + 2 * c * s
        poly = half(b * gram + c * (gram @ gram), 8)
        x = a * x + poly @ hi
        if rounding:
            hi = half(x, 12)
            x = hi + half(x - hi, 12)
    return x.t() if turned else x
