"""Cases of the feed-forward layer's operators: a product with bias, activation and residual in its epilogue, its
gradients, a whole layer of experts for a few tokens, and the orthogonalised update of its weights.

`run` computes an operator in elementary torch operations, or, where `own` is
true, through the framework's entry points.  Activations and weights are bf16
or fp16; the experts' weights may be 8-bit codes (OCP E4M3 or E5M2) with an
fp32 scale per 128 x 128 block, scale[expert][k // 128][row // 128].
"""
import math

import torch

own = False

DEVICE = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
COEFFICIENTS = (3.4445, -4.7750, 2.0315)  # of the odd polynomial of degree five that each step applies
EPS = 1e-7


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the second product of a feed-forward layer in one decode step of 16 sequences: bias, and the residual stream added
        dict(name="linear decode 16x4096x16384", op="linear", M=16, N=4096, K=16384, type="bf16", order="nk", act="none",
             bias=True, residual=True, keep=False),
        # the first product in a training step: GELU, its input kept for the gradient
        dict(name="linear train 4096x16384x4096", op="linear", M=4096, N=16384, K=4096, type="bf16", order="nk", act="gelu",
             bias=True, residual=False, keep=True),
        # ragged in every dimension, weights stored along the outputs
        dict(name="linear 4095x4097x1001", op="linear", M=4095, N=4097, K=1001, type="f16", order="kn", act="silu",
             bias=True, residual=True, keep=False),
        # the gradient of the first product's output, through the activation, and its bias's gradient
        dict(name="linear backward 4096x16384x4096", op="linear_backward", M=4096, N=16384, K=4096, type="bf16", order="kn",
             act="gelu", into=0.0),
        # a small one, ragged; the bias's gradient added to what earlier micro-batches left
        dict(name="linear backward 250x1000x515", op="linear_backward", M=250, N=1000, K=515, type="f16", order="nk",
             act="silu", into=1.0),
        # the same gradients where no product makes the incoming one
        dict(name="activation backward 8192x4096", op="activation_backward", M=8192, N=4096, type="bf16", act="gelu", into=0.0),
        dict(name="activation backward 129x4097", op="activation_backward", M=129, N=4097, type="f16", act="relu", into=1.0),
        # the experts of one token: 8 of 64
        dict(name="experts 1 token of 64", op="experts_layer", tokens=1, experts=64, top_k=8, D=4096, H=1024, type="bf16",
             weights="same", act="silu", padded=False, into=0.0),
        # one decode step of 32 sequences, 8-bit weights, a shared expert's output added to
        dict(name="experts 32 tokens of 64, 8 bits", op="experts_layer", tokens=32, experts=64, top_k=8, D=4096, H=1024,
             type="bf16", weights="e4m3", act="silu", padded=False, into=1.0),
        # the updates of the heads of one layer
        dict(name="orthogonalize 16 of 128x128", op="orthogonalize", batch=16, M=128, N=128, type="f32", steps=5, alpha=1.0,
             beta=0.0),
        # a square weight's update
        dict(name="orthogonalize 4096x4096", op="orthogonalize", batch=1, M=4096, N=4096, type="bf16", steps=5, alpha=1.0,
             beta=0.0),
        # tall and ragged, applied to the weights with their decay
        dict(name="orthogonalize 2049x1000 into", op="orthogonalize", batch=1, M=2049, N=1000, type="f32", steps=5,
             alpha=-0.02, beta=0.99),
    ]


def _size(rng, low, high):
    """A size between low and high, spread over its logarithm; every other one odd or ragged."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if rng.random() < 0.5 and n >= 128:
        n = n // 128 * 128
    return max(low, min(high, n))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_backward", "activation_backward", "experts_layer", "orthogonalize"])
    type_, act = rng.choice(["bf16", "bf16", "f16"]), rng.choice(["none", "relu", "gelu", "silu"])
    into = rng.choice([0.0, 1.0])
    if op in ("linear", "linear_backward"):
        c = dict(op=op, M=_size(rng, 1, 4096), N=_size(rng, 64, 8192), K=_size(rng, 64, 4096), type=type_,
                 order=rng.choice(["nk", "nk", "kn"]), act=act)
        if op == "linear":
            return dict(c, bias=rng.random() < 0.75, residual=rng.random() < 0.5, keep=rng.random() < 0.5)
        return dict(c, into=into)
    if op == "activation_backward":
        return dict(op=op, M=_size(rng, 1, 8192), N=_size(rng, 64, 8192), type=type_, act=act, into=into)
    if op == "experts_layer":
        experts = rng.choice([8, 16, 60, 64])
        return dict(op=op, tokens=_size(rng, 1, 64), experts=experts, top_k=rng.choice([k for k in (1, 2, 4, 6, 8) if k <= experts // 2]),
                    D=_size(rng, 256, 4096), H=_size(rng, 128, 2048), type=type_, weights=rng.choice(["same", "same", "e4m3", "e5m2"]),
                    act=rng.choice(["gelu", "silu", "silu"]), padded=rng.random() < 0.3, into=into)
    batch = rng.choice([1, 1, 1, 4, 12])
    return dict(op=op, batch=batch, M=_size(rng, 16, 2048 // (1 if batch == 1 else 4)), N=_size(rng, 16, 2048 // (1 if batch == 1 else 4)),
                type=rng.choice(["f32", "bf16"]), steps=rng.choice([5, 5, 6]), alpha=rng.choice([1.0, -0.02]),
                beta=rng.choice([0.0, 0.99]))


# ---------------------------------------------------------------- inputs
def _activations(rows, cols, g):
    """Features of unlike sizes, a few of them large, and tokens of unlike sizes."""
    feature = torch.exp(0.6 * torch.randn(cols, device=DEVICE, generator=g))
    token = torch.exp(0.4 * torch.randn(rows, 1, device=DEVICE, generator=g))
    return torch.randn(rows, cols, device=DEVICE, generator=g) * feature * token


def _codes(w, fmt):
    """Weights (experts x rows x K) as bytes in rows of a multiple of 16, and a scale for each block of 128 x 128."""
    E, R, K = w.shape
    v = torch.nn.functional.pad(w, (0, -K % 128, 0, -R % 128)).view(E, -(-R // 128), 128, -(-K // 128), 128)
    scale = (v.abs().amax(dim=(2, 4)) / LARGEST[fmt]).clamp(min=2.0 ** -126)
    q = (v / scale[:, :, None, :, None]).to(F8[fmt]).view(E, v.shape[1] * 128, v.shape[3] * 128)[:, :R, :K]
    codes = torch.zeros(E, R, -(-K // 16) * 16, dtype=torch.uint8, device=w.device)
    codes[:, :, :K] = q.contiguous().view(torch.uint8)
    return codes, scale.transpose(1, 2).contiguous()


def _expert_weights(s, name, E, R, K, c, g):
    """Rows start at a multiple of 16 bytes."""
    parts = [0.02 * torch.randn(R, K, device=DEVICE, generator=g) for _ in range(E)]
    if c["weights"] == "same":
        w = torch.zeros(E, R, -(-K // 8) * 8, dtype=TYPES[c["type"]], device=DEVICE)
        for e, p in enumerate(parts):
            w[e, :, :K] = p
        s[name] = w
    else:
        coded = [_codes(p[None], c["weights"]) for p in parts]
        s[name], s[name + "_scale"] = (torch.cat([q[i] for q in coded]) for i in (0, 1))


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    s = {"case": c}
    op = c["op"]
    t = TYPES[c["type"]]
    randn = lambda *shape: torch.randn(*shape, device=DEVICE, generator=g)  # noqa: E731
    empty = lambda *shape, dtype=t: torch.zeros(*shape, dtype=dtype, device=DEVICE)  # noqa: E731
    if op in ("linear", "linear_backward"):
        M, N, K = c["M"], c["N"], c["K"]
        s["b"] = (K ** -0.5 * (randn(N, K) if c["order"] == "nk" else randn(K, N))).to(t)
        s["out"] = empty(M, N)
        if op == "linear":
            s["a"] = _activations(M, K, g).to(t)
            s["bias"] = (0.1 * randn(N)).to(t) if c["bias"] else None
            s["residual"] = _activations(M, N, g).to(t) if c["residual"] else None
            s["z"] = empty(M, N) if c["keep"] else None
    if op in ("linear_backward", "activation_backward"):
        M, N = c["M"], c["N"]
        s["d"] = (0.01 * _activations(M, c["K"] if op == "linear_backward" else N, g)).to(t)
        s["z"] = randn(M, N).to(t)
        s["out"] = empty(M, N)
        s["d_bias"] = empty(N, dtype=torch.float32)
        s["d_bias_before"] = 0.1 * randn(N) if c["into"] else None
    if op == "experts_layer":
        T, E, k, D, H = c["tokens"], c["experts"], c["top_k"], c["D"], c["H"]
        # rows of a multiple of 16 bytes, as the weights' are
        s["x"] = empty(T, -(-D // 8) * 8)
        s["x"][:, :D] = _activations(T, D, g)
        best = torch.sort(1.5 * randn(T, E), dim=1, descending=True)
        s["ids"] = best.indices[:, :k].to(torch.int32).contiguous()
        s["gates"] = torch.softmax(best.values[:, :k], 1).contiguous()
        if c["padded"]:  # the tokens of sequences that have ended
            gone = torch.rand(T, device=DEVICE, generator=g) < 0.25
            s["ids"][gone] = -1
            s["gates"][gone] = 0
        _expert_weights(s, "up", E, 2 * H, D, c, g)
        _expert_weights(s, "down", E, D, H, c, g)
        s["out"] = empty(T, D)
        s["before"] = _activations(T, D, g).to(t) if c["into"] else None
    if op == "orthogonalize":
        b, M, N = c["batch"], c["M"], c["N"]
        # a momentum: a few directions that most steps agree on, and noise
        r = max(1, min(M, N) // 16)
        s["g"] = (1e-3 * (torch.bmm(randn(b, M, r), randn(b, r, N)) * (2.0 / r) ** 0.5 + randn(b, M, N))).to(t)
        s["before"] = (0.02 * randn(b, M, N)).bfloat16() if c["beta"] else None
        s["out"] = empty(b, M, N, dtype=torch.bfloat16)
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    if own:
        return globals()["_own_" + c["op"]](s, c)
    return globals()["_plain_" + c["op"]](s, c)


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "gelu":  # z times the normal distribution's mass below z
        return 0.5 * z * torch.erfc(-z * math.sqrt(0.5))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * torch.erfc(-z * math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    return torch.ones_like(z)


def _plain_product(a, b, order):
    b = b.float()
    return torch.matmul(a.float(), b.t() if order == "nk" else b)


def _plain_linear(s, c):
    t = TYPES[c["type"]]
    z = _plain_product(s["a"], s["b"], c["order"])
    if c["bias"]:
        z = z + s["bias"].float()
    y = _act(z, c["act"])
    if c["residual"]:
        y = y + s["residual"].float()
    return {"out": y.to(t), "z": z.to(t)} if c["keep"] else {"out": y.to(t)}


def _plain_through(d, s, c):
    """The gradient d of an activation's output taken to its input and its bias."""
    d = d * _act_slope(s["z"].float(), c["act"])
    d_bias = d.sum(0)
    if c["into"]:
        d_bias = d_bias + c["into"] * s["d_bias_before"]
    return {"out": d.to(s["out"].dtype), "d_bias": d_bias}


def _plain_linear_backward(s, c):
    return _plain_through(_plain_product(s["d"], s["b"], c["order"]), s, c)


def _plain_activation_backward(s, c):
    return _plain_through(s["d"].float(), s, c)


def _plain_weights(s, name, c, rows, K, chosen):
    """The weights of all experts, or of the chosen ones, in fp32."""
    w = s[name] if chosen is None else s[name].index_select(0, chosen)
    w = w[:, :, :K]
    if c["weights"] == "same":
        return w.float()
    scale = s[name + "_scale"] if chosen is None else s[name + "_scale"].index_select(0, chosen)
    scale = scale.transpose(1, 2).repeat_interleave(128, 1)[:, :rows].repeat_interleave(128, 2)[:, :, :K]
    return w.view(F8[c["weights"]]).float() * scale


def _plain_experts_layer(s, c):
    T, E, k, D, H = c["tokens"], c["experts"], c["top_k"], c["D"], c["H"]
    x, ids = s["x"][:, :D].float(), s["ids"].long()
    gates = torch.where(ids >= 0, s["gates"], 0.0)
    few = 2 * T * k <= E  # a copy of each slot's expert, or all experts for all tokens
    chosen = ids.clamp(min=0).view(-1) if few else None
    up = _plain_weights(s, "up", c, 2 * H, D, chosen).transpose(1, 2)
    down = _plain_weights(s, "down", c, D, H, chosen).transpose(1, 2)
    h = torch.matmul(x.repeat_interleave(k, 0)[:, None] if few else x, up)
    h = _act(h[..., :H], c["act"]) * h[..., H:]
    if few:
        y = torch.matmul(h, down).view(T, k, D)
        y = (y * gates[..., None]).sum(1)
    else:
        share = torch.zeros(T, E, device=x.device).scatter_add_(1, ids.clamp(min=0), gates)
        h = (h * share.t()[..., None]).transpose(0, 1).reshape(T, E * H)
        y = torch.matmul(h, down.reshape(E * H, D))
    if c["into"]:
        y = y + c["into"] * s["before"].float()
    return y.to(s["out"].dtype)


def _plain_orthogonalize(s, c):
    x = s["g"].float()
    norm = torch.sqrt(torch.sum(x * x, dim=(1, 2), keepdim=True))
    x = x / torch.clamp(norm, min=EPS)
    wide = c["M"] <= c["N"]
    x = x if wide else x.transpose(1, 2).contiguous()
    p, q, r = COEFFICIENTS
    for _ in range(c["steps"]):
        gram = torch.matmul(x, x.transpose(1, 2))
        x = p * x + torch.matmul(q * gram + r * torch.matmul(gram, gram), x)
    y = c["alpha"] * (x if wide else x.transpose(1, 2))
    if c["beta"]:
        y = y + c["beta"] * s["before"].float()
    return y.to(s["out"].dtype)


# ---------------------------------------------------------------- through the framework
def _binding():
    from dense_gemm_optimisation_amd import binding
    return binding


def _input(lib, t):
    return {torch.float32: lib.INPUT_F32, torch.bfloat16: lib.INPUT_BF16, torch.float16: lib.INPUT_F16}[t]


def _output(lib, t):
    return {torch.float32: lib.OUTPUT_F32, torch.bfloat16: lib.OUTPUT_BF16, torch.float16: lib.OUTPUT_F16}[t]


def _activation(lib, act):
    return {"none": lib.ACT_NONE, "relu": lib.ACT_RELU, "gelu": lib.ACT_GELU, "silu": lib.ACT_SILU}[act]


def _workspace(s, size):
    """Made once, as a user's program keeps it from call to call."""
    if "workspace" not in s:
        s["workspace"] = torch.empty(max(1, size), dtype=torch.uint8, device=DEVICE)
    return s["workspace"].data_ptr(), s["workspace"].numel()


def _at(t):
    return (0, 0) if t is None else (t.data_ptr(), t.stride(0))


def _own_linear(s, c):
    lib = _binding()
    M, N, K = c["M"], c["N"], c["K"]
    a, b, out = s["a"], s["b"], s["out"]
    order = lib.COL_MAJOR if c["order"] == "nk" else lib.ROW_MAJOR
    space = _workspace(s, lib.linear_workspace_size(M, N, K))
    lib.gemm_linear(M, N, K, 1.0, a.data_ptr(), a.stride(0), b.data_ptr(), b.stride(0), order, _input(lib, a.dtype),
                    0 if s["bias"] is None else s["bias"].data_ptr(), _activation(lib, c["act"]),
                    1.0 if c["residual"] else 0.0, *_at(s["residual"]), out.data_ptr(), out.stride(0), _output(lib, out.dtype),
                    *_at(s["z"]), *space)
    return {"out": out, "z": s["z"]} if c["keep"] else {"out": out}


def _own_linear_backward(s, c):
    lib = _binding()
    M, N, K = c["M"], c["N"], c["K"]
    d, b, z, out, d_bias = s["d"], s["b"], s["z"], s["out"], s["d_bias"]
    if c["into"]:
        d_bias.copy_(s["d_bias_before"])
    order = lib.COL_MAJOR if c["order"] == "nk" else lib.ROW_MAJOR
    space = _workspace(s, lib.linear_workspace_size(M, N, K))
    lib.gemm_linear_backward(M, N, K, 1.0, d.data_ptr(), d.stride(0), b.data_ptr(), b.stride(0), order, _input(lib, d.dtype),
                             z.data_ptr(), z.stride(0), _activation(lib, c["act"]), out.data_ptr(), out.stride(0),
                             _output(lib, out.dtype), c["into"], d_bias.data_ptr(), *space)
    return {"out": out, "d_bias": d_bias}


def _own_activation_backward(s, c):
    lib = _binding()
    d, z, out, d_bias = s["d"], s["z"], s["out"], s["d_bias"]
    if c["into"]:
        d_bias.copy_(s["d_bias_before"])
    space = _workspace(s, lib.activation_backward_workspace_size(c["M"], c["N"]))
    lib.gemm_activation_backward(c["M"], c["N"], d.data_ptr(), d.stride(0), _input(lib, d.dtype), z.data_ptr(), z.stride(0),
                                 _input(lib, z.dtype), _activation(lib, c["act"]), out.data_ptr(), out.stride(0),
                                 _output(lib, out.dtype), c["into"], d_bias.data_ptr(), *space)
    return {"out": out, "d_bias": d_bias}


def _own_experts_layer(s, c):
    lib = _binding()
    T, E, k, D, H = c["tokens"], c["experts"], c["top_k"], c["D"], c["H"]
    x, out = s["x"], s["out"]
    if c["into"]:
        out.copy_(s["before"])
    weights = {"same": lib.WEIGHTS_SAME, "e4m3": lib.WEIGHTS_E4M3, "e5m2": lib.WEIGHTS_E5M2}[c["weights"]]

    def operand(name):
        w, scale = s[name], s.get(name + "_scale")
        return (w.data_ptr(), w.stride(1), w.stride(0)) + ((0, 0, 0) if scale is None else
                                                          (scale.data_ptr(), scale.stride(1), scale.stride(0)))
    space = _workspace(s, lib.experts_layer_workspace_size(T, E, k, D, H))
    lib.gemm_experts_layer(T, E, k, D, H, x.data_ptr(), x.stride(0), _input(lib, x.dtype), s["ids"].data_ptr(),
                           s["gates"].data_ptr(), weights, *operand("up"), *operand("down"), _activation(lib, c["act"]),
                           c["into"], out.data_ptr(), out.stride(0), _output(lib, out.dtype), *space)
    return out


def _own_orthogonalize(s, c):
    lib = _binding()
    b, M, N = c["batch"], c["M"], c["N"]
    x, out = s["g"], s["out"]
    if c["beta"]:
        out.copy_(s["before"])
    space = _workspace(s, lib.orthogonalize_workspace_size(M, N, b))
    lib.gemm_orthogonalize(M, N, x.data_ptr(), x.stride(1), _input(lib, x.dtype), c["steps"], None, EPS, c["alpha"], c["beta"],
                           out.data_ptr(), out.stride(1), _output(lib, out.dtype), *space, batch=b, stride_g=x.stride(0),
                           stride_o=out.stride(0))
    return out


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    op = c["op"]
    size = {"f32": 4, "bf16": 2, "f16": 2}[c["type"]]
    if op == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": size * ((M + N) * K + N * c["bias"] + M * N * (1 + c["residual"] + c["keep"])), "flops": 2 * M * N * K}
    if op == "linear_backward":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": size * ((M + N) * K + 2 * M * N) + 4 * N * (1 + (c["into"] != 0)), "flops": 2 * M * N * K}
    if op == "activation_backward":
        M, N = c["M"], c["N"]
        return {"bytes": size * 3 * M * N + 4 * N * (1 + (c["into"] != 0)), "flops": 10 * M * N}
    if op == "experts_layer":
        T, E, k, D, H = c["tokens"], c["experts"], c["top_k"], c["D"], c["H"]
        T = 0.75 * T if c["padded"] else T
        live = E * (1 - (1 - k / E) ** T)  # experts that any token chose, on average
        weights = live * 3 * D * H * (size if c["weights"] == "same" else 1 + 4 / 128 ** 2)
        return {"bytes": weights + c["tokens"] * (8 * k + D * size * (2 + (c["into"] != 0))), "flops": T * k * 6 * D * H}
    b, M, N = c["batch"], c["M"], c["N"]
    m, n = min(M, N), max(M, N)
    # of the symmetric products one half
    flops = b * c["steps"] * (m * (m + 1) * n + m * (m + 1) * m + 2 * m * m * n)
    return {"bytes": b * M * N * (size + 2 * (1 + (c["beta"] != 0))), "flops": flops}


# ---------------------------------------------------------------- from the definitions, in 64 bits
def _exact_act(z, act):
    """The activation and its slope."""
    if act == "gelu":
        below = torch.special.ndtr(z)
        return z * below, below + z * torch.exp(-z ** 2 / 2) / math.sqrt(2 * math.pi)
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * torch.sigmoid(-z)
    on = (z > 0) | (act == "none")
    return z * on, on.double()


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    op = c["op"]
    if op == "linear":
        z = torch.mm(s["a"].double(), s["b"].double().t().contiguous() if c["order"] == "nk" else s["b"].double())
        z = z if s["bias"] is None else z + s["bias"].double()
        y = _exact_act(z, c["act"])[0]
        y = y if s["residual"] is None else y + s["residual"].double()
        return {"out": y, "z": z} if c["keep"] else {"out": y}
    if op in ("linear_backward", "activation_backward"):
        d = s["d"].double()
        if op == "linear_backward":
            d = torch.mm(d, s["b"].double().t().contiguous() if c["order"] == "nk" else s["b"].double())
        d = d * _exact_act(s["z"].double(), c["act"])[1]
        total = torch.mv(d.t(), torch.ones(c["M"], dtype=torch.float64, device=DEVICE))
        return {"out": d, "d_bias": total if s["d_bias_before"] is None else total + c["into"] * s["d_bias_before"].double()}
    if op == "experts_layer":
        T, D, H = c["tokens"], c["D"], c["H"]
        y = torch.zeros(T, D, dtype=torch.float64, device=DEVICE)

        def weight(name, e, rows, K):
            w = s[name][e, :, :K]
            if c["weights"] == "same":
                return w.double()
            w = w.contiguous().view(F8[c["weights"]]).double()
            for i in range(0, rows, 128):
                for j in range(0, K, 128):
                    w[i: i + 128, j: j + 128] *= s[name + "_scale"][e, j // 128, i // 128].double()
            return w
        ids = s["ids"].cpu()
        for e in sorted(set(ids.view(-1).tolist()) - {-1}):
            at = (ids == e).nonzero()
            t, j = at[:, 0].to(DEVICE), at[:, 1].to(DEVICE)
            h = torch.mm(s["x"][t, :D].double(), weight("up", e, 2 * H, D).t().contiguous())
            h = _exact_act(h[:, :H], c["act"])[0] * h[:, H:]
            y.index_add_(0, t, s["gates"][t, j, None].double() * torch.mm(h, weight("down", e, D, H).t().contiguous()))
        return y if s["before"] is None else y + c["into"] * s["before"].double()
    out = []
    p, q, r = COEFFICIENTS
    for g in s["g"].double():
        x = g / max(torch.linalg.matrix_norm(g).item(), EPS)
        if c["M"] > c["N"]:
            x = x.t().contiguous()
        for _ in range(c["steps"]):
            gram = torch.mm(x, x.t().contiguous())
            x = p * x + q * torch.mm(gram, x) + r * torch.mm(gram, torch.mm(gram, x))
        out.append(x if c["M"] <= c["N"] else x.t())
    y = c["alpha"] * torch.stack(out)
    return y if s["before"] is None else y + c["beta"] * s["before"].double()
