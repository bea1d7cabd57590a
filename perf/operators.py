"""Cases of the block-scaled 8-bit operators: quantising, the product, the experts' products and their routing.

`run` computes an operator in elementary torch operations, or, where `own` is
true, through the framework's entry points.  8-bit values are kept as bytes
(OCP E4M3 or E5M2); scales are fp32, one per 128 along the contracted
dimension of a row, or per 128 x 128 block; scale k-blocks are the outer
dimension, scale[k // 128][row // block].
"""
import math

import torch

own = False

DEVICE = "cuda"
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the activations of one decode step of 32 sequences, before a projection
        dict(name="quantize decode 32x4096", op="quantize", rows=32, cols=4096, type="bf16", format="e4m3",
             block=1, direct=True, transposed=False, gather=False),
        # a training step's activations: along the features for the forward product, along the tokens for the weights' gradient
        dict(name="quantize train 8192x4096", op="quantize", rows=8192, cols=4096, type="bf16", format="e4m3",
             block=1, direct=True, transposed=True, gather=False),
        # a projection of one decode step of 16 sequences
        dict(name="product decode 16x4096x4096", op="product", M=16, N=4096, K=4096, block_a=1, block_b=128,
             format_a="e4m3", format_b="e4m3", out="bf16"),
        # a projection over a prompt
        dict(name="product 4096x4096x4096", op="product", M=4096, N=4096, K=4096, block_a=1, block_b=128,
             format_a="e4m3", format_b="e4m3", out="bf16"),
        # ragged in every dimension, the last scale block of K not whole
        dict(name="product 4095x4097x1001", op="product", M=4095, N=4097, K=1001, block_a=1, block_b=128,
             format_a="e4m3", format_b="e4m3", out="f16"),
        # a weight's gradient: both operands scaled along the tokens, row by row
        dict(name="product wgrad 4096x4096x8192", op="product", M=4096, N=4096, K=8192, block_a=1, block_b=1,
             format_a="e5m2", format_b="e4m3", out="bf16"),
        # the experts' products of one decode step: 16 tokens, 8 of 64 experts each
        dict(name="experts decode 128 of 64", op="experts", experts=64, rows=128, N=2048, K=4096, skew=0.0,
             format_a="e4m3", format_b="e4m3", out="bf16"),
        # a training step's: 8192 tokens, 2 of 8 experts each, some chosen more often than others
        dict(name="experts train 16384 of 8", op="experts", experts=8, rows=16384, N=4096, K=4096, skew=0.4,
             format_a="e4m3", format_b="e4m3", out="bf16"),
        # the experts' weight gradients of a training step
        dict(name="experts wgrad 8192 of 8", op="experts_wgrad", experts=8, rows=8192, M=4096, N=2048, skew=0.4,
             format_a="e5m2", format_b="e4m3", out="bf16"),
        # the router of one decode step of 64 sequences: sigmoid scores, balance bias, 4 of 8 groups
        dict(name="route decode 64 of 256", op="route", tokens=64, experts=256, type="f32", score="sigmoid", bias=True,
             padded=False, groups=8, top_groups=4, group_top=2, top_k=8, renormalise=True, scale=2.5, align=1),
        # a training step's, sequences padded to one length, segments whole blocks of 128 rows
        dict(name="route train 16384 of 64", op="route", tokens=16384, experts=64, type="bf16", score="softmax", bias=False,
             padded=True, groups=1, top_groups=1, group_top=1, top_k=6, renormalise=True, scale=1.0, align=128),
        # the router's gradient in a training step
        dict(name="route backward 16384 of 128", op="route_backward", tokens=16384, experts=128, type="bf16",
             score="softmax", top_k=8, renormalise=False, scale=1.0),
    ]


def _size(rng, low, high):
    """A size between low and high, spread over its logarithm; every other one odd or ragged."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if rng.random() < 0.5 and n >= 128:
        n = n // 128 * 128
    return max(low, min(high, n))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "experts", "experts_wgrad", "route", "route", "route_backward"])
    fa, fb = rng.choice([("e4m3", "e4m3"), ("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
    out = rng.choice(["bf16", "bf16", "f16"])
    if op == "quantize":
        direct = rng.random() < 0.75
        transposed = not direct or rng.random() < 0.5
        return dict(op=op, rows=_size(rng, 1, 8192), cols=_size(rng, 128, 4096), type=rng.choice(["bf16", "bf16", "f16", "f32"]),
                    format=rng.choice(["e4m3", "e4m3", "e5m2"]), block=rng.choice([1, 1, 128]), direct=direct,
                    transposed=transposed, gather=rng.random() < 0.3)
    if op == "product":
        block_a, block_b = rng.choice([(1, 128), (1, 128), (1, 128), (1, 1), (128, 128)])
        return dict(op=op, M=_size(rng, 1, 4096), N=_size(rng, 256, 4096), K=_size(rng, 128, 8192), block_a=block_a,
                    block_b=block_b, format_a=fa, format_b=fb, out=out)
    if op == "experts":
        experts = rng.choice([4, 8, 16, 32, 60, 64])
        return dict(op=op, experts=experts, rows=_size(rng, 1, 16384), N=_size(rng, 256, 2048), K=_size(rng, 256, 4096),
                    skew=rng.choice([0.0, 0.4, 1.0]), format_a=fa, format_b=fb, out=out)
    if op == "experts_wgrad":
        return dict(op=op, experts=rng.choice([4, 7, 8, 16]), rows=_size(rng, 1, 8192), M=_size(rng, 128, 2048),
                    N=_size(rng, 128, 2048), skew=rng.choice([0.0, 0.4, 1.0]), format_a=fa, format_b=fb, out=out)
    experts = rng.choice([8, 16, 60, 64, 128, 160, 256, 384])
    score = rng.choice(["softmax", "sigmoid"])
    top_k = rng.choice([k for k in (1, 2, 4, 6, 8, 12) if k <= experts // 2])
    tokens = _size(rng, 1, 16384)
    type_ = rng.choice(["f32", "bf16", "f16"])
    renormalise, scale = rng.random() < 0.5, rng.choice([1.0, 2.5])
    if op == "route_backward":
        renormalise = renormalise and top_k > 1  # one renormalised weight is constant
        return dict(op=op, tokens=tokens, experts=experts, type=type_, score=score, top_k=top_k, renormalise=renormalise,
                    scale=scale)
    groups = rng.choice([1, 1, 4])
    top_groups = 1 if groups == 1 else rng.choice([2, 3])
    top_k = min(top_k, top_groups * (experts // groups))
    return dict(op=op, tokens=tokens, experts=experts, type=type_, score=score, bias=rng.random() < 0.5,
                padded=rng.random() < 0.3, groups=groups, top_groups=top_groups, group_top=rng.choice([1, 2]), top_k=top_k,
                renormalise=renormalise, scale=scale, align=rng.choice([1, 16, 128]))


# ---------------------------------------------------------------- 8-bit values in blocks
def _blocks(x, block):
    """x (rows x cols, fp32) in blocks of `block` rows and 128 columns: (row blocks, block, column blocks, 128), zero-filled."""
    r, c = x.shape
    x = torch.nn.functional.pad(x, (0, -c % 128, 0, -r % block))
    return x.view(x.shape[0] // block, block, x.shape[1] // 128, 128)


def _quantize(x, fmt, block):
    """(codes as 8-bit floats, scales[k block][row block]) of x, its blocks running along the columns."""
    v = _blocks(x, block)
    amax = v.abs().amax(dim=(1, 3))
    scale = torch.where(amax.isfinite(), (amax / LARGEST[fmt]).clamp(min=2.0 ** -126), torch.full_like(amax, math.nan))
    q = (v / scale[:, None, :, None]).to(F8[fmt])
    q = q.view(v.shape[0] * block, v.shape[2] * 128)[: x.shape[0], : x.shape[1]]
    return q, scale.t().contiguous()


def _values(codes, fmt, scale, rows, K, block):
    """The fp32 values of codes (rows x ld bytes, K of them in use) under scale[k block][row block]."""
    v = codes[..., :K].view(F8[fmt]).to(torch.float32)
    s = scale.transpose(-1, -2).repeat_interleave(block, dim=-2)[..., :rows, :].repeat_interleave(128, dim=-1)[..., :K]
    return v * s


def _round_up(n, m):
    return (n + m - 1) // m * m


def _operand(x, fmt, block):
    """x (rows x K) as a product takes it: bytes in rows of a multiple of 16, and scales."""
    q, s = _quantize(x, fmt, block)
    codes = torch.zeros(x.shape[0], _round_up(x.shape[1], 16), dtype=torch.uint8, device=x.device)
    codes[:, : x.shape[1]] = q.view(torch.uint8)
    return codes, s


def _activations(rows, cols, g):
    """Features of unlike sizes, a few of them large, and tokens of unlike sizes."""
    feature = torch.exp(0.6 * torch.randn(cols, device=DEVICE, generator=g))
    token = torch.exp(0.4 * torch.randn(rows, 1, device=DEVICE, generator=g))
    return torch.randn(rows, cols, device=DEVICE, generator=g) * feature * token


# ---------------------------------------------------------------- routing in 64 bits
def _scores(logits, score):
    return torch.softmax(logits, dim=-1) if score == "softmax" else torch.sigmoid(logits)


def _ranked(keys):
    """Indices along the last dimension by falling key, equal keys by rising index."""
    return torch.sort(keys, dim=-1, descending=True, stable=True).indices


def _choose(logits, bias, c):
    keys = _scores(logits, c["score"]) + (0.0 if bias is None else bias.double())
    T, E = keys.shape
    if c["groups"] > 1:
        grouped = keys.view(T, c["groups"], -1)
        best = torch.sort(grouped, dim=-1, descending=True).values[..., : c["group_top"]].sum(-1)
        kept = _ranked(best)[:, : c["top_groups"]]
        allowed = torch.zeros_like(best, dtype=torch.bool).scatter_(1, kept, True)
        keys = torch.where(allowed[..., None], grouped, -math.inf).view(T, E)
    return _ranked(keys)[:, : c["top_k"]]


def _weights(logits, ids, c):
    w = _scores(logits, c["score"]).gather(1, ids)
    if c["renormalise"]:
        w = w / w.sum(-1, keepdim=True)
    return w * c["scale"]


def _route_rows(c):
    """Rows that the segments need at most."""
    slots = c["tokens"] * c["top_k"]
    return slots + min(c["experts"], slots) * (c["align"] - 1)


# ---------------------------------------------------------------- inputs
def _segments(c, align, seed):
    """Rows of each expert, as boundaries on the host."""
    g = torch.Generator().manual_seed(seed)
    p = torch.exp(c["skew"] * torch.randn(c["experts"], generator=g))
    counts = torch.bincount(torch.multinomial(p, c["rows"], replacement=True, generator=g), minlength=c["experts"])
    return [0] + torch.cumsum((counts + align - 1) // align * align, 0).tolist()


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    s = {"case": c}
    op = c["op"]
    empty = lambda *shape, dtype: torch.zeros(*shape, dtype=dtype, device=DEVICE)  # noqa: E731
    if op == "quantize":
        R, C, b = c["rows"], c["cols"], c["block"]
        held = max(1, R // 2) if c["gather"] else R
        s["x"] = _activations(held, C, g).to(TYPES[c["type"]])
        if c["gather"]:  # tokens of one dispatch: some repeated, some rows padding
            s["index"] = torch.randint(-1, held, (R,), device=DEVICE, generator=g, dtype=torch.int32)
        if c["direct"]:
            s["q"], s["s"] = empty(R, _round_up(C, 16), dtype=torch.uint8), empty(-(-C // 128), -(-R // b), dtype=torch.float32)
        if c["transposed"]:
            s["qt"], s["st"] = empty(C, _round_up(R, 16), dtype=torch.uint8), empty(-(-R // 128), -(-C // b), dtype=torch.float32)
    elif op == "product":
        s["a"], s["sa"] = _operand(_activations(c["M"], c["K"], g), c["format_a"], c["block_a"])
        s["b"], s["sb"] = _operand(0.02 * torch.randn(c["N"], c["K"], device=DEVICE, generator=g), c["format_b"], c["block_b"])
        s["c"] = empty(c["M"], c["N"], dtype=TYPES[c["out"]])
    elif op == "experts":
        E, N, K = c["experts"], c["N"], c["K"]
        s["bounds"] = _segments(c, 1, seed)
        s["offsets"] = torch.tensor(s["bounds"], dtype=torch.int32, device=DEVICE)
        s["a"], s["sa"] = _operand(_activations(c["rows"], K, g), c["format_a"], 1)
        weights = [_operand(0.02 * torch.randn(N, K, device=DEVICE, generator=g), c["format_b"], 128) for _ in range(E)]
        s["b"], s["sb"] = (torch.stack([w[i] for w in weights]) for i in (0, 1))
        s["c"] = empty(c["rows"], N, dtype=TYPES[c["out"]])
    elif op == "experts_wgrad":
        s["bounds"] = _segments(c, 128, seed)
        s["offsets"] = torch.tensor(s["bounds"], dtype=torch.int32, device=DEVICE)
        total = s["bounds"][-1]
        s["a"], s["sa"] = _operand(_activations(total, c["M"], g).t().contiguous(), c["format_a"], 1)
        s["b"], s["sb"] = _operand(_activations(total, c["N"], g).t().contiguous(), c["format_b"], 1)
        s["c"] = empty(c["experts"], c["M"], c["N"], dtype=TYPES[c["out"]])
    else:
        T, E, k = c["tokens"], c["experts"], c["top_k"]
        s["logits"] = (1.5 * torch.randn(T, E, device=DEVICE, generator=g)).to(TYPES[c["type"]])
        if op == "route":
            s["bias"] = 0.1 * torch.randn(E, device=DEVICE, generator=g) if c["bias"] else None
            s["keep"] = None
            if c["padded"]:  # sequences of up to 512 tokens, each filled to that length
                length = torch.randint(128, 513, (-(-T // 512),), device=DEVICE, generator=g)
                s["keep"] = (torch.arange(512, device=DEVICE) < length[:, None]).view(-1)[:T].to(torch.uint8).contiguous()
            rows = _route_rows(c)
            s["ids"], s["weights"] = empty(T, k, dtype=torch.int32), empty(T, k, dtype=torch.float32)
            s["offsets"], s["row_tokens"] = empty(E + 1, dtype=torch.int32), empty(rows, dtype=torch.int32)
            s["places"] = empty(T, k, dtype=torch.int32)
        else:
            whole = dict(c, groups=1)
            s["ids"] = _choose(s["logits"].double(), None, whole).to(torch.int32).contiguous()
            s["d_weights"] = torch.randn(T, k, device=DEVICE, generator=g)
            s["d_logits"] = empty(T, E, dtype=TYPES[c["type"]])
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    if own:
        return globals()["_own_" + c["op"]](s, c)
    return globals()["_plain_" + c["op"]](s, c)


def _plain_quantize(s, c):
    x = s["x"].to(torch.float32)
    if c["gather"]:
        x = torch.where(s["index"][:, None] >= 0, x[s["index"].clamp(min=0).long()], 0.0)
    r = {}
    if c["direct"]:
        r["q"], r["s"] = _quantize(x, c["format"], c["block"])
    if c["transposed"]:
        r["qt"], r["st"] = _quantize(x.t(), c["format"], c["block"])
    return r


def _plain_product(s, c):
    a = _values(s["a"], c["format_a"], s["sa"], c["M"], c["K"], c["block_a"])
    b = _values(s["b"], c["format_b"], s["sb"], c["N"], c["K"], c["block_b"])
    return torch.matmul(a, b.t()).to(s["c"].dtype)


def _padded_rows(s, rows):
    """Each segment's rows filled to the longest one's length: (experts x length indices, which of them are rows)."""
    o = s["offsets"].long()
    longest = max(1, max(b - a for a, b in zip(s["bounds"], s["bounds"][1:])))
    at = o[:-1, None] + torch.arange(longest, device=o.device)
    live = at < o[1:, None]
    return torch.where(live, at, 0), live


def _plain_experts(s, c):
    a = _values(s["a"], c["format_a"], s["sa"], c["rows"], c["K"], 1)
    b = _values(s["b"], c["format_b"], s["sb"], c["N"], c["K"], 128)
    at, live = _padded_rows(s, c["rows"])
    r = torch.bmm(a[at], b.transpose(1, 2))
    out = torch.zeros(c["rows"], c["N"], device=a.device)
    out[at[live]] = r[live]
    return out.to(s["c"].dtype)


def _plain_experts_wgrad(s, c):
    total = s["bounds"][-1]
    a = _values(s["a"], c["format_a"], s["sa"], c["M"], total, 1)
    b = _values(s["b"], c["format_b"], s["sb"], c["N"], total, 1)
    at, live = _padded_rows(s, total)
    a = torch.where(live[:, None], a[:, at].transpose(0, 1), 0.0)
    b = b[:, at].permute(1, 2, 0)
    return torch.bmm(a.contiguous(), b.contiguous()).to(s["c"].dtype)


def _plain_route(s, c):
    T, E, k = c["tokens"], c["experts"], c["top_k"]
    logits = s["logits"].double()  # neighbours in rank may be close: 64 bits
    ids = _choose(logits, s["bias"], c)
    weights = _weights(logits, ids, c)
    if s["keep"] is not None:
        gone = s["keep"][:, None] == 0
        ids, weights = torch.where(gone, -1, ids), torch.where(gone, 0.0, weights)
    flat = torch.where(ids < 0, E, ids).view(-1)
    order = torch.sort(flat, stable=True).indices
    counts = (flat[:, None] == torch.arange(E, device=flat.device)).sum(0)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=flat.device)
    offsets[1:] = torch.cumsum((counts + c["align"] - 1) // c["align"] * c["align"], 0)
    before = torch.cumsum(counts, 0) - counts
    e = flat[order]
    used = e < E
    e = e.clamp(max=E - 1)
    place = torch.where(used, offsets[e] + torch.arange(T * k, device=flat.device) - before[e], -1)
    places = torch.empty_like(flat).scatter_(0, order, place)
    rows = _route_rows(c)
    tokens = torch.full((rows + 1,), -1, dtype=torch.int64, device=flat.device)
    tokens.scatter_(0, torch.where(used, place, rows), torch.where(used, order // k, -1))
    i32 = torch.int32
    return {"ids": ids.to(i32), "weights": weights.float(), "offsets": offsets.to(i32), "row_tokens": tokens[:rows].to(i32),
            "places": places.view(T, k).to(i32)}


def _plain_route_backward(s, c):
    x, ids = s["logits"].float(), s["ids"].long()
    dw = s["d_weights"] * c["scale"]
    p = _scores(x, c["score"])
    w = p.gather(1, ids)
    if c["renormalise"]:  # of w / sum w
        total = w.sum(-1, keepdim=True)
        dw = (dw - (dw * w).sum(-1, keepdim=True) / total) / total
    if c["score"] == "sigmoid":
        d = torch.zeros_like(x).scatter_(1, ids, dw * w * torch.sigmoid(-x).gather(1, ids))
    else:
        d = -p * (dw * w).sum(-1, keepdim=True)
        d.scatter_add_(1, ids, dw * w)
    return d.to(s["logits"].dtype)


# ---------------------------------------------------------------- through the framework
def _binding():
    from dense_gemm_optimisation_amd import binding
    return binding


def _own_quantize(s, c):
    lib = _binding()
    type_ = {"f32": lib.INPUT_F32, "bf16": lib.INPUT_BF16, "f16": lib.INPUT_F16}[c["type"]]
    fmt = lib.F8_E4M3 if c["format"] == "e4m3" else lib.F8_E5M2
    x, index = s["x"], s.get("index")
    q, sc, qt, st = (s.get(n) for n in ("q", "s", "qt", "st"))
    lib.gemm_f8_block_quantize(
        c["rows"], c["cols"], x.data_ptr(), x.stride(0), type_, 0 if index is None else index.data_ptr(), x.shape[0], fmt,
        c["block"], 0 if q is None else q.data_ptr(), 0 if q is None else q.stride(0), 0 if q is None else sc.data_ptr(),
        0 if q is None else sc.stride(0), 0 if qt is None else qt.data_ptr(), 0 if qt is None else qt.stride(0),
        0 if qt is None else st.data_ptr(), 0 if qt is None else st.stride(0))
    r = {}
    if q is not None:
        r["q"], r["s"] = q[:, : c["cols"]].view(F8[c["format"]]), sc
    if qt is not None:
        r["qt"], r["st"] = qt[:, : c["rows"]].view(F8[c["format"]]), st
    return r


def _formats(lib, c):
    f = {"e4m3": lib.F8_E4M3, "e5m2": lib.F8_E5M2}
    return f[c["format_a"]], f[c["format_b"]], {"f32": lib.OUTPUT_F32, "bf16": lib.OUTPUT_BF16, "f16": lib.OUTPUT_F16}[c["out"]]


def _own_product(s, c):
    lib = _binding()
    fa, fb, out = _formats(lib, c)
    a, sa, b, sb, o = s["a"], s["sa"], s["b"], s["sb"], s["c"]
    lib.gemm_f8_block(c["M"], c["N"], c["K"], 1.0, a.data_ptr(), a.stride(0), fa, sa.data_ptr(), sa.stride(0), c["block_a"],
                      b.data_ptr(), b.stride(0), fb, sb.data_ptr(), sb.stride(0), c["block_b"], 0.0, o.data_ptr(), o.stride(0),
                      lib.ROW_MAJOR, out)
    return o


def _own_experts(s, c):
    lib = _binding()
    fa, fb, out = _formats(lib, c)
    a, sa, b, sb, o = s["a"], s["sa"], s["b"], s["sb"], s["c"]
    lib.gemm_experts_f8(c["experts"], c["rows"], c["N"], c["K"], s["offsets"].data_ptr(), 1.0, a.data_ptr(), a.stride(0), fa,
                        sa.data_ptr(), sa.stride(0), b.data_ptr(), b.stride(1), fb, sb.data_ptr(), sb.stride(1), 128,
                        b.stride(0), sb.stride(0), 0.0, o.data_ptr(), o.stride(0), out)
    return o


def _own_experts_wgrad(s, c):
    lib = _binding()
    fa, fb, out = _formats(lib, c)
    a, sa, b, sb, o = s["a"], s["sa"], s["b"], s["sb"], s["c"]
    lib.gemm_experts_f8_wgrad(c["experts"], c["M"], c["N"], s["bounds"][-1], s["offsets"].data_ptr(), 1.0, a.data_ptr(),
                              a.stride(0), fa, sa.data_ptr(), sa.stride(0), b.data_ptr(), b.stride(0), fb, sb.data_ptr(),
                              sb.stride(0), 0.0, o.data_ptr(), o.stride(1), o.stride(0), out)
    return o


def _route_type(lib, c):
    return {"f32": lib.INPUT_F32, "bf16": lib.INPUT_BF16, "f16": lib.INPUT_F16}[c["type"]], \
        lib.SCORE_SOFTMAX if c["score"] == "softmax" else lib.SCORE_SIGMOID


def _own_route(s, c):
    lib = _binding()
    type_, score = _route_type(lib, c)
    x, bias, keep = s["logits"], s["bias"], s["keep"]
    if "workspace" not in s:  # a user's program keeps it from call to call
        s["workspace"] = torch.empty(lib.experts_route_workspace_size(c["tokens"], c["experts"], c["top_k"]), dtype=torch.uint8,
                                     device=x.device)
    lib.gemm_experts_route(
        c["tokens"], c["experts"], x.data_ptr(), x.stride(0), type_, 0 if bias is None else bias.data_ptr(),
        0 if keep is None else keep.data_ptr(), score, c["groups"], c["top_groups"], c["group_top"], c["top_k"],
        c["renormalise"], c["scale"], s["ids"].data_ptr(), s["weights"].data_ptr(), c["align"], s["row_tokens"].numel(),
        s["offsets"].data_ptr(), s["row_tokens"].data_ptr(), s["places"].data_ptr(), s["workspace"].data_ptr(),
        s["workspace"].numel())
    return {n: s[n] for n in ("ids", "weights", "offsets", "row_tokens", "places")}


def _own_route_backward(s, c):
    lib = _binding()
    type_, score = _route_type(lib, c)
    x, d = s["logits"], s["d_logits"]
    lib.gemm_experts_route_backward(c["tokens"], c["experts"], x.data_ptr(), x.stride(0), type_, score, c["top_k"],
                                    c["renormalise"], c["scale"], s["ids"].data_ptr(), s["d_weights"].data_ptr(), d.data_ptr(),
                                    d.stride(0))
    return d


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    op = c["op"]
    size = {"f32": 4, "bf16": 2, "f16": 2}
    if op == "quantize":
        R, C = c["rows"], c["cols"]
        read = (max(1, R // 2) if c["gather"] else R) * C * size[c["type"]] + (4 * R if c["gather"] else 0)
        out = (R * C + 4 * -(-R // c["block"]) * -(-C // 128)) * c["direct"]
        out += (R * C + 4 * -(-C // c["block"]) * -(-R // 128)) * c["transposed"]
        return {"bytes": read + out, "flops": 2 * R * C * (c["direct"] + c["transposed"])}
    if op == "product":
        M, N, K = c["M"], c["N"], c["K"]
        kb = -(-K // 128)
        scales = 4 * kb * (-(-M // c["block_a"]) + -(-N // c["block_b"]))
        return {"bytes": (M + N) * K + scales + M * N * size[c["out"]], "flops": 2 * M * N * K}
    if op == "experts":
        E, R, N, K = c["experts"], c["rows"], c["N"], c["K"]
        live = E * (1 - (1 - 1 / E) ** R)  # experts that any row chose, on average
        weights = live * (N * K + 4 * -(-N // 128) * -(-K // 128))
        return {"bytes": weights + R * (K + 4 * -(-K // 128)) + R * N * size[c["out"]] + 4 * (E + 1), "flops": 2 * R * N * K}
    if op == "experts_wgrad":
        E, R, M, N = c["experts"], c["rows"], c["M"], c["N"]
        return {"bytes": (M + N) * (R + 4 * -(-R // 128)) + E * M * N * size[c["out"]], "flops": 2 * R * M * N}
    T, E, k = c["tokens"], c["experts"], c["top_k"]
    if op == "route":
        return {"bytes": T * E * size[c["type"]] + 12 * T * k + 4 * (E + 1) + 4 * _route_rows(c), "flops": 4 * T * E}
    return {"bytes": 2 * T * E * size[c["type"]] + 8 * T * k, "flops": 6 * T * E}


# ---------------------------------------------------------------- from the definitions, in 64 bits
def _nearest(v, fmt):
    """v rounded to the nearest value of an 8-bit format, ties to even."""
    bits, low = (3, -6) if fmt == "e4m3" else (2, -14)
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), torch.clamp(e - 1, min=low) - bits)
    return torch.clamp(torch.round(v / step) * step, -LARGEST[fmt], LARGEST[fmt])


def _exact_quantize(x, fmt, block):
    """Column block by column block."""
    q, scales = torch.empty_like(x), []
    for k in range(0, x.shape[1], 128):
        part = x[:, k: k + 128]
        rows = part.abs().amax(1)
        rows = torch.nn.functional.pad(rows, (0, -len(rows) % block)).view(-1, block).amax(1)
        s = torch.clamp(rows / LARGEST[fmt], min=2.0 ** -126)
        scales.append(s)
        q[:, k: k + 128] = _nearest(part / s.repeat_interleave(block)[: len(part), None], fmt)
    return q, torch.stack(scales)


def _exact_product(a, sa, fa, block_a, b, sb, fb, block_b, K):
    """The sum over K's blocks of each block's product times its scales."""
    out = torch.zeros(a.shape[0], b.shape[0], dtype=torch.float64, device=a.device)
    for i in range(-(-K // 128)):
        k = slice(128 * i, min(128 * i + 128, K))
        part = torch.mm(a[:, k].view(F8[fa]).double(), b[:, k].view(F8[fb]).double().t().contiguous())
        part *= sa[i].double().repeat_interleave(block_a)[: a.shape[0], None]
        out += part * sb[i].double().repeat_interleave(block_b)[: b.shape[0]]
    return out


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    op = c["op"]
    if op == "quantize":
        x = s["x"].double()
        if c["gather"]:
            x = torch.cat([x, torch.zeros_like(x[:1])])[s["index"].long()]  # -1 names the added row of zeros
        r = {}
        if c["direct"]:
            r["q"], r["s"] = _exact_quantize(x, c["format"], c["block"])
        if c["transposed"]:
            r["qt"], r["st"] = _exact_quantize(x.t().contiguous(), c["format"], c["block"])
        return r
    if op == "product":
        return _exact_product(s["a"], s["sa"], c["format_a"], c["block_a"], s["b"], s["sb"], c["format_b"], c["block_b"], c["K"])
    if op == "experts":
        out = torch.zeros(c["rows"], c["N"], dtype=torch.float64, device=DEVICE)
        for e, (lo, hi) in enumerate(zip(s["bounds"], s["bounds"][1:])):
            if hi > lo:
                out[lo:hi] = _exact_product(s["a"][lo:hi], s["sa"][:, lo:hi], c["format_a"], 1, s["b"][e], s["sb"][e],
                                            c["format_b"], 128, c["K"])
        return out
    if op == "experts_wgrad":
        return torch.stack([
            _exact_product(s["a"][:, lo:hi], s["sa"][lo // 128:], c["format_a"], 1, s["b"][:, lo:hi], s["sb"][lo // 128:],
                           c["format_b"], 1, hi - lo) for lo, hi in zip(s["bounds"], s["bounds"][1:])])
    x = s["logits"].double()
    score = (lambda v: torch.exp(v - torch.logsumexp(v, 1, keepdim=True))) if c["score"] == "softmax" else \
        (lambda v: 1 / (1 + torch.exp(-v)))
    if op == "route":
        p = score(x)
        keys = p.clone() if s["bias"] is None else p + s["bias"].double()
        if c["groups"] > 1:  # the groups one by one, by the sum of their largest keys
            by_group = keys.view(c["tokens"], c["groups"], -1)
            rank = by_group.topk(c["group_top"], dim=2).values.sum(2)
            for _ in range(c["groups"] - c["top_groups"]):  # the last of the smallest goes
                worst = c["groups"] - 1 - rank.flip(1).argmin(1)
                by_group[torch.arange(c["tokens"]), worst] = -math.inf
                rank[torch.arange(c["tokens"]), worst] = math.inf
        w = []
        for _ in range(c["top_k"]):
            at = keys.argmax(1, keepdim=True)
            w.append(p.gather(1, at))
            keys.scatter_(1, at, -math.inf)
        w = torch.cat(w, 1)
        w = c["scale"] * (w / w.sum(1, keepdim=True) if c["renormalise"] else w)
        if s["keep"] is not None:
            w[s["keep"] == 0] = 0
        return {"ids": None, "weights": w, "offsets": None, "row_tokens": None, "places": None}
    x.requires_grad_(True)
    with torch.enable_grad():
        w = score(x).gather(1, s["ids"].long())
        w = w / w.sum(1, keepdim=True) if c["renormalise"] else w
        (c["scale"] * w * s["d_weights"].double()).sum().backward()
    return x.grad
