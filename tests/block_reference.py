"""Definitions, in 64 bits and on the CPU, of what libgemm_experts.h declares.

Values and sums are computed in float64 from the stored bytes and scales.
Only where the interface fixes a rounding (a scale is rounded to fp32, and so
is a value's quotient by it) is that rounding applied.
"""
import numpy as np

LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
_BITS = {"e4m3": (4, 3, 7), "e5m2": (5, 2, 15)}  # exponent bits, fraction bits, bias


def _table(fmt):
    e_bits, f_bits, bias = _BITS[fmt]
    v = np.zeros(256)
    for b in range(256):
        e, f = (b >> f_bits) & ((1 << e_bits) - 1), b & ((1 << f_bits) - 1)
        x = f * 2.0 ** (1 - bias - f_bits) if e == 0 else (1 + f / (1 << f_bits)) * 2.0 ** (e - bias)
        if fmt == "e4m3" and (b & 0x7F) == 0x7F:
            x = np.nan
        if fmt == "e5m2" and e == 31:
            x = np.inf if f == 0 else np.nan
        v[b] = -x if b & 0x80 else x
    return v


TABLE = {f: _table(f) for f in _BITS}


def encode(x, fmt):
    """Bytes of the nearest values (ties to even, saturated), NaN as 0x7F."""
    positive = np.array([v for v in TABLE[fmt][:128] if np.isfinite(v)])  # rising with the byte
    m = np.minimum(np.abs(x), LARGEST[fmt])
    hi = np.clip(np.searchsorted(positive, np.where(np.isnan(m), 0, m)), 0, len(positive) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = m - positive[lo], positive[hi] - m
    near = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    b = np.where(np.isnan(x), 0x7F, near + np.where(np.signbit(x), 128, 0))
    return b.astype(np.uint8)


def quantize(x, fmt, block):
    """(bytes, scales[k block][row block]) of x (rows x cols, float64), blocks along the columns."""
    R, C = x.shape
    codes = np.zeros((R, C), np.uint8)
    scales = np.zeros((-(-C // 128), -(-R // block)), np.float32)
    f32 = np.float32
    with np.errstate(all="ignore"):
        for kb in range(scales.shape[0]):
            for rb in range(scales.shape[1]):
                at = np.s_[rb * block:(rb + 1) * block, kb * 128:(kb + 1) * 128]
                part = x[at]
                if not np.all(np.isfinite(part)):
                    s = f32(np.nan)
                    codes[at] = 0x7F
                else:
                    s = max(f32(np.max(np.abs(part))) / f32(LARGEST[fmt]), f32(2.0 ** -126))
                    codes[at] = encode((part.astype(f32) / s).astype(np.float64), fmt)
                scales[kb, rb] = s
    return codes, scales


def values(codes, fmt, scales, block):
    """The float64 values of codes (rows x K) under scales[k block][row block]."""
    R, K = codes.shape
    s = scales.astype(np.float64).T
    return TABLE[fmt][codes] * np.repeat(np.repeat(s, block, 0)[:R], 128, 1)[:, :K]


def choose(logits, bias, keep, sigmoid, groups, top_groups, group_top, top_k, renormalise, scale):
    """(ids, weights) by the definition, token by token."""
    T, E = logits.shape
    ids, weights = np.full((T, top_k), -1, np.int32), np.zeros((T, top_k))
    with np.errstate(all="ignore"):
        for t in range(T):
            if keep is not None and keep[t] == 0:
                continue
            x = logits[t]
            if sigmoid:
                p = 1 / (1 + np.exp(-x))
            else:
                if np.any(np.isnan(x)) or np.any(x == np.inf):
                    weights[t] = np.nan
                    continue
                if np.all(x == -np.inf):
                    continue
                p = np.exp(x - x.max())
                p = p / p.sum()
            key = p if bias is None else p + bias
            can = ~np.isnan(x) & (x != -np.inf) & ~np.isnan(key) & (key != -np.inf)
            if bias is None and groups == 1:
                key = x  # the same order, without underflow
            if groups > 1:
                per = E // groups
                rank = []
                for g in range(groups):
                    mine = sorted((key[e] for e in range(g * per, (g + 1) * per) if can[e]), reverse=True)
                    rank.append(sum(mine[:group_top]) if mine else -np.inf)
                kept = sorted(range(groups), key=lambda g: (-rank[g], g))[:top_groups]
                can = can & np.isin(np.arange(E) // per, kept)
            order = sorted((e for e in range(E) if can[e]), key=lambda e: (-key[e], e))[:top_k]
            n = len(order)
            ids[t, :n] = order
            w = p[order]
            if renormalise and n:
                if not sigmoid:
                    w = np.exp(x[order] - x[order].max())
                w = w / w.sum() if w.sum() > 0 else np.zeros(n)
            weights[t, :n] = w * scale
    return ids, weights


def layout(ids, experts, align, rows):
    """(offsets, row_tokens, places) of the chosen rows, expert by expert and token by token."""
    T, k = ids.shape
    offsets, row_tokens = np.zeros(experts + 1, np.int32), np.full(rows, -1, np.int32)
    places = np.full((T, k), -1, np.int32)
    at = 0
    for e in range(experts):
        offsets[e] = at
        for t, j in zip(*np.nonzero(ids == e)):
            row_tokens[at], places[t, j] = t, at
            at += 1
        at = offsets[e] + -(-(at - offsets[e]) // align) * align
    offsets[experts] = at
    return offsets, row_tokens, places


def route_gradient(logits, ids, d_weights, sigmoid, renormalise, scale):
    """d logits of sum(weights * d_weights), the choice held fixed."""
    T, E = logits.shape
    d = np.zeros((T, E))
    for t in range(T):
        chosen = [(e, g) for e, g in zip(ids[t], d_weights[t]) if 0 <= e < E]
        if not chosen:
            continue
        e, g = np.array([c[0] for c in chosen]), scale * np.array([c[1] for c in chosen])
        x = logits[t]
        p = 1 / (1 + np.exp(-x)) if sigmoid else np.exp(x - x.max()) / np.exp(x - x.max()).sum()
        w = p[e]
        if renormalise:
            g = (g - (g * w).sum() / w.sum()) / w.sum()
        dp = np.zeros(E)
        np.add.at(dp, e, g)
        d[t] = dp * p * (1 - p) if sigmoid else p * (dp - (dp * p).sum())
    return d
