"""Plain 64-bit references of the MoE gating, the expert combination and the INT8 products (numpy, loops over
tokens), with the error bounds the GPU tests use."""
import numpy as np

EPS = 1e-20
U = 2.0 ** -24  # unit roundoff of fp32


def scores(x, kind):
    """float64 scores of one token's logits (masked experts 0)."""
    x = np.minimum(np.asarray(x, np.float64), np.finfo(np.float32).max)
    ok = x > -np.inf  # false for NaN
    s = np.zeros(len(x))
    if kind == "sigmoid":
        with np.errstate(over="ignore"):
            s[ok] = 1.0 / (1.0 + np.exp(-x[ok]))
    elif ok.any():
        with np.errstate(over="ignore"):
            e = np.exp(x[ok] - x[ok].max())
        s[ok] = e / e.sum()
    return s, ok


def gate_token(x, k, kind, bias, n_group, topk_group, group_top, renorm, scale):
    """(experts, weights, gap) of one token; gap is the smallest relative difference between two neighbouring
    keys (or group values) that decided the choice, inf when every such pair was equal or masked."""
    s, ok = scores(x, kind)
    E = len(s)
    key = [s[e] + (0.0 if bias is None else float(bias[e])) if ok[e] else None for e in range(E)]
    size = E // n_group
    gap = np.inf

    def note(a, b):
        nonlocal gap
        if a != b and np.isfinite(a) and np.isfinite(b):
            gap = min(gap, abs(a - b) / max(abs(a), abs(b)))

    kept = set(range(n_group))
    if topk_group < n_group:
        value = []
        for g in range(n_group):
            best = sorted((key[e] for e in range(g * size, (g + 1) * size) if key[e] is not None), reverse=True)
            value.append(sum(best[:group_top]) if best else -np.inf)
        order = sorted(range(n_group), key=lambda g: (-value[g], g))
        kept = set(order[:topk_group])
        note(value[order[topk_group - 1]], value[order[topk_group]])
    cand = sorted((e for e in range(E) if key[e] is not None and e // size in kept), key=lambda e: (-key[e], e))
    for a, b in zip(cand[:k], cand[1:k + 1]):
        note(key[a], key[b])
    chosen = cand[:k]
    w = np.zeros(k)
    v = s[chosen]
    w[:len(chosen)] = scale * (v / (v.sum() + EPS) if renorm else v)
    return chosen + [-1] * (k - len(chosen)), w, gap


def layout(idx, E, rows):
    """The expert-sorted layout of idx [T][k] as fp8q_moe_route_topk documents it, with -1 slots left out."""
    T, k = idx.shape
    offsets = np.zeros(E + 1, np.int32)
    row_of = np.full((T, k), -1, np.int32)
    row_token = np.full(rows, -1, np.int32)
    load = np.bincount(idx[idx >= 0], minlength=E).astype(np.int32)
    offsets[1:] = np.cumsum((load + 127) // 128 * 128)
    nxt = offsets[:-1].copy()
    for t in range(T):
        for j in range(k):
            e = idx[t, j]
            if e >= 0:
                row_of[t, j] = nxt[e]
                row_token[nxt[e]] = t
                nxt[e] += 1
    return offsets, row_of, row_token, load


def gate_weights(x, idx, kind, renorm, scale):
    """Weights of a fixed choice (float64), the function whose gradient the backward pass computes."""
    s, _ = scores(x, kind)
    v = np.array([s[e] if e >= 0 else 0.0 for e in idx])
    return scale * (v / (v.sum() + EPS) if renorm else v)


def gate_grad(x, idx, dw, kind, renorm, scale):
    """Gradient of sum(dw * weights) with respect to the logits, from the formula, and the sum of the magnitudes
    of the terms it adds up (for error bounds)."""
    s, ok = scores(x, kind)
    E = len(s)
    slots = [(int(e), float(d)) for e, d in zip(idx, dw) if e >= 0]
    S = sum(s[e] for e, _ in slots) + EPS
    ds, mag = np.zeros(E), np.zeros(E)
    D = sum(scale * d * s[e] for e, d in slots)
    Dm = sum(abs(scale * d) * s[e] for e, d in slots)
    for e, d in slots:
        ds[e] = (scale * d - D / S) / S if renorm else scale * d
        mag[e] = (abs(scale * d) + Dm / S) / S if renorm else abs(scale * d)
    if kind == "sigmoid":
        xc = np.minimum(np.where(ok, x, 0.0).astype(np.float64), np.finfo(np.float32).max)
        with np.errstate(over="ignore"):
            f = np.where(ok, s / (1.0 + np.exp(xc)), 0.0)  # s (1 - s)
        return ds * f, mag * f
    c = float((ds * s).sum())
    cm = float((mag * s).sum())
    return s * (ds - c), s * (mag + cm)


def quant_int8(x):
    """(codes int8, scales float32) of float32 rows x, every step in IEEE fp32."""
    x = np.asarray(x, np.float32)
    amax = np.abs(x).max(axis=1) if x.shape[1] else np.zeros(len(x), np.float32)
    s = (amax / np.float32(127.0)).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        v = np.where(s[:, None] > 0, x / s[:, None], np.float32(0))
    return np.rint(v).astype(np.int8), s


def gemm_int8(qa, sa, qw, sw):
    """float32 [M, N], the value every fp32 output has to equal: exact integer sums, one rounding to fp32, times
    the fp32 product of the scales.  (The sums are formed in float64: below 2^31, hence exact.)"""
    acc = np.asarray(qa, np.float64) @ np.asarray(qw, np.float64).T
    return acc.astype(np.float32) * (np.asarray(sa, np.float32)[:, None] * np.asarray(sw, np.float32)[None, :])


def bf16_round(f):
    """float32 -> the uint16 pattern of its nearest-even bf16 (finite values)."""
    b = np.ascontiguousarray(f, np.float32).view(np.uint32)
    return ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)
