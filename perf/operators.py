"""Cases that time the MoE routing, expert combination and INT8 matrix product operators.

Each case is one pass through one operator.  ``run`` computes it either through this package's entry points
(``own`` is true) or in a plain form of elementary torch operations in 32 bits (``own`` is false); ``exact``
gives the same answer from the definition in 64 bits.  The operators:

  route             router logits -> each token's experts, their weights, the expert-sorted 128-row layout and
                    the experts' loads
  route_backward    the gradient of the weights -> the gradient of the logits
  combine           the experts' output rows, weighted and added up per token
  combine_backward  the gradient of the combined rows -> of the expert rows and of the weights
  linear            tokens quantized to INT8 (one scale per token) times INT8 weights (one scale per channel)
  experts           the same per expert, on the routed rows of an expert-sorted layout
"""
import math

import torch

own = False

EPS = 1e-20  # added to the sum of the chosen scores before dividing by it
BIG = torch.finfo(torch.float32).max


def listed():
    return [
        # One token of a serving step through 256 experts in 8 groups: launch latency.
        dict(name="route 1 of 256", op="route", T=1, E=256, k=8, score="sigmoid", bias=True, n_group=8, topk_group=4,
             group_top=2, renorm=True, scale=2.5, dtype="f32", offline=0),
        # A long prompt (or a training microbatch) through the same router.
        dict(name="route 8192 of 256", op="route", T=8192, E=256, k=8, score="sigmoid", bias=True, n_group=8,
             topk_group=4, group_top=2, renorm=True, scale=2.5, dtype="f32", offline=0),
        # Training: the router's gradient, softmax scores, bf16 logits.
        dict(name="route backward 8192 of 64", op="route_backward", T=8192, E=64, k=8, score="softmax", renorm=False,
             scale=1.0, dtype="bf16"),
        # A decode batch's expert outputs gathered back to tokens.
        dict(name="combine 64 tokens", op="combine", T=64, E=64, k=8, H=7168, add=True, dtype="bf16"),
        # A prompt's expert outputs, with the shared expert's rows added.
        dict(name="combine 8192 tokens", op="combine", T=8192, E=64, k=8, H=7168, add=True, dtype="bf16"),
        # Training: gradients of the expert rows and of the weights, an odd token count.
        dict(name="combine backward 4093", op="combine_backward", T=4093, E=64, k=6, H=2048, dtype="bf16"),
        # One token through an up projection: the weight matrix read once.
        dict(name="linear 1x18432x7168", op="linear", M=1, N=18432, K=7168, dtype="bf16"),
        # A decode batch through the same projection.
        dict(name="linear 64x18432x7168", op="linear", M=64, N=18432, K=7168, dtype="bf16"),
        # Ragged sizes: an odd token count, N and K that no tile divides, fp32 output.
        dict(name="linear 1037x4104x2064", op="linear", M=1037, N=4104, K=2064, dtype="f32"),
        # A prompt through the up projection: the matrix cores.
        dict(name="linear 4096x18432x7168", op="linear", M=4096, N=18432, K=7168, dtype="bf16"),
        # A decode batch through 64 experts: few rows each, every expert's weights read once.
        dict(name="experts 32 tokens", op="experts", T=32, E=64, k=8, N=2048, K=7168, dtype="bf16"),
        # A prompt through 64 experts.
        dict(name="experts 8192 tokens", op="experts", T=8192, E=64, k=8, N=2048, K=7168, dtype="bf16"),
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of ``step`` in [lo, hi], spread evenly over the logarithm; odd multiples come up too."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    v = min(max(v, lo), hi // step * step)
    return v if v != 3072 else v + step


def draw(rng):
    op = rng.choice(["route", "route_backward", "combine", "combine_backward", "linear", "experts"])
    if op == "route":
        G = rng.choice([1, 1, 2, 4, 8, 3])
        gs = _spread(rng, 4, 64 if G > 1 else 512)
        tg = rng.randint((G + 1) // 2, G)
        return dict(op=op, T=_spread(rng, 1, 8192), E=G * gs, k=rng.randint(1, min(16, tg * gs - tg)),
                    score=rng.choice(["sigmoid", "softmax"]), bias=rng.random() < 0.5, n_group=G, topk_group=tg,
                    group_top=rng.choice([1, 2]), renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]),
                    dtype=rng.choice(["f32", "bf16"]), offline=rng.choice([0, 0, 1]))
    if op == "route_backward":
        E, k = _spread(rng, 8, 512), rng.randint(1, 16)
        k = min(k, E)
        # (A single renormalised weight is the constant `scale`: its gradient is zero but for rounding.)
        return dict(op=op, T=_spread(rng, 1, 8192), E=E, k=k, score=rng.choice(["sigmoid", "softmax"]),
                    renorm=k > 1 and rng.random() < 0.7, scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["f32", "bf16"]))
    if op in ("combine", "combine_backward"):
        E = _spread(rng, 8, 256)
        d = dict(op=op, T=_spread(rng, 1, 8192 if op == "combine" else 4096), E=E, k=rng.randint(1, min(8, E)),
                 H=_spread(rng, 64, 7168, 8), dtype=rng.choice(["bf16", "bf16", "f32"]))
        if op == "combine":
            d["add"] = rng.random() < 0.5
        if d["dtype"] == "f32":  # as many bytes as the largest listed case at most
            d["T"] = (d["T"] + 1) // 2
        return d
    if op == "linear":
        d = dict(op=op, M=_spread(rng, 1, 4096), N=_spread(rng, 64, 18432, 8), K=_spread(rng, 64, 18432, 16),
                 dtype=rng.choice(["bf16", "bf16", "f32"]))
        while d["M"] * d["N"] * d["K"] > 4096 * 18432 * 7168:
            d["M"] = (d["M"] + 1) // 2
        return d
    E = _spread(rng, 4, 64)
    return dict(op=op, T=_spread(rng, 1, 8192), E=E, k=rng.randint(1, min(8, E)), N=_spread(rng, 128, 2048, 8),
                K=_spread(rng, 128, 7168, 16), dtype=rng.choice(["bf16", "bf16", "f32"]))


# --------------------------------------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------------------------------------

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _capacity(T, E, k):
    return (T * k + 127 * E + 127) // 128 * 128


def _layout(idx, E, rows):
    """The expert-sorted layout of ``idx`` [T, k] (-1: no expert): segment starts padded to 128 rows, the row of
    every (token, slot), the token of every row, and the experts' loads."""
    T, k = idx.shape
    dev = idx.device
    e = torch.where(idx < 0, E, idx).reshape(-1).long()
    load = torch.zeros(E + 1, dtype=torch.long, device=dev).index_add_(0, e, torch.ones_like(e))
    seg = torch.zeros(E + 2, dtype=torch.long, device=dev)
    seg[1:] = torch.cumsum((load + 127) // 128 * 128, 0)
    start = torch.cumsum(load, 0) - load
    order = torch.argsort(e, stable=True)
    es = e[order]
    row = seg[es] + torch.arange(T * k, device=dev) - start[es]
    row = torch.where(es < E, row, -1)
    row_of = torch.empty(T * k, dtype=torch.int32, device=dev)
    row_of[order] = row.int()
    row_token = torch.full((rows + 1,), -1, dtype=torch.int32, device=dev)
    row_token[torch.where(row < 0, rows, row)] = (order // k).int()
    row_token[rows] = -1
    return seg[:E + 1].int(), row_of.view(T, k), row_token[:rows].contiguous(), load[:E].int()


def _logits(T, E, g, dev):
    """Router logits of a trained model: per-expert popularity plus per-token variation."""
    pop = 0.3 * torch.randn(E, device=dev, generator=g)
    return pop, torch.randn((T, E), device=dev, generator=g) + pop


def _undecided(logits, case, bias):
    """Tokens whose choice hangs on the rounding of a score: two neighbours of the ranking up to the first one
    left out (of the groups: the last one taken and the first left out) differ, but by less than 1e-5 of their
    size.  Equal scores are decided (the lower index wins) and stay."""
    x = logits.double()
    s = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, 1)
    s = torch.where(torch.isinf(x), torch.full_like(s, -math.inf), s if bias is None else s + bias.double())
    T, E = s.shape
    G, tg = case["n_group"], case["topk_group"]

    def close(a, b):
        d = (a - b).abs()
        return (d > 0) & (d < 1e-5 * torch.maximum(a.abs(), b.abs())) & torch.isfinite(d)

    bad = torch.zeros(T, dtype=torch.bool, device=s.device)
    if tg < G:
        v = torch.sort(s.view(T, G, E // G), dim=2, descending=True)[0][:, :, :min(case["group_top"], E // G)]
        v = torch.where(torch.isinf(v), torch.zeros_like(v), v).sum(2)
        gs, gi = torch.sort(v, dim=1, descending=True, stable=True)
        bad |= close(gs[:, tg - 1], gs[:, tg])
        keep = torch.zeros((T, G), dtype=torch.bool, device=s.device).scatter_(1, gi[:, :tg], True)
        s = torch.where(keep.repeat_interleave(E // G, 1), s, torch.full_like(s, -math.inf))
    top = torch.sort(s, dim=1, descending=True)[0][:, :case["k"] + 1]
    return bad | close(top[:, :-1], top[:, 1:]).any(1)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    st = dict(case=case)
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        dt = _DT[case["dtype"]]
        pop, x = _logits(T, E, g, dev)
        x = x.to(dt)
        off = torch.zeros(E, dtype=torch.bool, device=dev)
        if case["offline"]:  # one expert in 16 is out of service: its logit is -inf for every token
            off[torch.randperm(E, device=dev, generator=g)[:max(1, E // 16)]] = True
        x = x.masked_fill(off, -math.inf)
        bias = 0.05 * torch.randn(E, device=dev, generator=g) if case["bias"] else None
        for _ in range(20):
            redo = _undecided(x, case, bias)
            n = int(redo.sum())
            if n == 0:
                break
            x[redo] = (torch.randn((n, E), device=dev, generator=g) + pop).to(dt).masked_fill(off, -math.inf)
        rows = _capacity(T, E, k)
        i32 = dict(dtype=torch.int32, device=dev)
        st.update(logits=x, bias=bias, rows=rows,
                  workspace=torch.empty(4 * E * ((T + 63) // 64) + 64, dtype=torch.uint8, device=dev),
                  out=(torch.empty((T, k), **i32), torch.empty((T, k), device=dev), torch.empty(E + 1, **i32),
                       torch.empty((T, k), **i32), torch.empty(rows, **i32), torch.empty(E, **i32)))
        return st
    if op == "route_backward":
        T, E, k = case["T"], case["E"], case["k"]
        _, x = _logits(T, E, g, dev)
        x = x.to(_DT[case["dtype"]])
        st.update(logits=x, idx=torch.sort(x.float(), dim=1, descending=True, stable=True)[1][:, :k].int().contiguous(),
                  grad=torch.randn((T, k), device=dev, generator=g), out=torch.empty_like(x))
        return st
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        st.update(x=_tokens(M, K, g, dev), c=torch.zeros((M, N), dtype=_DT[case["dtype"]], device=dev),
                  q=torch.empty((M, K), dtype=torch.int8, device=dev), s=torch.empty(M, device=dev))
        st["qw"], st["sw"] = _weights((N, K), g, dev)
        return st
    T, E, k = case["T"], case["E"], case["k"]
    rows = _capacity(T, E, k)
    _, x = _logits(T, E, g, dev)
    top, idx = torch.sort(x, dim=1, descending=True, stable=True)
    offsets, row_of, row_token, _ = _layout(idx[:, :k].int(), E, rows)
    st.update(offsets=offsets, row_of=row_of, row_token=row_token, weight=torch.softmax(top[:, :k], 1).contiguous())
    if op == "experts":
        N, K = case["N"], case["K"]
        # Rows past the layout's end are not written by the operator; the buffer starts as zeros.
        st.update(x=_tokens(T, K, g, dev), c=torch.zeros((rows, N), dtype=_DT[case["dtype"]], device=dev),
                  q=torch.empty((T, K), dtype=torch.int8, device=dev), s=torch.empty(T, device=dev))
        st["qw"], st["sw"] = _weights((E, N, K), g, dev)
        return st
    H, dt = case["H"], _DT[case["dtype"]]
    c = torch.randn((rows, H), device=dev, generator=g).to(dt)
    c[row_token < 0] = 0  # empty rows are zeros, as the grouped products leave them
    st["c"] = c
    if op == "combine":
        st.update(add=torch.randn((T, H), device=dev, generator=g).to(dt) if case["add"] else None,
                  y=torch.empty((T, H), dtype=dt, device=dev))
    else:
        st.update(grad=torch.randn((T, H), device=dev, generator=g).to(dt),
                  grad_c=torch.zeros((rows, H), dtype=dt, device=dev), grad_w=torch.empty((T, k), device=dev))
    return st


def _tokens(M, K, g, dev):
    """bf16 activations ~ N(0, 1) with one channel in a hundred 20 times as large."""
    x = torch.randn((M, K), device=dev, generator=g)
    x[:, torch.randperm(K, device=dev, generator=g)[:K // 100]] *= 20.0
    return x.to(torch.bfloat16)


def _weights(shape, g, dev):
    """INT8 weights as a user keeps them: normal values whose largest of a few thousand takes code +-127, and
    one scale per output channel."""
    q = torch.empty(shape, dtype=torch.int8, device=dev)
    flat = q.view(-1)
    for i in range(0, flat.numel(), 1 << 27):
        n = min(1 << 27, flat.numel() - i)
        flat[i:i + n] = (33.0 * torch.randn(n, device=dev, generator=g)).round().clamp(-127, 127).to(torch.int8)
    return q, (0.02 / 33.0) * (0.8 + 0.4 * torch.rand(shape[:-1], device=dev, generator=g))


# --------------------------------------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------------------------------------

def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state, state["case"])


def _own_route(st, c):
    import fine_grained_quantization_amd as fq

    idx, w, off, row_of, row_token, load = fq.fp8q_moe_gate_topk(
        st["logits"], c["k"], score=c["score"], bias=st["bias"], n_group=c["n_group"], topk_group=c["topk_group"],
        group_top=c["group_top"], renormalize=c["renorm"], scale=c["scale"], rows=st["rows"],
        workspace=st["workspace"], out=st["out"])
    return dict(idx=idx, weight=w, offsets=off, row_of=row_of, row_token=row_token, load=load)


def _own_route_backward(st, c):
    import fine_grained_quantization_amd as fq

    return fq.fp8q_moe_gate_backward(st["logits"], st["idx"], st["grad"], score=c["score"], renormalize=c["renorm"],
                                     scale=c["scale"], grad_logits=st["out"])


def _own_combine(st, c):
    import fine_grained_quantization_amd as fq

    return fq.fp8q_moe_combine(st["c"], st["row_of"], st["weight"], add=st["add"], y=st["y"])


def _own_combine_backward(st, c):
    import fine_grained_quantization_amd as fq

    dc, dw = fq.fp8q_moe_combine_backward(st["grad"], st["c"], st["row_of"], st["weight"], st["row_token"],
                                          st["offsets"], grad_c=st["grad_c"], grad_weight=st["grad_w"])
    return dict(grad_c=dc, grad_weight=dw)


def _own_linear(st, c):
    import fine_grained_quantization_amd as fq

    q, s = fq.fp8q_quant_int8(st["x"], q=st["q"], s=st["s"])
    return fq.fp8q_gemm_int8(q, s, st["qw"], st["sw"], out_dtype=_DT[c["dtype"]], c=st["c"])


def _own_experts(st, c):
    import fine_grained_quantization_amd as fq

    q, s = fq.fp8q_quant_int8(st["x"], q=st["q"], s=st["s"])
    return fq.fp8q_grouped_gemm_int8_gather(q, s, st["row_token"], st["qw"], st["sw"], st["offsets"],
                                            out_dtype=_DT[c["dtype"]], c=st["c"])


_own = dict(route=_own_route, route_backward=_own_route_backward, combine=_own_combine,
            combine_backward=_own_combine_backward, linear=_own_linear, experts=_own_experts)


def _scores(x, kind):
    x = x.float().clamp(max=BIG)
    if kind == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    e = torch.exp(x - x.max(1, keepdim=True)[0].clamp(min=-BIG))
    return e / e.sum(1, keepdim=True).clamp(min=1e-30)


def _plain_route(st, c):
    x, k, G = st["logits"], c["k"], c["n_group"]
    T, E = x.shape
    s = _scores(x, c["score"])
    gone = torch.isneginf(x)
    key = (s if st["bias"] is None else s + st["bias"]).masked_fill(gone, -math.inf)
    if c["topk_group"] < G:
        v = torch.sort(key.view(T, G, E // G), dim=2, descending=True)[0][:, :, :min(c["group_top"], E // G)]
        v = torch.where(torch.isneginf(v[:, :, 0]), v[:, :, 0], v.clamp(min=-BIG).masked_fill(torch.isneginf(v), 0.0).sum(2))
        best = torch.sort(v, dim=1, descending=True, stable=True)[1][:, :c["topk_group"]]
        keep = torch.zeros((T, G), dtype=torch.bool, device=x.device).scatter_(1, best, True)
        key = key.masked_fill(~keep.repeat_interleave(E // G, 1), -math.inf)
    val, idx = torch.sort(key, dim=1, descending=True, stable=True)
    val, idx = val[:, :k], idx[:, :k]
    none = torch.isneginf(val)
    w = torch.gather(s, 1, idx).masked_fill(none, 0.0)
    if c["renorm"]:
        w = w / (w.sum(1, keepdim=True) + EPS)
    idx = idx.masked_fill(none, -1).int()
    off, row_of, row_token, load = _layout(idx, E, st["rows"])
    return dict(idx=idx, weight=w * c["scale"], offsets=off, row_of=row_of, row_token=row_token, load=load)


def _plain_route_backward(st, c):
    s = _scores(st["logits"], c["score"])
    idx, d = st["idx"].long(), st["grad"] * c["scale"]
    v = torch.gather(s, 1, idx)
    if c["renorm"]:
        total = v.sum(1, keepdim=True) + EPS
        d = (d - (d * v).sum(1, keepdim=True) / total) / total
    ds = torch.zeros_like(s).scatter_(1, idx, d)
    if c["score"] == "sigmoid":
        return (ds * s * (1.0 - s)).to(st["logits"].dtype)
    return (s * (ds - (ds * s).sum(1, keepdim=True))).to(st["logits"].dtype)


def _plain_combine(st, c):
    v = st["c"].float()[st["row_of"].long()]  # [T, k, H]
    y = (v * st["weight"][:, :, None]).sum(1)
    if st["add"] is not None:
        y = y + st["add"].float()
    return y.to(st["c"].dtype)


def _plain_combine_backward(st, c):
    row, g = st["row_of"].long(), st["grad"].float()
    dw = (st["c"].float()[row] * g[:, None, :]).sum(2)
    dc = torch.zeros(st["c"].shape, device=g.device)
    dc[row.reshape(-1)] = (st["weight"][:, :, None] * g[:, None, :]).reshape(-1, g.shape[1])
    return dict(grad_c=dc.to(st["c"].dtype), grad_weight=dw)


def _plain_quant(x):
    x = x.float()
    amax = x.abs().amax(1)
    s = amax / torch.full_like(amax, 127.0)
    return torch.where(s[:, None] > 0, x / s[:, None], torch.zeros_like(x)).round().clamp(-127, 127), s


def _plain_linear(st, c):
    q, s = _plain_quant(st["x"])
    return ((q @ st["qw"].float().t()) * (s[:, None] * st["sw"][None, :])).to(_DT[c["dtype"]])


def _plain_experts(st, c):
    q, s = _plain_quant(st["x"])
    E, N, K = st["qw"].shape
    tok = st["row_token"].long()
    q = torch.cat([q, torch.zeros_like(q[:1])])[tok]  # token -1: a row of zeros
    s = torch.cat([s, torch.zeros_like(s[:1])])[tok]
    # Every 128 rows belong to one expert.
    first = torch.arange(0, tok.numel(), 128, device=tok.device, dtype=torch.int32)
    e = torch.searchsorted(st["offsets"][1:].contiguous(), first, right=True).clamp(max=E - 1)
    acc = torch.bmm(q.view(-1, 128, K), st["qw"][e].float().transpose(1, 2))
    return (acc * (s.view(-1, 128, 1) * st["sw"][e][:, None, :])).view(-1, N).to(_DT[c["dtype"]])


_plain = dict(route=_plain_route, route_backward=_plain_route_backward, combine=_plain_combine,
              combine_backward=_plain_combine_backward, linear=_plain_linear, experts=_plain_experts)


# --------------------------------------------------------------------------------------------------------
# The definition in 64 bits
# --------------------------------------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("route", "route_backward"):
        x = st["logits"].double()
        gone = x == -math.inf
        p = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, dim=1)
        if op == "route_backward":
            leaf = x.clone().requires_grad_(True)
            p = torch.sigmoid(leaf) if case["score"] == "sigmoid" else torch.softmax(leaf, dim=1)
            w = p.gather(1, st["idx"].long())
            if case["renorm"]:
                w = w / (w.sum(dim=1, keepdim=True) + EPS)
            (w * case["scale"]).backward(st["grad"].double())
            return leaf.grad
        rank = p if st["bias"] is None else p + st["bias"].double()
        rank = rank.masked_fill(gone, -math.inf)
        G, size = case["n_group"], case["E"] // case["n_group"]
        if case["topk_group"] < G:
            parts = rank.unflatten(1, (G, size)).topk(min(case["group_top"], size), dim=2).values
            total = parts.nan_to_num(neginf=0.0).sum(dim=2).masked_fill(parts[:, :, 0] == -math.inf, -math.inf)
            left_out = total.argsort(dim=1, descending=True, stable=True)[:, case["topk_group"]:]
            out = torch.zeros_like(total, dtype=torch.bool).scatter(1, left_out, True)
            rank = rank.unflatten(1, (G, size)).masked_fill(out[:, :, None], -math.inf).flatten(1)
        chosen = rank.argsort(dim=1, descending=True, stable=True)[:, :case["k"]]
        w = p.gather(1, chosen) * (rank.gather(1, chosen) > -math.inf)
        if case["renorm"]:
            w = w / (w.sum(dim=1, keepdim=True) + EPS)
        return dict(idx=None, weight=w * case["scale"], offsets=None, row_of=None, row_token=None, load=None)
    if op == "combine":
        y = torch.zeros((case["T"], case["H"]), dtype=torch.float64, device="cuda") if st["add"] is None else st["add"].double()
        for j in range(case["k"]):
            y += st["weight"][:, j:j + 1].double() * st["c"].index_select(0, st["row_of"][:, j].long()).double()
        return y
    if op == "combine_backward":
        g = st["grad"].double()
        dc = torch.zeros(st["c"].shape, dtype=torch.float64, device="cuda")
        dw = []
        for j in range(case["k"]):
            at = st["row_of"][:, j].long()
            dc.index_copy_(0, at, st["weight"][:, j:j + 1].double() * g)
            dw.append(torch.linalg.vecdot(st["c"].index_select(0, at).double(), g))
        return dict(grad_c=dc, grad_weight=torch.stack(dw, dim=1))
    # INT8 products: a token's scale is its largest magnitude over 127, rounded to 32 bits, and its codes are the
    # 32-bit quotients rounded to whole numbers; both are parts of the definition.
    x = st["x"].double()
    sa = (x.abs().max(dim=1, keepdim=True).values / 127.0).float().double()
    q = torch.round((x / sa.clamp(min=1e-300)).float()).double()
    if op == "linear":
        return sa * (q @ st["qw"].double().t()) * st["sw"].double()
    c = torch.zeros(st["c"].shape, dtype=torch.float64, device="cuda")
    bounds = st["offsets"].tolist()
    for e in range(case["E"]):
        t = st["row_token"][bounds[e]:bounds[e + 1]].long()
        at = torch.nonzero(t >= 0).flatten()
        t = t[at]
        c[bounds[e] + at] = sa[t] * (q[t] @ st["qw"][e].double().t()) * st["sw"][e].double()
    return c


# --------------------------------------------------------------------------------------------------------
# What a pass cannot do without
# --------------------------------------------------------------------------------------------------------

def work(case):
    op = case["op"]
    size = 2 if case["dtype"] == "bf16" else 4
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return dict(bytes=2 * M * K + N * K + 4 * N + size * M * N, flops=2 * M * N * K)
    T, E, k = case["T"], case["E"], case["k"]
    if op == "route":  # logits; expert, weight and row per slot; the token of every row; offsets and loads
        return dict(bytes=size * T * E + 12 * T * k + 4 * _capacity(T, E, k) + 8 * E, flops=0)
    if op == "route_backward":
        return dict(bytes=2 * size * T * E + 8 * T * k, flops=0)
    if op == "combine":
        H = case["H"]
        return dict(bytes=size * T * H * (k + 1 + bool(case["add"])) + 8 * T * k, flops=2 * T * k * H)
    if op == "combine_backward":
        H = case["H"]
        return dict(bytes=size * T * H * (2 * k + 1) + 12 * T * k, flops=3 * T * k * H)
    N, K = case["N"], case["K"]
    used = E * (1.0 - (1.0 - k / E) ** T)  # experts that some token reaches
    return dict(bytes=int(2 * T * K + used * N * (K + 4) + size * T * k * N + 4 * T * k), flops=2 * T * k * N * K)
