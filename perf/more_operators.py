"""Cases that time the root-mean-square norm in front of an FP8 Linear and the backward pass from 8-bit checkpoints.

Each case is one pass through one operator.  ``run`` computes it either through this package's entry points
(``own`` is true) or in a plain form of elementary torch operations in 32 bits (``own`` is false); ``exact``
gives the same answer from the definition in 64 bits.  The operators:

  norm             residual + x in bf16, its root-mean-square norm times a weight, in 1x128 E4M3 groups
  norm_backward    the norm's gradients: of its input (the residual's gradient added) and of its weight
  swiglu_backward  SwiGLU recomputed from its 8-bit inputs: their gradients in 1x128 groups and transposed (groups of
                   128 tokens, power-of-two scales), and the recomputed output transposed
  transpose        the transposed copy of an 8-bit checkpoint, or of a bf16 gradient, routed rows included
  wgrad            a Linear's weight gradient from two transposed copies, added to an older one where asked
  wgrad_experts    the same for every expert of an expert-sorted layout

Codes come back as float8_e4m3fn and power-of-two scales as float8_e8m0fnu: the values that they stand for.
"""
import math

import torch

own = False

EPS = 1e-6


def listed():
    return [
        # One token of a serving step in front of a projection: launch latency.
        dict(name="norm 1x7168", op="norm", M=1, K=7168, residual=True, y=False, pow2=False, weight="bf16"),
        # A prompt, or a training microbatch, in front of the up projection.
        dict(name="norm 4096x7168", op="norm", M=4096, K=7168, residual=True, y=False, pow2=False, weight="bf16"),
        # The first norm of a model (nothing to add) in front of a router, which reads the bf16 output too; odd tokens.
        dict(name="norm 1021x2048", op="norm", M=1021, K=2048, residual=False, y=True, pow2=True, weight="f32"),
        # Training: the same norm's gradients.
        dict(name="norm backward 4096x7168", op="norm_backward", M=4096, K=7168, residual=True, weight="bf16"),
        # A short sequence's.
        dict(name="norm backward 61x2048", op="norm_backward", M=61, K=2048, residual=False, weight="f32"),
        # Training: the dense feed-forward's gate and up projections.
        dict(name="swiglu backward 4096x18432", op="swiglu_backward", M=4096, F=18432),
        # An expert's width and a ragged token count.
        dict(name="swiglu backward 77x2048", op="swiglu_backward", M=77, F=2048),
        # The tokens' checkpoint brought into the rows of 64 experts for their weight gradients.
        dict(name="transpose 8192 routed", op="transpose", src="codes", T=8192, K=7168, E=64, k=8, pow2=True),
        # The gradient of a Linear's output, an odd token count.
        dict(name="transpose 1037x7168 bf16", op="transpose", src="bf16", T=1037, K=7168, E=0, k=0, pow2=False),
        # The up projection's weight gradient, accumulated in fp32 over microbatches.
        dict(name="wgrad 4096x18432x7168", op="wgrad", M=4096, N=18432, K=7168, dtype="f32", accumulate=True),
        # A small Linear and few tokens: neither dimension is a multiple of a tile.
        dict(name="wgrad 300x576x2064", op="wgrad", M=300, N=576, K=2064, dtype="bf16", accumulate=False),
        # 64 experts' weight gradients of one microbatch.
        dict(name="wgrad experts 8192", op="wgrad_experts", T=8192, E=64, k=8, N=2048, K=7168, dtype="bf16",
             accumulate=False),
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of ``step`` in [lo, hi], spread evenly over the logarithm; odd multiples come up too."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    return min(max(v, lo), hi // step * step)


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "swiglu_backward", "transpose", "wgrad", "wgrad_experts"])
    if op in ("norm", "norm_backward"):
        d = dict(op=op, M=_spread(rng, 1, 8192), K=_spread(rng, 128, 18432, 128), residual=rng.random() < 0.6,
                 weight=rng.choice(["bf16", "f32"]))
        if op == "norm":
            d.update(y=rng.random() < 0.3, pow2=rng.random() < 0.3)
        return d
    if op == "swiglu_backward":
        return dict(op=op, M=_spread(rng, 1, 4096), F=_spread(rng, 128, 18432, 128))
    if op == "transpose":
        E = rng.choice([0, 0, _spread(rng, 4, 64)])
        return dict(op=op, src=rng.choice(["codes", "bf16"]), T=_spread(rng, 1, 8192), K=_spread(rng, 128, 7168, 128),
                    E=E, k=rng.randint(1, min(8, E)) if E else 0, pow2=rng.random() < 0.5)
    if op == "wgrad":
        d = dict(op=op, M=_spread(rng, 1, 8192), N=_spread(rng, 64, 18432, 16), K=_spread(rng, 64, 18432, 16),
                 dtype=rng.choice(["f32", "f32", "bf16"]), accumulate=rng.random() < 0.5)
        while d["M"] * d["N"] * d["K"] > 4096 * 18432 * 7168:
            d["M"] = (d["M"] + 1) // 2
        while d["N"] * d["K"] > 18432 * 7168:
            d["N"] = (d["N"] // 2 + 15) // 16 * 16
        return d
    E = _spread(rng, 4, 64)
    return dict(op=op, T=_spread(rng, 1, 8192), E=E, k=rng.randint(1, min(8, E)), N=_spread(rng, 128, 2048, 16),
                K=_spread(rng, 128, 7168, 16), dtype=rng.choice(["f32", "bf16"]), accumulate=rng.random() < 0.3)


# --------------------------------------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------------------------------------

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _blocks(n):
    return (n + 127) // 128


def _capacity(T, E, k):
    return (T * k + 127 * E + 127) // 128 * 128


def _layout(T, E, k, g, dev):
    """An expert-sorted layout of T tokens to k of E experts of uneven popularity: segment starts (each padded to 128
    rows), every row's token (-1: none) and the longest segment."""
    pop = 0.3 * torch.randn(E, device=dev, generator=g)
    idx = torch.sort(torch.randn((T, E), device=dev, generator=g) + pop, dim=1, descending=True)[1][:, :k].reshape(-1)
    load = torch.bincount(idx, minlength=E)
    seg = torch.zeros(E + 1, dtype=torch.long, device=dev)
    seg[1:] = torch.cumsum((load + 127) // 128 * 128, 0)
    first = torch.cumsum(load, 0) - load
    order = torch.argsort(idx, stable=True)
    row = seg[idx[order]] + torch.arange(T * k, device=dev) - first[idx[order]]
    row_token = torch.full((_capacity(T, E, k),), -1, dtype=torch.int32, device=dev)
    row_token[row] = (order // k).int()
    return seg.int(), row_token, int((seg[1:] - seg[:-1]).max())


def _activations(M, K, g, dev):
    """bf16 ~ N(0, 1) with one channel in a hundred 20 times as large."""
    x = torch.randn((M, K), device=dev, generator=g)
    x[:, torch.randperm(K, device=dev, generator=g)[:K // 100]] *= 20.0
    return x.to(torch.bfloat16)


def _gradient(M, K, g, dev):
    """bf16 gradients: small values, tokens of different sizes."""
    x = 1e-3 * torch.randn((M, K), device=dev, generator=g)
    return (x * torch.exp(torch.randn((M, 1), device=dev, generator=g))).to(torch.bfloat16)


def _codes(rows, cols, g, dev):
    """E4M3 codes whose largest of 128 are about the largest the format has."""
    q = torch.empty((rows, cols), dtype=torch.uint8, device=dev)
    step = max(1, (1 << 27) // cols)
    for i in range(0, rows, step):
        v = 130.0 * torch.randn((min(step, rows - i), cols), device=dev, generator=g)
        q[i:i + step] = v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return q


def _transposed(C, cols, g, dev):
    """A transposed copy of ``cols`` tokens: codes [C, cols], power-of-two scales [cols / 128, C] of a few sizes."""
    return _codes(C, cols, g, dev), torch.randint(117, 123, (cols // 128, C), dtype=torch.uint8, device=dev, generator=g)


def _checkpoint(M, K, pow2, g, dev):
    """A 1x128 checkpoint: codes [M, K], fp32 scales [K / 128, M]."""
    s = 0.002 * torch.exp(0.5 * torch.randn((K // 128, M), device=dev, generator=g))
    return _codes(M, K, g, dev), torch.exp2(torch.round(torch.log2(s))) if pow2 else s


def _weight(K, kind, g, dev):
    return (1.0 + 0.2 * torch.randn(K, device=dev, generator=g)).to(_DT[kind])


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    st = dict(case=case)
    op = case["op"]
    u8 = dict(dtype=torch.uint8, device=dev)
    bf = dict(dtype=torch.bfloat16, device=dev)
    if op in ("norm", "norm_backward"):
        M, K = case["M"], case["K"]
        st["w"] = _weight(K, case["weight"], g, dev)
        st["x"] = _activations(M, K, g, dev)
        if op == "norm":
            st["residual"] = _activations(M, K, g, dev) if case["residual"] else None
            st.update(h=torch.empty((M, K), **bf) if case["residual"] else None, y=torch.empty((M, K), **bf) if case["y"] else None,
                      q=torch.empty((M, K), **u8), s=torch.empty((K // 128, M), device=dev), rstd=torch.empty(M, device=dev))
        else:
            st["rstd"] = torch.rsqrt(st["x"].float().square().mean(1) + EPS)
            st["gy"] = _gradient(M, K, g, dev)
            st["gres"] = _gradient(M, K, g, dev) if case["residual"] else None
            st.update(gx=torch.empty((M, K), **bf), gw=torch.empty(K, device=dev))
        return st
    if op == "swiglu_backward":
        M, F = case["M"], case["F"]
        Mp = 128 * _blocks(M)
        st["q"], st["s"] = _checkpoint(M, 2 * F, False, g, dev)
        st["gh"] = _gradient(M, F, g, dev)
        st["out"] = (torch.empty((M, 2 * F), **u8), torch.empty((2 * F // 128, M), device=dev),
                     torch.empty((2 * F, Mp), **u8), torch.empty((Mp // 128, 2 * F), **u8),
                     torch.empty((F, Mp), **u8), torch.empty((Mp // 128, F), **u8))
        return st
    if op == "transpose":
        T, K, E = case["T"], case["K"], case["E"]
        st["row_token"] = _layout(T, E, case["k"], g, dev)[1] if E else None
        rows = st["row_token"].numel() if E else T
        if case["src"] == "codes":
            st["q"], st["s"] = _checkpoint(T, K, case["pow2"], g, dev)
        else:
            st["x"] = _gradient(T, K, g, dev)
        st["out"] = (torch.empty((K, 128 * _blocks(rows)), **u8), torch.empty((_blocks(rows), K), **u8))
        return st
    N, K, dt = case["N"], case["K"], _DT[case["dtype"]]
    if op == "wgrad":
        M, shape = case["M"], (N, K)
        cols = 128 * _blocks(M)
        gone = torch.arange(cols, device=dev) >= M
    else:
        shape = (case["E"], N, K)
        st["offsets"], row_token, st["longest"] = _layout(case["T"], case["E"], case["k"], g, dev)
        cols = row_token.numel()
        gone = row_token < 0
    st["gt"], st["eg"] = _transposed(N, cols, g, dev)
    st["xt"], st["ex"] = _transposed(K, cols, g, dev)
    st["gt"][:, gone] = 0  # columns of no token hold zeros
    st["xt"][:, gone] = 0
    st["dw"] = torch.randn(shape, device=dev, generator=g).to(dt) if case["accumulate"] else torch.empty(shape, dtype=dt, device=dev)
    return st


# --------------------------------------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------------------------------------

def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state, state["case"])


def _named(names, tensors):
    """Outputs by name, 8-bit codes and scales as the values that they stand for."""
    kinds = dict(q=torch.float8_e4m3fn, qt=torch.float8_e4m3fn, ht=torch.float8_e4m3fn, et=torch.float8_e8m0fnu,
                 eh=torch.float8_e8m0fnu)
    return {n: t.view(kinds[n]) if t.dtype == torch.uint8 else t for n, t in zip(names, tensors) if t is not None}


def _own_norm(st, c):
    import fine_grained_quantization_amd as fq

    q, s, h, rstd = fq.fp8q_rmsnorm_quant_act_1x128(st["x"], st["w"], residual=st["residual"], eps=EPS, pow2=c["pow2"],
                                                    h=st["h"], q=st["q"], s=st["s"], rstd=st["rstd"], y=st["y"])
    return _named(("q", "s", "h", "rstd", "y"), (q, s, h if c["residual"] else None, rstd, st["y"]))


def _own_norm_backward(st, c):
    import fine_grained_quantization_amd as fq

    gx, gw = fq.fp8q_rmsnorm_backward(st["gy"], st["x"], st["w"], st["rstd"], gres=st["gres"], gx=st["gx"], gw=st["gw"])
    return dict(gx=gx, gw=gw)


def _own_swiglu_backward(st, c):
    import fine_grained_quantization_amd as fq

    return _named(("q", "s", "qt", "et", "ht", "eh"), fq.fp8q_swiglu_backward_quant(st["q"], st["s"], st["gh"], out=st["out"]))


def _own_transpose(st, c):
    import fine_grained_quantization_amd as fq

    qt, et = st["out"]
    if c["src"] == "codes":
        return _named(("qt", "et"), fq.fp8q_transpose_act_128x1(st["q"], st["s"], row_token=st["row_token"], qt=qt, et=et))
    return _named(("qt", "et"), fq.fp8q_quant_act_128x1(st["x"], row_token=st["row_token"], qt=qt, et=et))


def _own_wgrad(st, c):
    import fine_grained_quantization_amd as fq

    return fq.fp8q_gemm_wgrad(st["gt"], st["eg"], st["xt"], st["ex"], out_dtype=_DT[c["dtype"]],
                              accumulate=c["accumulate"], dw=st["dw"])


def _own_wgrad_experts(st, c):
    import fine_grained_quantization_amd as fq

    return fq.fp8q_grouped_gemm_wgrad(st["gt"], st["eg"], st["xt"], st["ex"], st["offsets"], out_dtype=_DT[c["dtype"]],
                                      accumulate=c["accumulate"], dw=st["dw"])


_own = dict(norm=_own_norm, norm_backward=_own_norm_backward, swiglu_backward=_own_swiglu_backward,
            transpose=_own_transpose, wgrad=_own_wgrad, wgrad_experts=_own_wgrad_experts)


def _pow2_byte(amax):
    """The byte (exponent + 127) of the least power of two that brings ``amax`` to 448 or less; 0 for a group of zeros."""
    m, e = torch.frexp(amax)
    return torch.where(amax > 0, (e - 9 + (m > 0.875) + 127).clamp(0, 254), torch.zeros_like(e)).to(torch.uint8)


def _pow2_value(byte):
    return torch.ldexp(torch.ones((), device=byte.device), byte.int() - 127)


def _encode(v):
    return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _plain_1x128(y, pow2=False):
    """1x128 groups of fp32 values: codes [M, K] and fp32 scales [K / 128, M]."""
    M, K = y.shape
    v = y.view(M, K // 128, 128)
    amax = v.abs().amax(2)
    s = _pow2_value(_pow2_byte(amax)) if pow2 else amax / torch.full_like(amax, 448.0)
    s = torch.where(amax > 0, s, torch.zeros_like(s))
    q = torch.where(s[:, :, None] > 0, v / s[:, :, None], v)
    return _encode(q).view(M, K), s.t().contiguous()


def _plain_128x1(v):
    """Groups of 128 tokens of fp32 values [M, C], transposed: codes [C, Mp] and scale bytes [Mp / 128, C]."""
    M, C = v.shape
    nb = _blocks(M)
    v = torch.cat([v, torch.zeros((128 * nb - M, C), device=v.device)]).view(nb, 128, C)
    e = _pow2_byte(v.abs().amax(1))
    q = _encode(v / _pow2_value(e)[:, None, :])
    return q.view(torch.uint8).view(nb * 128, C).t().contiguous(), e


def _plain_decode(q, s):
    """fp32 values of a 1x128 checkpoint."""
    M, K = q.shape
    return (q.view(torch.float8_e4m3fn).float().view(M, K // 128, 128) * s.t()[:, :, None]).view(M, K)


def _plain_norm(st, c):
    h = st["x"] if st["residual"] is None else (st["x"].float() + st["residual"].float()).to(torch.bfloat16)
    hf = h.float()
    rstd = torch.rsqrt(hf.square().mean(1) + EPS)
    y = hf * rstd[:, None] * st["w"].float()
    q, s = _plain_1x128(y, c["pow2"])
    return _named(("q", "s", "h", "rstd", "y"),
                  (q, s, h if c["residual"] else None, rstd, y.to(torch.bfloat16) if c["y"] else None))


def _plain_norm_backward(st, c):
    h, g, r = st["x"].float(), st["gy"].float(), st["rstd"][:, None]
    gh = g * h * r
    gx = r * (g * st["w"].float() - h * r * (gh * st["w"].float()).mean(1, keepdim=True))
    if st["gres"] is not None:
        gx = gx + st["gres"].float()
    return dict(gx=gx.to(torch.bfloat16), gw=gh.sum(0))


def _plain_swiglu_backward(st, c):
    x, u = _plain_decode(st["q"], st["s"]).chunk(2, dim=1)
    g = st["gh"].float()
    sig = 1.0 / (1.0 + torch.exp(-x))
    silu = x * sig
    d = torch.cat([g * u * (sig * (1.0 + x * (1.0 - sig))), g * silu], dim=1)
    return _named(("q", "s", "qt", "et", "ht", "eh"), (*_plain_1x128(d), *_plain_128x1(d), *_plain_128x1(silu * u)))


def _plain_transpose(st, c):
    v = _plain_decode(st["q"], st["s"]) if c["src"] == "codes" else st["x"].float()
    if st["row_token"] is not None:
        v = torch.cat([v, torch.zeros_like(v[:1])])[st["row_token"].long()]  # token -1: a row of zeros
    return _named(("qt", "et"), _plain_128x1(v))


def _plain_untransposed(qt, et):
    """fp32 values [C, cols] of a transposed copy."""
    C, cols = qt.shape
    return (qt.view(torch.float8_e4m3fn).float().view(C, cols // 128, 128) * _pow2_value(et).t()[:, :, None]).view(C, cols)


def _plain_store(st, c, acc):
    if c["accumulate"]:
        st["dw"].copy_(acc.add_(st["dw"]))
        return st["dw"]
    return acc.to(_DT[c["dtype"]])


def _plain_wgrad(st, c):
    return _plain_store(st, c, _plain_untransposed(st["gt"], st["eg"]) @ _plain_untransposed(st["xt"], st["ex"]).t())


def _plain_wgrad_experts(st, c):
    E, L = c["E"], st["longest"]
    at = st["offsets"][:-1, None].long() + torch.arange(L, device=st["gt"].device)  # [E, L]
    there = at < st["offsets"][1:, None]
    at = torch.where(there, at, torch.zeros_like(at)).view(-1)
    gs = _plain_untransposed(st["gt"], st["eg"]).t()[at].view(E, L, c["N"]) * there[:, :, None]
    xs = _plain_untransposed(st["xt"], st["ex"]).t()[at].view(E, L, c["K"])
    return _plain_store(st, c, torch.bmm(gs.transpose(1, 2).contiguous(), xs))


_plain = dict(norm=_plain_norm, norm_backward=_plain_norm_backward, swiglu_backward=_plain_swiglu_backward,
              transpose=_plain_transpose, wgrad=_plain_wgrad, wgrad_experts=_plain_wgrad_experts)


# --------------------------------------------------------------------------------------------------------
# The definition in 64 bits
# --------------------------------------------------------------------------------------------------------

def _e4m3(v):
    """Nearest E4M3 value of a float64, ties to even: steps of 2^-9 below 2^-6, of an eighth of the power of two above."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3.0)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _least_power(amax):
    """The least power of two p (at least 2^-127) with amax <= 448 p."""
    e = torch.ceil(torch.log2(amax.clamp(min=1e-300) / 448.0)).clamp(min=-127.0)
    p = torch.exp2(e)
    p = torch.where(amax > 448.0 * p, 2.0 * p, p)  # a logarithm on the wrong side of a whole number
    return torch.where((amax <= 224.0 * p) & (e > -127.0), 0.5 * p, p)


def _exact_rows(t, pow2=False, factor=None):
    """Codes and scales of ``t`` times a factor of each row.  (t / (top / 448) does not depend on the factor, and products
    of bf16 values often lie right between two codes: a factor's rounding would decide those.)"""
    groups = (t * factor if pow2 and factor is not None else t).unflatten(1, (-1, 128))
    top = groups.abs().max(dim=2, keepdim=True).values
    gone = top == 0
    if pow2:
        s = _least_power(top).masked_fill(gone, 0.0)
        return _e4m3(groups / s.masked_fill(gone, 1.0)).flatten(1), s.squeeze(2).t()
    q = _e4m3(groups * 448.0 / top.masked_fill(gone, 1.0)).flatten(1)
    s = top.squeeze(2) / 448.0
    return q, (s if factor is None else s * factor).t()


def _exact_columns(y):
    pad = -y.shape[0] % 128
    groups = torch.nn.functional.pad(y, (0, 0, 0, pad)).unflatten(0, (-1, 128))
    p = _least_power(groups.abs().max(dim=1, keepdim=True).values)
    return _e4m3(groups / p).flatten(0, 1).t(), p.squeeze(1)


def _decoded(codes, scale):
    return codes.view(torch.float8_e4m3fn).double() * scale.double().t().repeat_interleave(128, dim=1)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = st["x"].double()
        if case["residual"]:
            h = (h + st["residual"].double()).to(torch.bfloat16).double()
        rstd = (h.pow(2).sum(dim=1, keepdim=True) / case["K"] + EPS) ** -0.5
        y = h * st["w"].double()
        q, s = _exact_rows(y, case["pow2"], rstd)
        got = dict(q=q, s=s, rstd=rstd.squeeze(1))
        if case["residual"]:
            got["h"] = h
        if case["y"]:
            got["y"] = y * rstd
        return got
    if op == "norm_backward":
        h, w = st["x"].double().requires_grad_(True), st["w"].double().requires_grad_(True)
        # (the norm with the saved reciprocal, which is the input's own but for its rounding)
        (h * (h.pow(2).mean(dim=1, keepdim=True) + EPS) ** -0.5 * w).backward(st["gy"].double())
        return dict(gx=h.grad if st["gres"] is None else h.grad + st["gres"].double(), gw=w.grad)
    if op == "swiglu_backward":
        F = case["F"]
        both = _decoded(st["q"], st["s"])
        gate, up, g = both[:, :F], both[:, F:], st["gh"].double()
        p = torch.sigmoid(gate)
        d = torch.cat([g * up * (p + gate * p * (1.0 - p)), g * gate * p], dim=1)
        h = gate * p * up
        del both, gate, up, g, p
        q, s = _exact_rows(d)
        qt, et = _exact_columns(d)
        ht, eh = _exact_columns(h)
        return dict(q=q, s=s, qt=qt, et=et, ht=ht, eh=eh)
    if op == "transpose":
        v = _decoded(st["q"], st["s"]) if case["src"] == "codes" else st["x"].double()
        if case["E"]:
            t = st["row_token"].long()
            v = v.index_select(0, t.clamp(min=0)) * (t >= 0).unsqueeze(1)
        qt, et = _exact_columns(v)
        return dict(qt=qt, et=et)
    power = [torch.exp2(e.double() - 127.0) for e in (st["eg"], st["ex"])]
    dw = st["dw"].double() if case["accumulate"] else torch.zeros(st["dw"].shape, dtype=torch.float64, device="cuda")
    bounds = st["offsets"].tolist() if op == "wgrad_experts" else [0, st["gt"].shape[1]]
    for e in range(len(bounds) - 1):
        a, b = bounds[e], bounds[e + 1]
        if a < b:
            gs, xs = (_decoded(t[:, a:b].contiguous(), p[a // 128:b // 128]) for t, p in zip((st["gt"], st["xt"]), power))
            (dw[e] if op == "wgrad_experts" else dw).add_(gs @ xs.t())
    return dw


# --------------------------------------------------------------------------------------------------------
# What a pass cannot do without
# --------------------------------------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "norm":  # x (and the residual) in; codes, scales, the sum and the bf16 output out
        M, K = case["M"], case["K"]
        res, y = bool(case["residual"]), bool(case["y"])
        return dict(bytes=M * K * (2 + 4 * res + 1 + 2 * y) + M * K // 32 + 4 * M + 4 * K, flops=6 * M * K)
    if op == "norm_backward":
        M, K = case["M"], case["K"]
        return dict(bytes=M * K * (6 + 2 * bool(case["residual"])) + 4 * M + 8 * K, flops=12 * M * K)
    if op == "swiglu_backward":  # codes and gradient in; the gradients' codes twice and the output's out
        M, F = case["M"], case["F"]
        Mp = 128 * _blocks(M)
        return dict(bytes=4 * M * F + 2 * M * F + 3 * Mp * F + 2 * M * F // 16 + 3 * Mp * F // 128, flops=30 * M * F)
    if op == "transpose":
        T, K, E = case["T"], case["K"], case["E"]
        rows = 128 * _blocks(_capacity(T, E, case["k"]) if E else T)
        size = T * K + T * K // 32 if case["src"] == "codes" else 2 * T * K
        return dict(bytes=size + rows * K + rows * K // 128 + 4 * rows * bool(E), flops=2 * rows * K)
    N, K = case["N"], case["K"]
    out = (2 if case["dtype"] == "bf16" else 4) * N * K * (1 + bool(case["accumulate"]))
    if op == "wgrad":
        M = case["M"]
        return dict(bytes=M * (N + K) + M * (N + K) // 128 + out, flops=2 * M * N * K)
    used = case["T"] * case["k"]
    return dict(bytes=used * (N + K) + used * (N + K) // 128 + case["E"] * out, flops=2 * used * N * K)
