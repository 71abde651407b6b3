"""Backward copies (transposes in groups of 128 tokens, power-of-two scales) and SwiGLU's gradient from 8-bit inputs.

The copies are exact but for E4M3's rounding: codes and scale bytes are compared bit for bit.  SwiGLU's values are fp32: p =
1 / (1 + e^-x) is within 8 u (1 + |x|), u = 2^-24 (the exponent's argument is off by u |x log2 e|, its exp2, the addition and
the reciprocal by an ulp or so each), the products add a rounding each; E4M3 then rounds by at most 2^-4 of a value, or half
of its smallest step, 2^-10, times the scale."""
import pytest
import torch

import fine_grained_quantization_amd as fq
from backward_reference import backward_copy, copy_values, decode, e4m3, power, rows_of, swiglu_grad64
from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def checkpoint(M, K, seed=0, pow2=False):
    g = torch.Generator(device="cuda").manual_seed(seed + M * 3 + K)
    q = e4m3(130 * torch.randn((M, K), device="cuda", generator=g))
    s = 0.002 * torch.exp(torch.randn((K // 128, M), device="cuda", generator=g))
    return q, torch.exp2(torch.round(torch.log2(s))) if pow2 else s


def same(got, want):
    assert torch.equal(got[1], want[1])
    assert torch.equal(got[0], want[0])


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("M,K", [(1, 128), (127, 256), (128, 384), (129, 1152), (1000, 2048), (515, 7168)])
def test_copy_of_a_checkpoint(M, K, pow2):
    q, s = checkpoint(M, K, pow2=pow2)
    say(f"copy of a checkpoint M={M} K={K} pow2={pow2}")
    got = fq.fp8q_transpose_act_128x1(q, s)
    same(got, backward_copy(decode(q, s)))
    if pow2:  # the values survive, but for those that fall below E4M3's normal range in their new group
        v, w = decode(q, s).double().t(), copy_values(*got)[:, :M]
        floor = 2.0 ** -6 * power(got[1]).t().repeat_interleave(128, 1)[:, :M]
        assert bool(((v == w) | (v.abs() < floor)).all())


@pytest.mark.parametrize("M,K", [(1, 128), (130, 256), (1001, 1408), (77, 7168)])
def test_copy_of_bf16_rows(M, K):
    g = torch.Generator(device="cuda").manual_seed(M)
    wide = (torch.randn((M, 2 * K), device="cuda", generator=g) * torch.exp(2 * torch.randn((M, 1), device="cuda", generator=g))).bfloat16()
    say(f"copy of bf16 rows M={M} K={K}")
    x = wide[:, K:]
    want = backward_copy(x.float())
    same(fq.fp8q_quant_act_128x1(x), want)
    same(fq.fp8q_quant_act_128x1(x.contiguous()), want)


def test_scale_bytes_at_their_borders():
    """Groups whose maximum is every bf16 value: 448 2^e itself, its neighbours, subnormals, the largest, and 0."""
    bits = torch.arange(0, 0x7F80, dtype=torch.int32)
    x = torch.zeros((128, (bits.numel() + 127) // 128 * 128), dtype=torch.int16)
    x[17, :bits.numel()] = bits.to(torch.int16)
    x[90, :bits.numel()] = (bits // 2 * 1).to(torch.int16) | -32768  # a smaller, negative one beside it
    x = x.cuda().view(torch.bfloat16)
    same(fq.fp8q_quant_act_128x1(x), backward_copy(x.float()))


def test_checkpoint_values_beyond_bf16():
    """Scales that make 24-bit values: the copy rounds code * scale to fp32 once, then to E4M3."""
    q, s = checkpoint(256, 256, 9)
    s = s * (1 + torch.rand_like(s) * 2.0 ** -20)
    same(fq.fp8q_transpose_act_128x1(q, s), backward_copy(decode(q, s)))
    s[0, :128] = 0
    s[1, 5] = 3e38 / 448
    s[1, 9] = 1e-40
    same(fq.fp8q_transpose_act_128x1(q, s), backward_copy(decode(q, s)))


@pytest.mark.parametrize("T,E,k,K", [(1, 8, 2, 256), (100, 16, 4, 384), (700, 5, 3, 1024)])
def test_copy_of_routed_rows(T, E, k, K):
    g = torch.Generator(device="cuda").manual_seed(T)
    _, _, off, _, row_token, _ = fq.fp8q_moe_gate_topk(torch.randn((T, E), device="cuda", generator=g), k)
    q, s = checkpoint(T, K)
    say(f"copy of routed rows T={T} E={E} k={k} K={K}")
    same(fq.fp8q_transpose_act_128x1(q, s, row_token=row_token), backward_copy(rows_of(decode(q, s), row_token, T)))
    x = torch.randn((T, K), device="cuda", generator=g).bfloat16()
    same(fq.fp8q_quant_act_128x1(x, row_token=row_token), backward_copy(rows_of(x.float(), row_token, T)))


def test_rows_of_any_tokens():
    """Tokens in any order and more than once, outside the tokens, the least and the largest int32, an odd row count."""
    q, s = checkpoint(50, 256, 2)
    t = torch.tensor([3, 3, 49, 0, -1, 50, -2147483648, 2147483647, 7] + list(range(50)) * 3, dtype=torch.int32, device="cuda")
    same(fq.fp8q_transpose_act_128x1(q, s, row_token=t), backward_copy(rows_of(decode(q, s), t, 50)))
    none = fq.fp8q_transpose_act_128x1(q[:0], s[:, :0].contiguous(), row_token=t)
    assert int(none[0].max()) == 0 and int(none[1].max()) == 0 and none[0].shape == (256, 256)
    empty = fq.fp8q_transpose_act_128x1(q, s, row_token=t[:0])
    assert empty[0].shape == (256, 0) and empty[1].shape == (0, 256)


def test_given_outputs_are_filled():
    q, s = checkpoint(200, 256, 4)
    qt = torch.full((256, 256), 0x55, dtype=torch.uint8, device="cuda")
    et = torch.full((2, 256), 0x55, dtype=torch.uint8, device="cuda")
    got = fq.fp8q_transpose_act_128x1(q, s, qt=qt, et=et)
    assert got[0] is qt and got[1] is et
    same(got, backward_copy(decode(q, s)))


# ------------------------------------------------------------------------------------------------------
# SwiGLU
# ------------------------------------------------------------------------------------------------------

def check_rows(q, s, want, tol):
    """1x128 groups of values within `tol` of `want`."""
    M, K = want.shape
    amax = want.abs().view(M, -1, 128).amax(2)
    slack = tol.view(M, -1, 128).amax(2)
    sc = s.t().double()
    assert bool(((sc * 448 - amax).abs() <= slack + 4 * U * amax).all())
    got = q.view(torch.float8_e4m3fn).double() * sc.repeat_interleave(128, 1)
    step = 2.0 ** -10 * sc.repeat_interleave(128, 1)
    assert bool(((got - want).abs() <= (2.0 ** -4 + 8 * U) * want.abs() + step + 1.1 * tol).all())


def check_copy(qt, et, want, tol):
    """The backward copy of values within `tol` of `want` [M, C]."""
    M, C = want.shape
    pad = -M % 128
    want, tol = (torch.nn.functional.pad(t, (0, 0, 0, pad)) for t in (want, tol))
    amax, slack = (t.abs().view(-1, 128, C).amax(1) for t in (want, tol))
    p = power(et)
    assert bool((amax - slack <= 448 * p).all()) and bool(((amax + slack > 224 * p) | (et == 0)).all())
    got = copy_values(qt, et).t()
    step = 2.0 ** -10 * p.repeat_interleave(128, 0)
    assert bool(((got - want).abs() <= 2.0 ** -4 * want.abs() + step + 1.1 * tol).all())
    assert bool((got[M:] == 0).all())


def check_swiglu(out, q, s, gh):
    gq, gs, gqt, get, hqt, het = out
    v = decode(q, s)
    x, u = v.chunk(2, 1)
    dx, du, h = swiglu_grad64(x, u, gh)
    xa = x.double().abs()
    rel = (16 + 8 * xa) * U
    tx = gh.double().abs() * u.double().abs() * rel * (1 + xa) + 1e-36
    tu = gh.double().abs() * xa * rel + 1e-36
    th = u.double().abs() * xa * rel + 1e-36
    d, t = torch.cat([dx, du], 1), torch.cat([tx, tu], 1)
    check_rows(gq, gs, d, t)
    check_copy(gqt, get, d, t)
    check_copy(hqt, het, h, th)
    # the two copies of one value agree to both roundings
    both = gq.view(torch.float8_e4m3fn).double() * gs.t().double().repeat_interleave(128, 1)
    cols = copy_values(gqt, get).t()[:both.shape[0]]
    assert float((both - cols).norm() / d.norm().clamp(min=1e-300)) < 2 * 2.0 ** -4


@pytest.mark.parametrize("M,F", [(1, 128), (127, 256), (128, 128), (200, 1152), (1030, 2048), (900, 5120), (4200, 1152)])
def test_swiglu_gradient(M, F):
    q, s = checkpoint(M, 2 * F, 3)
    g = torch.Generator(device="cuda").manual_seed(M)
    gh = (1e-3 * torch.randn((M, F), device="cuda", generator=g)).bfloat16()
    say(f"swiglu gradient M={M} F={F}")
    out = fq.fp8q_swiglu_backward_quant(q, s, gh)
    assert [tuple(t.shape) for t in out[2:]] == [(2 * F, (M + 127) // 128 * 128), ((M + 127) // 128, 2 * F),
                                                 (F, (M + 127) // 128 * 128), ((M + 127) // 128, F)]
    check_swiglu(out, q, s, gh)
    wide = torch.zeros((M, 3 * F), device="cuda").bfloat16()
    wide[:, F:2 * F] = gh
    again = fq.fp8q_swiglu_backward_quant(q, s, wide[:, F:2 * F], out=tuple(torch.full_like(t, 3) for t in out))
    assert all(torch.equal(a, b) for a, b in zip(out, again))


def test_swiglu_gradient_of_large_and_small_gates():
    """Gates where e^-x overflows or vanishes, zeros, and gradients of zero (groups of zeros)."""
    M, F = 256, 256
    q, s = checkpoint(M, 2 * F, 5)
    s[0] *= 400  # gates to several hundreds
    s[1] *= 1e-12
    s[2, :40] = 0
    gh = torch.randn((M, F), device="cuda").bfloat16()
    gh[100:130] = 0
    gh[:, 7] = 0
    say("swiglu gradient, large and small gates")
    check_swiglu(fq.fp8q_swiglu_backward_quant(q, s, gh), q, s, gh)


def test_swiglu_gradient_of_gates_that_vanish():
    """Gates around and far below -87, where p = 1 / (1 + e^-x) leaves fp32's normal numbers and then all of them, with inputs
    and gradients of 1e10 that keep the results normal: the relative bounds of check_swiglu, and what p and x p lose below
    2^-126 (half a step of 2^-149 each, times |x| and the other factors).  From -110 on p is below 2^-158: zeros."""
    gates = (80.0, 86.0, 87.2, 87.5, 88.0, 92.0, 97.0, 100.0, 103.0, 110.0, 150.0, 1000.0, 3e38)
    M, F = 128 * len(gates), 256
    g = torch.Generator(device="cuda").manual_seed(8)
    q = torch.full((M, 2 * F), 0x38, dtype=torch.uint8, device="cuda")
    q[:, :F] = torch.where(torch.rand((M, F), device="cuda", generator=g) < 0.5, 0xB8, 0xB9).to(torch.uint8)  # -1, -1.125
    s = torch.full((2 * F // 128, M), 1e10, device="cuda")
    s[:F // 128] = torch.tensor(gates, device="cuda").repeat_interleave(128)
    gh = (1e10 * torch.randn((M, F), device="cuda", generator=g)).bfloat16()
    say("swiglu gradient, gates that vanish")
    gq, gs, gqt, get, hqt, het = fq.fp8q_swiglu_backward_quant(q, s, gh)
    x, u = decode(q, s).chunk(2, 1)
    dx, du, h = swiglu_grad64(x, u, gh)
    xa, ga, ua = x.double().abs(), gh.double().abs(), u.double().abs()
    rel, least = 2 * (16 + 8 * xa) * U, 2.0 ** -149 * (2 + xa)
    d = torch.cat([dx, du], 1)
    t = torch.cat([rel * dx.abs() + least * ga * ua, rel * du.abs() + least * ga], 1)
    check_rows(gq, gs, d, t)
    check_copy(gqt, get, d, t)
    check_copy(hqt, het, h, rel * h.abs() + least * ua)
    gone = gates.index(110.0) * 128
    assert float(decode(gq, gs)[gone:].abs().max()) == 0.0 and float(gs[:, gone:].max()) == 0.0
    for code, byte in ((gqt, get), (hqt, het)):
        assert int((code[:, gone:] & 0x7F).max()) == 0 and int(byte[gone // 128:].max()) == 0


@pytest.mark.parametrize("size", [3e-34, 1e35])
def test_swiglu_gradient_of_extreme_gradients(size):
    """Groups whose maximum's reciprocal is beyond fp32's normal numbers, or near it.  Every value is within E4M3's half step,
    2^-4, of its own or, below E4M3's normal range, 2^-10 of the scale; scales here are at least 2^-126 / 2^4, kept to 2^-20."""
    M, F = 130, 128
    q, s = checkpoint(M, 2 * F, 7)
    s = torch.full_like(s, 0.01)
    gh = (size * torch.randn((M, F), device="cuda")).bfloat16()
    gq, gs = fq.fp8q_swiglu_backward_quant(q, s, gh)[:2]
    x, u = decode(q, s).chunk(2, 1)
    dx, du, _ = swiglu_grad64(x, u, gh)
    want = torch.cat([dx, du], 1)
    sc = gs.t().double().repeat_interleave(128, 1)
    got = gq.view(torch.float8_e4m3fn).double() * sc
    assert bool(((got - want).abs() <= (2.0 ** -4 + 2.0 ** -18) * want.abs() + 2.0 ** -10 * sc * (1 + 2.0 ** -18)).all())


def test_swiglu_gradient_against_differences():
    """Central differences (step 1e-5, error 1e-10) of sum(gh * silu(x) u) in float64 against the decoded gradients: within
    E4M3's half step."""
    M, F = 4, 128
    q, s = checkpoint(M, 2 * F, 6)
    gh = torch.randn((M, F), device="cuda").bfloat16()
    gq, gs = fq.fp8q_swiglu_backward_quant(q, s, gh)[:2]
    got = gq.view(torch.float8_e4m3fn).double() * gs.t().double().repeat_interleave(128, 1)
    v = decode(q, s).double()

    def rows(v):
        x, u = v.chunk(2, 1)
        return (gh.double() * torch.nn.functional.silu(x) * u).sum(1)

    for k in range(0, 2 * F, 5):
        step = torch.zeros_like(v)
        step[:, k] = 1e-5
        d = (rows(v + step) - rows(v - step)) / 2e-5
        assert bool(((d - got[:, k]).abs() <= 2.0 ** -4 * d.abs() + 2.0 ** -10 * gs[k // 128].double() + 1e-8).all())


def test_swiglu_no_rows():
    q, s = checkpoint(1, 512)
    out = fq.fp8q_swiglu_backward_quant(q[:0], s[:, :0].contiguous(), torch.empty((0, 256), device="cuda").bfloat16())
    assert [tuple(t.shape) for t in out] == [(0, 512), (4, 0), (512, 0), (0, 512), (256, 0), (0, 256)]
