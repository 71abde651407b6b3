"""The root-mean-square norm with quantized output, and its gradients, against float64.

Rounding bounds, u = 2^-24: a sum of n fp32 terms is off by at most n u of the sum of their magnitudes whatever its order
(fewer roundings than n lie on any path); rstd's sum of squares has no cancellation, a quotient, an addition of eps, a square
root (which halves relative errors) and a quotient follow.  Codes are checked bit for bit: the quotient h w 448 / amax is formed
in double, where float64 gives the same fp32 value."""
import pytest
import torch

import fine_grained_quantization_amd as fq
from backward_reference import e4m3, norm64, power, power_byte
from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def inputs(M, K, w_dtype, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(1000 * seed + M * 7 + K)
    x = (scale * torch.randn((M, K), device="cuda", generator=g)).bfloat16()
    r = torch.randn((M, K), device="cuda", generator=g)
    r[:, ::97] *= 20
    w = (1 + 0.3 * torch.randn(K, device="cuda", generator=g)).to(w_dtype)
    return x, r.bfloat16(), w


def check_norm(q, s, h, rstd, y, want_h, w, eps, pow2):
    M, K = want_h.shape
    assert torch.equal(h.view(torch.int16), want_h.view(torch.int16))
    hd = want_h.double()
    r64 = (hd.pow(2).mean(1) + eps).rsqrt()
    tol_r = (K // 64 + 40) * U
    assert bool(((rstd.double() - r64).abs() <= tol_r * r64).all())
    t = (want_h.float() * w.float()).view(M, K // 128, 128)
    n = (t * rstd.view(M, 1, 1))
    if y is not None:
        assert torch.equal(y.view(torch.int16), n.bfloat16().view(M, K).view(torch.int16))
    got_s = s.t()  # [M, K / 128]
    if pow2:
        amax = n.abs().amax(2)
        sc = torch.where(amax > 0, power(power_byte(amax)), torch.zeros((), dtype=torch.float64, device="cuda"))
        assert torch.equal(got_s.double(), sc)
        want = (n.double() / torch.where(sc > 0, sc, 1.0)[:, :, None]).float()
    else:
        top = t.abs().amax(2).double()
        sc = top * rstd.double()[:, None] / 448
        assert bool(((got_s.double() - sc).abs() <= U * sc + 2.0 ** -149).all())
        want = (t.double() * (448.0 / torch.where(top > 0, top, 1.0))[:, :, None]).float()
    assert torch.equal(q.view(M, K // 128, 128), e4m3(want).view(M, K // 128, 128))


@pytest.mark.parametrize("w_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("M,K", [(1, 128), (1, 7168), (3, 256), (37, 2048), (130, 2176), (300, 7168), (5, 8192), (4, 8320),
                                 (300, 8320), (2, 18432), (3, 24576), (2, 24704)])
def test_norm_with_residual(M, K, pow2, w_dtype):
    x, r, w = inputs(M, K, w_dtype)
    say(f"norm M={M} K={K} pow2={pow2} {w_dtype}")
    y = torch.empty_like(x)
    q, s, h, rstd = fq.fp8q_rmsnorm_quant_act_1x128(x, w, residual=r, eps=1e-6, pow2=pow2, y=y)
    check_norm(q, s, h, rstd, y, (x.float() + r.float()).bfloat16(), w, 1e-6, pow2)


@pytest.mark.parametrize("M,K", [(1, 7168), (65, 1408), (9, 8320)])
def test_norm_without_residual_of_strided_rows(M, K):
    x, _, w = inputs(M, 2 * K, torch.bfloat16, 1)
    v, w = x[:, K:], w[:K].contiguous()
    say(f"norm of strided rows M={M} K={K}")
    q, s, h, rstd = fq.fp8q_rmsnorm_quant_act_1x128(v, w, eps=1e-5)
    assert h is v
    check_norm(q, s, h.contiguous(), rstd, None, v.contiguous(), w, 1e-5, False)
    r = torch.randn((M, 3 * K), device="cuda").bfloat16()[:, K:2 * K]
    q, s, h, rstd = fq.fp8q_rmsnorm_quant_act_1x128(v, w, residual=r, eps=1e-5, pow2=True)
    check_norm(q, s, h, rstd, None, (v.float() + r.float()).bfloat16(), w, 1e-5, True)


@pytest.mark.parametrize("K", [2048, 7168, 24704])
@pytest.mark.parametrize("which", ["x", "residual"])
def test_norm_in_place(which, K):
    x, r, w = inputs(21, K, torch.bfloat16, 2)
    say(f"norm in place of {which}, K={K}")
    want = (x.float() + r.float()).bfloat16()
    q, s, h, rstd = fq.fp8q_rmsnorm_quant_act_1x128(x, w, residual=r, h=x if which == "x" else r)
    assert h is (x if which == "x" else r)
    check_norm(q, s, h, rstd, None, want, w, 1e-6, False)


@pytest.mark.parametrize("M,K,residual", [(3700, 7168, True), (7200, 7296, False), (2100, 24704, False)])
def test_norm_of_inputs_past_the_cache(M, K, residual):
    """Inputs of 104 to 106 MB, which are read with streaming loads; the last rows are wider than the registers."""
    x, r, w = inputs(M, K, torch.bfloat16, 3)
    say(f"norm M={M} K={K} residual={residual}, streaming loads")
    q, s, h, rstd = fq.fp8q_rmsnorm_quant_act_1x128(x, w, residual=r if residual else None)
    check_norm(q, s, h, rstd, None, (x.float() + r.float()).bfloat16() if residual else x, w, 1e-6, False)


def test_norm_of_extreme_rows():
    """Rows of zeros (codes 0 with the product's sign, scale 0), one value in a row, a group of zeros, small and large rows,
    a weight of zeros and negative weights."""
    K = 512
    x = torch.zeros((7, K), device="cuda")
    x[1, 5] = -3.0
    x[2] = torch.randn(K, device="cuda")
    x[2, 128:256] = 0
    x[3] = 1e-18 * torch.randn(K, device="cuda")
    x[4] = 1e15 * torch.randn(K, device="cuda")
    x[5] = -0.0
    x[6] = 2.0 ** -130 * torch.randn(K, device="cuda")
    x = x.bfloat16()
    for w in (torch.randn(K, device="cuda").bfloat16(), torch.zeros(K, device="cuda")):
        for pow2 in (False, True):
            say(f"norm of extreme rows, pow2={pow2} {w.dtype}")
            y = torch.empty_like(x)
            q, s, h, rstd = fq.fp8q_rmsnorm_quant_act_1x128(x, w, eps=1e-6, pow2=pow2, y=y)
            check_norm(q, s, h, rstd, y, x, w, 1e-6, pow2)


def test_norm_codes_of_ties():
    """Weights of one and inputs of few bits: quotients that lie right between two codes, which go to the even one."""
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randint(-29, 29, (64, 1024), device="cuda", generator=g).bfloat16()
    x[:, ::128] = 28  # 448 / 28 = 16: every odd multiple of half a code step is a tie
    w = torch.ones(1024, device="cuda").bfloat16()
    q, s, h, rstd = fq.fp8q_rmsnorm_quant_act_1x128(x, w)
    want = (x.float().view(64, 8, 128) * (448.0 / x.float().view(64, 8, 128).abs().amax(2))[:, :, None])
    assert torch.equal(q, e4m3(want).view(64, 1024))


def test_no_rows():
    x = torch.empty((0, 256), device="cuda").bfloat16()
    w = torch.ones(256, device="cuda").bfloat16()
    q, s, h, rstd = fq.fp8q_rmsnorm_quant_act_1x128(x, w, residual=x.clone())
    assert q.shape == (0, 256) and s.shape == (2, 0) and h.shape == (0, 256) and rstd.shape == (0,)
    gx, gw = fq.fp8q_rmsnorm_backward(x, x, w, rstd, gw=torch.full((256,), 7.0, device="cuda"))
    assert gx.shape == (0, 256) and bool((gw == 0).all())


def check_grad(gx, gw, gy, h, w, rstd, gres):
    M, K = h.shape
    g, hd, wd, r = gy.double(), h.double(), w.double(), rstd.double()[:, None]
    dots = g * hd * wd
    f = r.pow(3) * dots.mean(1, keepdim=True)
    want = r * g * wd - hd * f
    tol = 8 * U * (r * g * wd).abs() + hd.abs() * ((K + 16) * U * r.pow(3) * dots.abs().mean(1, keepdim=True))
    if gres is not None:
        want = want + gres.double()
        tol = tol + 2 * U * gres.double().abs()
    assert bool(((gx.double() - want).abs() <= tol * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs() + 2.0 ** -134).all())
    part = g * hd * r
    assert bool(((gw.double() - part.sum(0)).abs() <= (M + 4) * U * part.abs().sum(0) + 2.0 ** -140).all())


@pytest.mark.parametrize("w_dtype,residual", [(torch.bfloat16, True), (torch.float32, False)])
@pytest.mark.parametrize("M,K", [(1, 128), (1, 7168), (37, 2048), (130, 2176), (128, 384), (129, 256), (700, 4096), (1500, 7168),
                                 (33, 8192), (140, 8320), (5, 18432), (150, 20480), (3, 20480)])
def test_norm_gradient(M, K, w_dtype, residual):
    h, gres, w = inputs(M, K, w_dtype, 3)
    gy = (1e-3 * torch.randn((M, K), device="cuda")).bfloat16()
    say(f"norm gradient M={M} K={K} {w_dtype} residual={residual}")
    rstd = (h.float().pow(2).mean(1) + 1e-6).rsqrt()
    gres = (1e-3 * gres.float()).bfloat16() if residual else None
    ws = torch.full((fq.load_library().fp8q_rmsnorm_backward_workspace_bytes(M, K),), 0xFF, dtype=torch.uint8, device="cuda")
    gx, gw = fq.fp8q_rmsnorm_backward(gy, h, w, rstd, gres=gres, workspace=ws)
    check_grad(gx, gw, gy, h, w, rstd, gres)
    again = fq.fp8q_rmsnorm_backward(gy, h, w, rstd, gres=gres)
    assert torch.equal(again[0].view(torch.int16), gx.view(torch.int16)) and torch.equal(again[1], gw)


@pytest.mark.parametrize("M,K", [(5, 256), (200, 384), (5, 8320)])
@pytest.mark.parametrize("eps", [1e-37, 1e-40, 1e-44])
def test_norm_gradient_of_small_rows_and_a_tiny_eps(M, K, eps):
    """Rows of zeros and of 1e-20 (squares 1e-40): 1 / sqrt(eps) up to 1e22, whose square is no fp32 number.  The bounds are
    check_grad's; squares of subnormal size do not enter the gradients, which take the returned rstd."""
    g = torch.Generator(device="cuda").manual_seed(M + K)
    h = (1e-20 * torch.randn((M, K), device="cuda", generator=g)).bfloat16()
    h[1] = 0
    w = (1 + 0.1 * torch.randn(K, device="cuda", generator=g)).bfloat16()
    gy = (1e-12 * torch.randn((M, K), device="cuda", generator=g)).bfloat16()
    say(f"norm gradient of small rows M={M} K={K} eps={eps}")
    rstd = fq.fp8q_rmsnorm_quant_act_1x128(h, w, eps=eps)[3]
    assert bool(torch.isfinite(rstd).all()) and float(rstd.max()) > (2.0 ** 64 if eps < 1e-39 else 1e18)
    gx, gw = fq.fp8q_rmsnorm_backward(gy, h, w, rstd)
    check_grad(gx, gw, gy, h, w, rstd, None)


def test_norm_gradient_strided_and_in_place():
    h, gres, w = inputs(50, 4096, torch.bfloat16, 4)
    gy = (1e-3 * torch.randn((50, 4096), device="cuda")).bfloat16()
    hv, gv, wv = h[:, :2048], gy[:, 2048:], w[:2048].contiguous()
    rstd = (hv.float().pow(2).mean(1) + 1e-6).rsqrt()
    res = (1e-3 * gres[:, :2048].float()).bfloat16()
    want = fq.fp8q_rmsnorm_backward(gv.contiguous(), hv.contiguous(), wv, rstd, gres=res)
    check_grad(*want, gv, hv, wv, rstd, res)
    got = fq.fp8q_rmsnorm_backward(gv, hv, wv, rstd, gres=res)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    mine = res.clone()
    got = fq.fp8q_rmsnorm_backward(gv, hv, wv, rstd, gres=mine, gx=mine)
    assert got[0] is mine and torch.equal(mine, want[0]) and torch.equal(got[1], want[1])
    own = gv.contiguous(), hv.contiguous()
    for gx in own:  # workgroups read them that do not write them
        with pytest.raises(RuntimeError, match="OPTION"):
            fq.fp8q_rmsnorm_backward(*own, wv, rstd, gres=res, gx=gx)


def test_norm_gradient_against_differences():
    """The loss sum(y * gy) in float64 along each of 8 inputs of every row and 8 weights: central differences with step 1e-5
    leave 1e-10 (relative); what remains is bf16's half step of gx and the fp32 bounds of check_grad."""
    M, K = 6, 256
    h, _, w = inputs(M, K, torch.float32, 6)
    gy = torch.randn((M, K), device="cuda").bfloat16()
    rstd = (h.float().pow(2).mean(1) + 1e-3).rsqrt()
    gx, gw = fq.fp8q_rmsnorm_backward(gy, h, w, rstd)
    hd, wd, g = h.double(), w.double(), gy.double()

    def loss(a, b):
        return (norm64(a, b, 1e-3) * g).sum()

    for i in range(8):
        k = 31 * i + 3
        for m in range(M):
            step = torch.zeros_like(hd)
            step[m, k] = 1e-5
            d = (loss(hd + step, wd) - loss(hd - step, wd)) / 2e-5
            assert abs(float(d - gx[m, k].double())) <= 2.0 ** -8 * abs(float(d)) + 1e-4
        step = torch.zeros_like(wd)
        step[k] = 1e-5
        d = (loss(hd, wd + step) - loss(hd, wd - step)) / 2e-5
        assert abs(float(d - gw[k].double())) <= 1e-4


def test_more_rows_than_workgroups_of_the_gradient():
    h, _, w = inputs(9000, 256, torch.bfloat16, 7)
    gy = torch.randn(h.shape, device="cuda").bfloat16()
    rstd = (h.float().pow(2).mean(1) + 1e-6).rsqrt()
    say("norm gradient of 9000 rows")
    check_grad(*fq.fp8q_rmsnorm_backward(gy, h, w, rstd), gy, h, w, rstd, None)
