"""The norm's and the backward pass's kernels past 2^31 elements and 4 GiB, and weight gradients of thousands of experts.

Rows, and blocks of 128 rows, do not depend on the others: the first and last of a large call have the bits of a call on them alone."""
import pytest
import torch

import fine_grained_quantization_amd as fq
from backward_reference import copy_values, e4m3
from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    torch.cuda.empty_cache()


def rows(M, K, seed):
    """bf16 [M, K], made 8192 rows at a time."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    for i in range(0, M, 8192):
        x[i:i + 8192] = torch.randn((min(8192, M - i), K), device="cuda", generator=g).bfloat16()
    return x


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


M, K = 300004, 7168  # 2.15e9 elements, 4.3 GB in bf16; the last block of 128 tokens has 100


def ends():
    return slice(0, 128), slice(M - 100, M), slice(2 ** 31 // K // 128 * 128, 2 ** 31 // K // 128 * 128 + 128)


def test_norm_and_its_gradients():
    x, w = rows(M, K, 1), 1 + 0.1 * torch.randn(K, device="cuda")
    r = x.flip(0)
    say("norm and its gradients, 300004 x 7168")
    q, s, h, rstd = fq.fp8q_rmsnorm_quant_act_1x128(x, w, residual=r)
    gx, gw = fq.fp8q_rmsnorm_backward(x, h, w, rstd, gres=r)
    total = torch.zeros(K, dtype=torch.float64, device="cuda")
    size = torch.zeros(K, dtype=torch.float64, device="cuda")
    for i in range(0, M, 8192):
        part = x[i:i + 8192].double() * h[i:i + 8192].double() * rstd[i:i + 8192, None].double()
        total += part.sum(0)
        size += part.abs().sum(0)
    # sums of M / (2 CUs) rows a part, then of the parts: fewer than 2000 roundings on any path
    assert bool(((gw.double() - total).abs() <= 2000 * 2.0 ** -24 * size).all())
    for at in ends():
        one = fq.fp8q_rmsnorm_quant_act_1x128(x[at], w, residual=r[at])
        assert same(one[0], q[at]) and same(one[1], s[:, at]) and same(one[2], h[at]) and same(one[3], rstd[at])
        assert same(fq.fp8q_rmsnorm_backward(x[at], h[at], w, rstd[at], gres=r[at])[0], gx[at])


def test_copies():
    x = rows(M, K, 2)
    q, s = fq.fp8q_quant_act_1x128(x)
    tok = torch.arange(M - 1, -1, -1, dtype=torch.int32, device="cuda")
    say("backward copies, 300004 x 7168")
    for name, whole, part in (
            ("codes", lambda: fq.fp8q_transpose_act_128x1(q, s),
             lambda at: fq.fp8q_transpose_act_128x1(q[at], s[:, at].contiguous())),
            ("bf16", lambda: fq.fp8q_quant_act_128x1(x), lambda at: fq.fp8q_quant_act_128x1(x[at])),
            ("codes, routed", lambda: fq.fp8q_transpose_act_128x1(q, s, row_token=tok),
             lambda at: fq.fp8q_transpose_act_128x1(q, s, row_token=tok[at])),
            ("bf16, routed", lambda: fq.fp8q_quant_act_128x1(x, row_token=tok),
             lambda at: fq.fp8q_quant_act_128x1(x, row_token=tok[at]))):
        qt, et = whole()
        for at in ends():
            block = at.start // 128
            one = part(at)
            assert same(one[0], qt[:, 128 * block:128 * block + 128]) and same(one[1], et[block:block + 1]), name
        say(f"  {name}: the same as its blocks alone")


def test_swiglu_gradient():
    rows_, F = 140004, 8192  # q, gq and gqt 2.3 GB each
    x = rows(rows_, 2 * F, 3)
    q, s = fq.fp8q_quant_act_1x128(x)
    gh = x[:, :F]
    say("swiglu gradient, 140004 x 8192")
    out = fq.fp8q_swiglu_backward_quant(q, s, gh)
    middle = 2 ** 31 // (2 * F) // 128 * 128
    for at in (slice(0, 128), slice(middle, middle + 128), slice(rows_ // 128 * 128, rows_)):
        one, b = fq.fp8q_swiglu_backward_quant(q[at], s[:, at].contiguous(), gh[at]), at.start // 128
        cols = slice(128 * b, 128 * b + 128)
        for a, w in zip(one, (out[0][at], out[1][:, at], out[2][:, cols], out[3][b:b + 1], out[4][:, cols], out[5][b:b + 1])):
            assert same(a, w)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_thousands_of_experts(dtype):
    """Many more experts than workgroups and lanes, half of them without tokens."""
    E, N, C = 20000, 16, 32
    off = torch.tensor([128 * ((e + 1) // 2 % 300) if e < 600 else 128 * 299 for e in range(E)] + [128 * 300], dtype=torch.int32)
    off = torch.cummax(off, 0)[0].int().cuda()
    cols = 128 * 300
    g = torch.Generator(device="cuda").manual_seed(4)

    def copy(n):
        v = torch.randint(-2, 3, (n, cols), device="cuda", generator=g).float()
        return e4m3(v), torch.randint(126, 129, (cols // 128, n), dtype=torch.uint8, device="cuda", generator=g)
    (gt, eg), (xt, ex) = copy(N), copy(C)
    say(f"weight gradients of {E} experts {dtype}")
    dw = fq.fp8q_grouped_gemm_wgrad(gt, eg, xt, ex, off, out_dtype=dtype, dw=torch.full((E, N, C), 7.0, dtype=dtype, device="cuda"))
    g64, x64, o = copy_values(gt, eg), copy_values(xt, ex), off.tolist()
    some = [e for e in range(E) if o[e] < o[e + 1]]
    assert 250 < len(some) < 600 and some[-1] == E - 1
    for e in some:
        a, b = o[e], o[e + 1]
        assert torch.equal(dw[e].double(), (g64[:, a:b] @ x64[:, a:b].t()).to(dtype).double()), e
    empty = torch.ones(E, dtype=torch.bool, device="cuda")
    empty[some] = False
    assert int((dw[empty] != 0).sum()) == 0
