"""A training step of FP8 blocks from the norm to the weights' gradients: the mixture-of-experts block of
examples/moe_block_fp8.py and a dense one, against float64 autograd through the same (dequantized) weights; the norm's
gradient against differences; micro-batches added up; and both steps captured in HIP graphs.

E4M3's error is at most 2^-4 of a value and, over a binade's mantissas, 2.6% rms (half a step over sqrt(3), times 0.72); the
errors of different values are independent, so a product's relative error in the 2-norm is the root of its operands' squares.
    up product: 2.6% (tokens).  SwiGLU multiplies two such values and its gate's slope is at most 1.1: 4% of h, and 2.6% more
    when h is quantized: 4.8% of the experts' part.  With SwiGLU's inputs kept in 8 bits (2.6% more on each): h 5.6%, its
    copy 6.2%; the slopes silu' vary with the gate as much as silu does: dgate and dup 6%, from gradients at 2.6% -> 6.6%.
    dW of down: 6.2% and 2.6% -> 6.7%.  dW of up: 6.6%, its copy's 2.6%, tokens' 2.6% -> 7.6%.  Gradient of the norm's
    output: 6.6% and 2.6% -> 7.1%; the norm's gradients are linear in it.
The bounds are 1.5 times these, for values in E4M3's subnormal range and small samples.  The gate's gradient is a Jacobian
times dots grad_y . c2, whose errors are sums over H of independent terms: 4.8% of |grad_y| |c2| / sqrt(H) each, whatever is
left of the dots' differences.  Its bound is 1.5 times that, and 3 times more for a single token's two or so dots."""
import importlib.util
import os

import pytest
import torch

import fine_grained_quantization_amd as fq
from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("moe_block_fp8", os.path.join(ROOT, "examples", "moe_block_fp8.py"))
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def randn(g, *shape, scale=1.0):
    return (scale * torch.randn(shape, device="cuda", generator=g)).bfloat16()


def build(T, H, F, E, k, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    up, down = randn(g, E, 2 * F, H, scale=H ** -0.5), randn(g, E, H, F, scale=F ** -0.5)
    norm = 1 + 0.1 * torch.randn(H, device="cuda", generator=g)
    block = example.Fp8MoEBlock(norm, up, down, k, scale=2.5)
    return block, randn(g, T, H), randn(g, T, H), torch.randn((T, E), device="cuda", generator=g), randn(g, T, H)


def off_by(got, want):
    got, want = got.detach().double(), want.detach()
    return float((got - want).norm() / want.norm())


@pytest.mark.parametrize("T,H,F,E,k", [(1, 256, 128, 4, 2), (60, 512, 256, 16, 4), (900, 1024, 640, 8, 3)])
def test_moe_block_against_float64(T, H, F, E, k):
    block, x, residual, logits, gy = build(T, H, F, E, k)
    say(f"fp8 block T={T} H={H} F={F} E={E}")
    y, saved = block.forward(x, residual, logits)
    gx, gl, gn, dup, ddown = block.backward(gy, saved)
    h = (x.float() + residual.float()).bfloat16().double()
    assert torch.equal(saved[2].double(), h)
    leaves = [t.double().requires_grad_() for t in (h, logits, block.norm, example.dequantized(*block.up),
                                                    example.dequantized(*block.down))]
    want = example.reference(leaves[0], 0.0, *leaves[1:], saved[5], 2.5)
    want.backward(gy.double())
    assert off_by(y.double() - h, want.detach() - h) < 1.5 * 0.048 + 2.0 ** -7  # (y is bf16: 2^-8 of h + experts' part)
    assert off_by(gx.double() - gy.double(), leaves[0].grad - gy.double()) < 1.5 * 0.071 + 2.0 ** -7
    idx, row_of = saved[5].long(), saved[8].long()
    z = logits.double().gather(1, idx)
    v = torch.sigmoid(z)
    w = v / v.sum(1, keepdim=True)
    jac = 2.5 * (torch.diag_embed(w) - w[:, :, None] * w[:, None, :]) * (1 - v)[:, None, :]  # d weight_i / d logit_j
    noise = 0.048 * gy.double().norm(dim=1)[:, None] * saved[11].double()[row_of].norm(dim=2) / H ** 0.5
    assert float((gl.double() - leaves[1].grad).norm()) < (1.5 + 3 / T ** 0.5) * float((noise[:, :, None] * jac).norm())
    assert off_by(gn, leaves[2].grad) < 1.5 * 0.071
    assert off_by(dup, leaves[3].grad) < 1.5 * 0.076
    assert off_by(ddown, leaves[4].grad) < 1.5 * 0.067
    load = saved[5].long().flatten().bincount(minlength=E)
    assert int((load == 0).sum()) == 0 or float(dup[load == 0].abs().max()) == 0.0


def test_micro_batches_add_up():
    """Gradients added to those of an earlier micro-batch: the sum of both alone, rounded once."""
    block, x, residual, logits, gy = build(300, 512, 256, 8, 2, 1)
    parts = [(x, residual, logits, gy), (residual[:130], x[:130], logits[:130].flip(0), gy[:130])]
    alone = []
    for a, r, z, g in parts:
        _, saved = block.forward(a, r, z)
        alone.append(block.backward(g, saved)[3:])
    kept = [block.forward(a, r, z)[1] for a, r, z, _ in parts]
    sums = block.backward(parts[0][3], kept[0])[3:]
    both = block.backward(parts[1][3], kept[1], sums)[3:]
    for a, b, c, s in zip(*alone, both, sums):
        assert c is s and torch.equal(c, a + b)


def dense(M, K, F, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    norm = 1 + 0.1 * torch.randn(K, device="cuda", generator=g)
    up, down = randn(g, 2 * F, K, scale=K ** -0.5), randn(g, K, F, scale=F ** -0.5)
    up, up_t = example.quantize_weights(up[None])
    down, down_t = example.quantize_weights(down[None])
    return randn(g, M, K), randn(g, M, K), norm, [(q[0], s[0]) for q, s in (up, up_t, down, down_t)]


def dense_step(x, gy, norm, weights, dups, ddowns):
    """Norm, up product, SwiGLU, down product and all gradients, the weights' added to `dups` and `ddowns`."""
    up, up_t, down, down_t = weights
    q, s, h, rstd = fq.fp8q_rmsnorm_quant_act_1x128(x, norm, pow2=True)
    c1 = fq.fp8q_gemm_blockscaled(q, s, *up)
    kept = fq.fp8q_quant_act_1x128(c1)
    y = fq.fp8q_gemm_blockscaled(*fq.fp8q_swiglu_quant_act_1x128(c1), *down)
    gh = fq.fp8q_gemm_blockscaled(*fq.fp8q_quant_act_1x128(gy), *down_t)
    g1, s1, g1t, e1t, ht, eht = fq.fp8q_swiglu_backward_quant(*kept, gh)
    fq.fp8q_gemm_wgrad(*fq.fp8q_quant_act_128x1(gy), ht, eht, accumulate=True, dw=ddowns)
    fq.fp8q_gemm_wgrad(g1t, e1t, *fq.fp8q_transpose_act_128x1(q, s), accumulate=True, dw=dups)
    gx, gn = fq.fp8q_rmsnorm_backward(fq.fp8q_gemm_blockscaled(g1, s1, *up_t), h, norm, rstd, gres=gy)
    return y, gx, gn


@pytest.mark.parametrize("M,K,F", [(1, 256, 128), (200, 512, 384), (1000, 1024, 2048)])
def test_dense_block_against_float64(M, K, F):
    x, gy, norm, weights = dense(M, K, F)
    up, down = (example.dequantized(q[None], s[None])[0] for q, s in (weights[0], weights[2]))
    say(f"fp8 dense block M={M} K={K} F={F}")
    dup, ddown = torch.zeros((2 * F, K), device="cuda"), torch.zeros((K, F), device="cuda")
    y, gx, gn = dense_step(x, gy, norm, weights, dup, ddown)
    h, n, u, d = leaves = [t.double().requires_grad_() for t in (x, norm, up, down)]
    a, b = ((h * (h.pow(2).mean(1, keepdim=True) + 1e-6).rsqrt() * n) @ u.t()).chunk(2, 1)
    part = (torch.nn.functional.silu(a) * b) @ d.t()
    (h + part).backward(gy.double())
    assert off_by(y, part.detach()) < 1.5 * 0.048
    assert off_by(gx.double() - gy.double(), leaves[0].grad - gy.double()) < 1.5 * 0.071 + 2.0 ** -7
    assert off_by(gn, leaves[1].grad) < 1.5 * 0.071
    assert off_by(dup, leaves[2].grad) < 1.5 * 0.076
    assert off_by(ddown, leaves[3].grad) < 1.5 * 0.067


def captured(step):
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        step()
    torch.cuda.current_stream().wait_stream(warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    torch.cuda.synchronize()
    return graph, out


@pytest.mark.parametrize("M,K,F", [(100, 512, 256), (4096, 256, 128)])
def test_dense_step_in_a_graph(M, K, F):
    """Forward, backward and the accumulation of the weights' gradients (at 4096 tokens with the tokens split over
    workgroups) in one graph; its replays against eager steps on the same new inputs."""
    x, gy, norm, weights = dense(M, K, F, 2)
    g = torch.Generator(device="cuda").manual_seed(3)
    dup, ddown = torch.zeros((2 * F, K), device="cuda"), torch.zeros((K, F), device="cuda")
    graph, out = captured(lambda: dense_step(x, gy, norm, weights, dup, ddown))
    for r in range(4):
        x.copy_(randn(g, M, K))
        gy.copy_(randn(g, M, K))
        start = [torch.randn(t.shape, device="cuda", generator=g) for t in (dup, ddown)]
        dup.copy_(start[0])
        ddown.copy_(start[1])
        for t in out:
            t.view(torch.uint8).fill_(0xA5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*out, dup, ddown)]
        want = [*dense_step(x, gy, norm, weights, *start), *start]
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want)), r
        say(f"fp8 dense step M={M}: replay {r} matches the eager step")


@pytest.mark.parametrize("T", [20, 300])
def test_moe_step_in_a_graph(T):
    block, x, residual, logits, gy = build(T, 512, 256, 8, 2, 4)
    g = torch.Generator(device="cuda").manual_seed(5)
    grads = torch.zeros((8, 512, 512), device="cuda"), torch.zeros((8, 512, 256), device="cuda")

    def step(grads):
        y, saved = block.forward(x, residual, logits)
        return (y, *block.backward(gy, saved, grads)[:3])

    graph, out = captured(lambda: step(grads))
    for r in range(4):
        for t in (x, residual, gy):
            t.copy_(randn(g, T, 512))
        logits.copy_(torch.randn(logits.shape, device="cuda", generator=g))
        start = [torch.randn(t.shape, device="cuda", generator=g) for t in grads]
        for t, s in zip(grads, start):
            t.copy_(s)
        for t in out:
            t.view(torch.uint8).fill_(0xA5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*out, *grads)]
        want = [*step(start), *start]
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want)), r
        say(f"fp8 block T={T}: replay {r} matches the eager step")


def test_example_runs(monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["moe_block_fp8.py", "--tokens", "130", "--hidden", "256", "--width", "128", "--experts", "4"])
    example.main()
    assert "forward and backward" in capsys.readouterr().out
