"""The gating, INT8 expert products and combination as one layer (examples/moe_layer_int8.py): against float64, its
router gradient against differences, on a stream of its own, and captured in a HIP graph.

INT8 with one scale per row: a token's codes are off by at most half a step, amax / 254, on values of rms about amax /
4 for normal rows, so the quantization noise of one operand is about 4 / 254 / sqrt(3) = 0.9% of it; three such
operands (tokens, weights, SwiGLU rows; the weights twice) and the bf16 roundings stay under 4% of the experts' part."""
import importlib.util
import os

import pytest
import torch

import fine_grained_quantization_amd as fq
from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("moe_layer_int8", os.path.join(ROOT, "examples", "moe_layer_int8.py"))
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def build(T, H, F, E, k, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, scale=1.0):
        return (scale * torch.randn(shape, device="cuda", generator=g)).bfloat16()

    up, down = randn(E, 2 * F, H, scale=H ** -0.5), randn(E, H, F, scale=F ** -0.5)
    bias = 0.05 * torch.randn(E, device="cuda", generator=g)
    layer = example.Int8MoE(up, down, k, bias=bias, n_group=4, topk_group=2, scale=2.5)
    return layer, up, down, randn(T, H), torch.randn((T, E), device="cuda", generator=g), randn(T, H)


@pytest.mark.parametrize("T,H,F,E,k", [(1, 256, 128, 8, 2), (50, 512, 272, 16, 4), (700, 1024, 512, 32, 4)])
def test_layer_against_float64(T, H, F, E, k):
    layer, up, down, x, logits, shared = build(T, H, F, E, k)
    say(f"int8 layer T={T} H={H} F={F} E={E}")
    y, saved = layer.forward(x, logits, shared)
    want = example.reference(x, logits, up, down, saved[1], shared, 2.5)
    part = want - shared.double()
    err = (y.double() - want).norm() / part.norm()
    assert float(err) < 0.04
    y2, _ = layer.forward(x, logits, None)
    err2 = (y2.double() - part).norm() / part.norm()
    assert float(err2) < 0.04
    assert int(saved[-1].sum()) == T * k


def test_router_gradient_against_differences():
    """The loss is linear in the gate's weights, so with the expert rows held fixed its difference along a logit is that
    of 64-bit weights: central differences with h = 1e-5 leave h^2 terms below 1e-8 of the magnitudes; fp32 sums of H =
    512 products and the weights' gradient leave 2^-24 * 64 of them."""
    layer, up, down, x, logits, shared = build(40, 512, 272, 16, 4, 3)
    y, saved = layer.forward(x, logits, shared)
    r = torch.randn(y.shape, device="cuda").bfloat16()
    _, gl = layer.backward(r, saved)
    idx, row_of = saved[1].long(), saved[4].long()
    dots = (layer.c2[row_of].double() * r[:, None, :].double())          # [T, k, H]
    mag = dots.abs().sum(2).sum(1, keepdim=True) * 2.5
    dots = dots.sum(2)

    def loss(z):
        v = torch.sigmoid(z).gather(1, idx)
        return (2.5 * v / (v.sum(1, keepdim=True) + 1e-20) * dots).sum(1)

    z = logits.double()
    for e in range(16):
        step = torch.zeros_like(z)
        step[:, e] = 1e-5
        diff = (loss(z + step) - loss(z - step)) / 2e-5
        assert bool(((diff - gl[:, e].double()).abs() <= (1e-8 + 64 * 2.0 ** -24) * mag[:, 0]).all())


def test_gradients_after_several_forward_calls():
    """Each backward is that of the forward call whose values it is given, as in gradient accumulation: the same bits as
    a backward right behind its forward call, also where a call with fewer tokens came between."""
    layer, _, _, x, logits, shared = build(200, 512, 272, 16, 4, 6)
    g = torch.Generator(device="cuda").manual_seed(7)
    parts = [(x, logits, shared), (torch.randn(x.shape, device="cuda", generator=g).bfloat16(), logits.flip(0), shared),
             (x[:40], logits[:40], None)]
    grads = [torch.randn(p[0].shape, device="cuda", generator=g).bfloat16() for p in parts]
    say("int8 layer: three forward calls, then their gradients")
    want = []
    for p, r in zip(parts, grads):
        y, saved = layer.forward(*p)
        gc, gl = layer.backward(r, saved)
        want.append((y.clone(), gc[:int(saved[3][-1])].clone(), gl.clone()))
    calls = [layer.forward(*p) for p in parts]
    for (y, saved), r, (wy, wc, wl) in zip(calls, grads, want):
        gc, gl = layer.backward(r, saved)
        assert torch.equal(gl, wl)
        assert torch.equal(gc[:int(saved[3][-1])].view(torch.int16), wc.view(torch.int16))
        assert torch.equal(y.view(torch.int16), wy.view(torch.int16))


def test_layer_on_another_stream():
    layer, _, _, x, logits, shared = build(300, 512, 272, 16, 4, 4)
    want, _ = layer.forward(x, logits, shared)
    torch.cuda.synchronize()
    late = torch.zeros_like(x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(200):
            late.copy_(x)
            late.zero_()
        late.copy_(x)
        got, _ = layer.forward(late, logits, shared)
    side.synchronize()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("T", [20, 300])
def test_graph_replays(T):
    """Gate, quantization, both products, combination and the gradients as one captured graph; every replay against the
    same calls made eagerly on new inputs, with the outputs overwritten in between."""
    layer, _, _, x, logits, shared = build(T, 512, 272, 16, 4, 5)
    E, k, H = 16, 4, 512
    rows = fq.fp8q_moe_route_capacity(T, E, k)
    i32 = dict(dtype=torch.int32, device="cuda")
    out = (torch.empty((T, k), **i32), torch.empty((T, k), device="cuda"), torch.empty(E + 1, **i32),
           torch.empty((T, k), **i32), torch.empty(rows, **i32), torch.empty(E, **i32))
    ws = torch.empty(max(4, fq.load_library().fp8q_moe_gate_workspace_bytes(T, E)), dtype=torch.uint8, device="cuda")
    q, s = torch.empty((T, H), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    qh, sh = torch.empty((rows, layer.F), dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    c1 = torch.zeros((rows, 2 * layer.F), dtype=torch.bfloat16, device="cuda")
    c2 = torch.zeros((rows, H), dtype=torch.bfloat16, device="cuda")
    h = torch.empty((rows, layer.F), dtype=torch.bfloat16, device="cuda")
    y, gc = torch.empty_like(x), torch.zeros_like(c2)
    gw, gl = torch.empty((T, k), device="cuda"), torch.empty_like(logits)

    def step():
        idx, w, off, row_of, row_token, _ = fq.fp8q_moe_gate_topk(logits, k, workspace=ws, out=out, **layer.gate)
        fq.fp8q_quant_int8(x, q=q, s=s)
        fq.fp8q_grouped_gemm_int8_gather(q, s, row_token, *layer.up, off, c=c1)
        fq.fp8q_swiglu_bf16(c1[:, :layer.F], c1[:, layer.F:], h=h)
        fq.fp8q_quant_int8(h, q=qh, s=sh)
        fq.fp8q_grouped_gemm_int8(qh, sh, *layer.down, off, c=c2)
        fq.fp8q_moe_combine(c2, row_of, w, add=shared, y=y)
        fq.fp8q_moe_combine_backward(shared, c2, row_of, w, row_token, off, grad_c=gc, grad_weight=gw)
        fq.fp8q_moe_gate_backward(logits, idx, gw, score="sigmoid", scale=2.5, grad_logits=gl)

    outputs = list(out) + [y, gw, gl]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for r in range(4):
        g = torch.Generator(device="cuda").manual_seed(100 + r)
        x.copy_(torch.randn(x.shape, device="cuda", generator=g))
        logits.copy_(torch.randn(logits.shape, device="cuda", generator=g))
        say(f"int8 layer graph T={T} replay {r}")
        for t in outputs:
            t.view(torch.uint8).fill_(0xA5)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outputs]
        for t in outputs:
            t.view(torch.uint8).fill_(0x5A)
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, outputs):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
