"""A mixture-of-experts layer with INT8 experts, forward, and the router's gradient.

    python examples/moe_layer_int8.py [--tokens 512] [--hidden 1024] [--width 512] [--experts 32] [--topk 4]

Gating with sigmoid scores, a balance bias and expert groups chooses each token's experts and lays the tokens out by
expert; the tokens are quantized once and read in place by the up projection of their experts; SwiGLU, a second
quantization and the down projection follow on the expert rows; the combination weights the rows and adds them to the
shared expert's output.  Weights are quantized once, per output channel.  The gradient of a loss on the layer's output
reaches the router's logits through the combination and the gate.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fine_grained_quantization_amd as fq  # noqa: E402


class Int8MoE:
    """Experts [E] of hidden size H and width F: up [E, 2F, H] (gate rows, then up rows), down [E, H, F], in bf16."""

    def __init__(self, up, down, topk, bias=None, n_group=1, topk_group=1, scale=1.0):
        self.E, F2, self.H = up.shape
        self.F, self.topk = F2 // 2, topk
        self.gate = dict(score="sigmoid", bias=bias, n_group=n_group, topk_group=topk_group, scale=scale)
        qu, su = fq.fp8q_quant_int8(up.view(-1, self.H))
        qd, sd = fq.fp8q_quant_int8(down.view(-1, self.F))
        self.up = qu.view_as(up), su.view(self.E, F2)
        self.down = qd.view_as(down), sd.view(self.E, self.H)

    def forward(self, x, logits, shared=None):
        """x bf16 [T, H], logits float32 [T, E], shared bf16 [T, H] or None -> y bf16 [T, H], and what backward needs
        (its own expert rows among it: any number of forward calls may come before a backward)."""
        idx, w, off, row_of, row_token, load = fq.fp8q_moe_gate_topk(logits, self.topk, **self.gate)
        q, s = fq.fp8q_quant_int8(x)
        # (Rows from off[E] on are not written: they hold what the memory held, and no result comes from them.)
        c1 = fq.fp8q_grouped_gemm_int8_gather(q, s, row_token, *self.up, off)
        h = fq.fp8q_swiglu_bf16(c1[:, :self.F], c1[:, self.F:])
        q, s = fq.fp8q_quant_int8(h)
        self.c2 = c2 = fq.fp8q_grouped_gemm_int8(q, s, *self.down, off)  # (self.c2: the last call's, to look at)
        y = fq.fp8q_moe_combine(c2, row_of, w, add=shared)
        return y, (logits, idx, w, off, row_of, row_token, c2, load)

    def backward(self, grad_y, saved):
        """Gradients of the forward call that gave `saved`: of the expert rows [rows, H] and of the logits [T, E]."""
        logits, idx, w, off, row_of, row_token, c2, _ = saved
        grad_c, grad_w = fq.fp8q_moe_combine_backward(grad_y, c2, row_of, w, row_token, off)
        return grad_c, fq.fp8q_moe_gate_backward(logits, idx, grad_w, score="sigmoid", scale=self.gate["scale"])


def reference(x, logits, up, down, idx, shared, scale):
    """The layer in float64 from the unquantized weights, for the experts that were chosen."""
    v = torch.sigmoid(logits.double()).gather(1, idx.long())
    w = scale * v / v.sum(1, keepdim=True)
    y = torch.zeros(x.shape, dtype=torch.float64, device=x.device) if shared is None else shared.double()
    for e in range(up.shape[0]):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        if t.numel():
            g, u = (x[t].double() @ up[e].double().t()).chunk(2, dim=1)
            y.index_add_(0, t, w[t, j, None] * ((torch.nn.functional.silu(g) * u) @ down[e].double().t()))
    return y


def main():
    ap = argparse.ArgumentParser()
    for name, value in (("tokens", 512), ("hidden", 1024), ("width", 512), ("experts", 32), ("topk", 4)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    g = torch.Generator(device="cuda").manual_seed(0)

    def randn(*shape, scale=1.0):
        return (scale * torch.randn(shape, device="cuda", generator=g)).bfloat16()

    x, shared = randn(a.tokens, a.hidden), randn(a.tokens, a.hidden)
    up, down = randn(a.experts, 2 * a.width, a.hidden, scale=a.hidden ** -0.5), randn(a.experts, a.hidden, a.width, scale=a.width ** -0.5)
    logits = torch.randn((a.tokens, a.experts), device="cuda", generator=g)
    layer = Int8MoE(up, down, a.topk, bias=0.05 * torch.randn(a.experts, device="cuda", generator=g), n_group=4,
                    topk_group=2, scale=2.5)
    y, saved = layer.forward(x, logits, shared)
    want = reference(x, logits, up, down, saved[1], shared, 2.5)
    print("relative error of the layer against float64: %.2e" % float((y.double() - want).norm() / want.norm()))
    print("tokens per expert: least %d, most %d" % (int(saved[-1].min()), int(saved[-1].max())))
    grad_c, grad_logits = layer.backward(torch.ones_like(y), saved)
    print("gradient of the router's logits: norm %.4f" % float(grad_logits.norm()))
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for _ in range(5):
        layer.forward(x, logits, shared)
    begin.record()
    for _ in range(20):
        layer.forward(x, logits, shared)
    end.record()
    torch.cuda.synchronize()
    print("forward: %.1f us" % (begin.elapsed_time(end) / 20 * 1e3))


if __name__ == "__main__":
    main()
