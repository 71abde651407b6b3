"""A training step of a pre-norm mixture-of-experts block in FP8: forward, and every gradient.

    python examples/moe_block_fp8.py [--tokens 1024] [--hidden 1024] [--width 512] [--experts 16] [--topk 4]

The block adds the residual, norms its input and quantizes it in one pass; the experts' up product reads the routed tokens
in place, SwiGLU and its quantization feed the down product, and the combination adds the experts' rows to the residual
stream.  What it keeps for the backward pass is in 8 bits: the normed tokens (with power-of-two scales, so that their
transposed copy keeps its values) and SwiGLU's inputs.  The backward pass turns them into transposed copies, recomputes
SwiGLU, and takes all products in FP8; the weights' gradients are fp32, and may be added to those of earlier micro-batches.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fine_grained_quantization_amd as fq  # noqa: E402


def quantize_weights(w):
    """bf16 [E, N, K] -> codes and 128x128 scales for the forward product, and those of every expert's transpose.  The blocks
    are square, so the transpose has the same codes and scales."""
    E, N, K = w.shape
    q, s = fq.fp8q_quant_w_128x128(w.view(E * N, K))
    q, s = q.view(E, N, K), s.view(E, N // 128, K // 128)
    return (q, s), (q.transpose(1, 2).contiguous(), s.transpose(1, 2).contiguous())


class Fp8MoEBlock:
    """y = h + experts(norm(h)), h = x + residual.  Experts [E] of hidden size H and width F (multiples of 128): up [E, 2F, H]
    (gate rows, then up rows), down [E, H, F], in bf16; the norm's weight float32 [H]."""

    def __init__(self, norm, up, down, topk, scale=1.0):
        self.E, F2, self.H = up.shape
        self.F, self.topk, self.norm = F2 // 2, topk, norm
        self.gate = dict(score="sigmoid", scale=scale)
        self.up, self.up_t = quantize_weights(up)
        self.down, self.down_t = quantize_weights(down)

    def forward(self, x, residual, logits):
        """x and residual bf16 [T, H], logits float32 [T, E] -> y bf16 [T, H], and what backward needs."""
        q, s, h, rstd = fq.fp8q_rmsnorm_quant_act_1x128(x, self.norm, residual=residual, pow2=True)
        idx, w, off, row_of, row_token, _ = fq.fp8q_moe_gate_topk(logits, self.topk, **self.gate)
        # (Rows from off[E] on are not written: they hold what the memory held, and no result comes from them.)
        c1 = fq.fp8q_grouped_gemm_blockscaled_gather(q, s, row_token, *self.up, off)
        act = fq.fp8q_swiglu_quant_act_1x128(c1)
        kept = fq.fp8q_quant_act_1x128(c1)
        c2 = fq.fp8q_grouped_gemm_blockscaled(*act, *self.down, off)
        y = fq.fp8q_moe_combine(c2, row_of, w, add=h)
        return y, (q, s, h, rstd, logits, idx, w, off, row_of, row_token, kept, c2)

    def backward(self, grad_y, saved, grads=None):
        """Gradients of the forward call that gave `saved`: of x (and of the residual), of the logits, of the norm's weight,
        and of up and down in float32, added to `grads` = (up, down) where given."""
        q, s, h, rstd, logits, idx, w, off, row_of, row_token, kept, c2 = saved
        dup, ddown = (None, None) if grads is None else grads
        add = grads is not None
        gc, gw = fq.fp8q_moe_combine_backward(grad_y, c2, row_of, w, row_token, off)
        glogits = fq.fp8q_moe_gate_backward(logits, idx, gw, **self.gate)
        gh = fq.fp8q_grouped_gemm_blockscaled(*fq.fp8q_quant_act_1x128(gc), *self.down_t, off)
        g1, s1, g1t, e1t, ht, eht = fq.fp8q_swiglu_backward_quant(*kept, gh)
        ddown = fq.fp8q_grouped_gemm_wgrad(*fq.fp8q_quant_act_128x1(gc), ht, eht, off, accumulate=add, dw=ddown)
        gr = fq.fp8q_grouped_gemm_blockscaled(g1, s1, *self.up_t, off)
        dup = fq.fp8q_grouped_gemm_wgrad(g1t, e1t, *fq.fp8q_transpose_act_128x1(q, s, row_token=row_token), off,
                                         accumulate=add, dw=dup)
        gn = fq.fp8q_moe_combine(gr, row_of, torch.ones_like(w))  # the sum of each token's rows
        gx, gnorm = fq.fp8q_rmsnorm_backward(gn, h, self.norm, rstd, gres=grad_y)
        return gx, glogits, gnorm, dup, ddown


def dequantized(q, s):
    """float64 [E, N, K] of weights in 128x128 blocks."""
    s = s.double().repeat_interleave(128, 1).repeat_interleave(128, 2)
    return q.view(torch.float8_e4m3fn).double() * s


def reference(x, residual, logits, norm, up, down, idx, scale, eps=1e-6):
    """The block in float64, for the experts that were chosen."""
    h = x + residual
    n = h * (h.pow(2).mean(1, keepdim=True) + eps).rsqrt() * norm
    v = torch.sigmoid(logits).gather(1, idx.long())
    w = scale * v / v.sum(1, keepdim=True)
    y = h
    for e in range(up.shape[0]):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        if t.numel():
            g, u = (n[t] @ up[e].t()).chunk(2, dim=1)
            y = y.index_add(0, t, w[t, j, None] * ((torch.nn.functional.silu(g) * u) @ down[e].t()))
    return y


def main():
    ap = argparse.ArgumentParser()
    for name, value in (("tokens", 1024), ("hidden", 1024), ("width", 512), ("experts", 16), ("topk", 4)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    g = torch.Generator(device="cuda").manual_seed(0)

    def randn(*shape, scale=1.0):
        return (scale * torch.randn(shape, device="cuda", generator=g)).bfloat16()

    x, residual, grad_y = (randn(a.tokens, a.hidden) for _ in range(3))
    up, down = randn(a.experts, 2 * a.width, a.hidden, scale=a.hidden ** -0.5), randn(a.experts, a.hidden, a.width, scale=a.width ** -0.5)
    norm = 1 + 0.1 * torch.randn(a.hidden, device="cuda", generator=g)
    logits = torch.randn((a.tokens, a.experts), device="cuda", generator=g)
    block = Fp8MoEBlock(norm, up, down, a.topk)
    y, saved = block.forward(x, residual, logits)
    got = block.backward(grad_y, saved)
    leaves = [t.double().requires_grad_() for t in (x, logits, norm, up, down)]
    want = reference(leaves[0], residual.double(), leaves[1], *leaves[2:], saved[5], 1.0)
    want.backward(grad_y.double())
    rel = lambda p, r: float((p.double() - r).norm() / r.norm())  # noqa: E731
    print("relative errors against float64 with unquantized weights: y %.1e" % rel(y, want.detach()), end="")
    for name, p, r in zip(("x", "logits", "norm", "up", "down"), got, leaves):
        print(", grad %s %.1e" % (name, rel(p, r.grad)), end="")
    print()
    kept = sum(t.numel() * t.element_size() for t in (*saved[:2], *saved[10]))
    print("kept in 8 bits: %.1f MB (the same values in bf16: %.1f MB)" % (
        kept / 1e6, 2 * (saved[0].numel() + saved[10][0].numel()) / 1e6))
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))

    def step():
        _, saved = block.forward(x, residual, logits)
        block.backward(grad_y, saved, got[3:])
    for _ in range(5):
        step()
    begin.record()
    for _ in range(20):
        step()
    end.record()
    torch.cuda.synchronize()
    print("forward and backward: %.1f us" % (begin.elapsed_time(end) / 20 * 1e3))


if __name__ == "__main__":
    main()
