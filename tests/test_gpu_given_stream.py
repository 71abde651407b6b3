"""Calls given a stream from outside its context: the memory that they allocate (workspaces nobody else sees, and
outputs that the caller may drop at once) is never handed to work of another stream that does not wait for them.

torch hands a freed block back to the stream that allocated it, without waiting.  So after a call on a busy side stream
the current stream allocates blocks of the same sizes, and none may be one that the call used; and no output may be
a block that the current stream freed before the call, where its own queued work may still write."""
import pytest
import torch

import fine_grained_quantization_amd as fq
from fine_grained_quantization_amd import _binding
from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


class Recorder:
    """The library, with the addresses that calls pass to it (every argument past the 2^32 that no size here reaches)."""

    def __init__(self, lib):
        self.lib, self.seen = lib, set()

    def __getattr__(self, name):
        f = getattr(self.lib, name)

        def call(*args):
            self.seen |= {a for a in args if isinstance(a, int) and a > 1 << 32}
            return f(*args)
        return call


def busy(stream, src):
    with torch.cuda.stream(stream):
        dst = torch.empty_like(src)
        for _ in range(40):  # 256 MB each: milliseconds
            dst.copy_(src)
    return dst


def overlap(tensors, addresses):
    return [a for a in addresses for t in tensors if t.data_ptr() <= a < t.data_ptr() + t.numel()]


def operands():
    g = torch.Generator(device="cuda").manual_seed(61)
    T, E, k, K, N = 700, 64, 4, 256, 128
    logits = torch.randn((T, E), device="cuda", generator=g)
    x = torch.randn((T, K), device="cuda", generator=g).bfloat16()
    qx, sx = fq.fp8q_quant_int8(x)
    qw, sw = fq.fp8q_quant_int8(torch.randn((E * N, K), device="cuda", generator=g).bfloat16())
    idx, w, off, row_of, row_token, _ = fq.fp8q_moe_gate_topk(logits, k)
    rows = row_token.numel()
    c = torch.randn((rows, N), device="cuda", generator=g).bfloat16()
    gy = torch.randn((T, N), device="cuda", generator=g).bfloat16()
    qa = torch.zeros((rows, K), dtype=torch.int8, device="cuda")
    sa = torch.zeros(rows, device="cuda")
    q8, s8 = fq.fp8q_quant_act_1x128(x)
    w8, v8 = fq.fp8q_quant_w_128x128(torch.randn((N, K), device="cuda", generator=g).bfloat16())
    return [
        ("gate", lambda **s: fq.fp8q_moe_gate_topk(logits, k, **s)),
        ("gate few", lambda **s: fq.fp8q_moe_gate_topk(logits[:20], k, **s)),
        ("route", lambda **s: fq.fp8q_moe_route_topk(logits, k, **s)),
        ("route without workspace", lambda **s: fq.fp8q_moe_route_topk_noalloc(logits, k, **s)),
        ("gate gradient", lambda **s: fq.fp8q_moe_gate_backward(logits, idx, w, **s)),
        ("combination", lambda **s: fq.fp8q_moe_combine(c, row_of, w, **s)),
        ("combination gradient", lambda **s: fq.fp8q_moe_combine_backward(gy, c, row_of, w, row_token, off, **s)[1]),
        ("int8 quantizer", lambda **s: fq.fp8q_quant_int8(x, **s)),
        ("int8 product", lambda **s: fq.fp8q_gemm_int8(qx, sx, qw[:N], sw[:N], **s)),
        ("int8 grouped", lambda **s: fq.fp8q_grouped_gemm_int8(qa, sa, qw.view(E, N, K), sw.view(E, N), off, **s)[:128]),
        ("int8 gather", lambda **s: fq.fp8q_grouped_gemm_int8_gather(qx, sx, row_token, qw.view(E, N, K), sw.view(E, N),
                                                                     off, **s)[:128]),
        ("fp8 quantizer", lambda **s: fq.fp8q_quant_act_1x128(x, **s)),
        ("fp8 product", lambda **s: fq.fp8q_gemm_blockscaled(q8, s8, w8, v8, **s)),
    ]


def bytes_of(out):
    out = out if isinstance(out, tuple) else (out,)
    return [t.contiguous().view(torch.uint8).clone() for t in out]


@pytest.mark.parametrize("which", range(13))
def test_memory_of_calls_on_a_given_stream(which, monkeypatch):
    name, f = operands()[which]
    src = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    want = bytes_of(f())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    spy = Recorder(fq.load_library())
    monkeypatch.setattr(_binding, "load_library", lambda: spy)
    say(f"given stream: {name}")
    held = busy(side, src)
    got = f(stream=side)
    used = spy.seen
    lib = fq.load_library()
    sizes = [lib.fp8q_moe_gate_workspace_bytes(700, 64), lib.fp8q_moe_route_workspace_bytes(700, 64)]
    sizes += [t.numel() for t in want] + [n for n in range(512, 1 << 20, 512 * 61)]
    mine = [torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    # (a call's operands keep their blocks; everything else that it used is not given out here)
    assert not overlap(mine, used)
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(bytes_of(got), want))
    # Outputs dropped while the stream is still busy, and outputs that reuse nothing the current stream has just freed.
    torch.cuda.synchronize()
    del mine, got
    spy.seen = set()
    mine = [torch.empty(t.numel(), dtype=torch.uint8, device="cuda") for t in want for _ in range(3)]
    freed = [t.data_ptr() for t in mine]
    held.zero_()
    torch.cuda.synchronize()
    held = busy(side, src)
    del mine
    got = f(stream=side)
    made = {t.data_ptr() for t in (got if isinstance(got, tuple) else (got,))}
    assert not made & set(freed)
    del got
    mine = [torch.empty(t.numel(), dtype=torch.uint8, device="cuda") for t in want for _ in range(3)]
    assert not overlap(mine, made)
    torch.cuda.synchronize()


def test_a_stream_that_is_only_a_handle():
    """A stream object of another kind: its ``cuda_stream`` is all that a call needs."""
    class Handle:
        def __init__(self, s):
            self.cuda_stream = s.cuda_stream
    side = torch.cuda.Stream()
    x = torch.randn((5, 64), device="cuda")
    torch.cuda.synchronize()
    a = fq.fp8q_moe_gate_topk(x, 3, stream=Handle(side))
    side.synchronize()
    b = fq.fp8q_moe_gate_topk(x, 3)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
