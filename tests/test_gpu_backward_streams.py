"""The norm's and the backward pass's calls on streams: memory that calls given a stream allocate (workspaces, outputs that
the caller may drop at once), calls on two streams at the same time, and calls that wait for their stream's earlier work."""
import pytest
import torch

import fine_grained_quantization_amd as fq
from fine_grained_quantization_amd import _binding
from gpu_util import require_gpu, say
from test_gpu_given_stream import Recorder, busy, bytes_of, overlap

pytestmark = pytest.mark.gpu
NAMES = ["norm", "norm without residual", "norm gradient", "norm gradient, few rows", "transpose", "transpose routed",
         "backward copy", "swiglu gradient", "weight gradient", "weight gradient, split", "experts"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def operands():
    g = torch.Generator(device="cuda").manual_seed(71)
    M, K, F = 4096, 512, 256

    def randn(*shape):
        return torch.randn(shape, device="cuda", generator=g).bfloat16()
    x, r, gy, gh, w = randn(M, K), randn(M, K), randn(M, K), randn(M, F), randn(K)
    q, s, _, rstd = fq.fp8q_rmsnorm_quant_act_1x128(x, w)
    gt, eg = fq.fp8q_quant_act_128x1(gy)
    gs, es = fq.fp8q_quant_act_128x1(gy[:128])
    xs, fs = fq.fp8q_transpose_act_128x1(q[:128], s[:, :128].contiguous())
    xt, ex = fq.fp8q_transpose_act_128x1(q, s)
    tok = torch.randint(-1, M, (700,), device="cuda", generator=g).int()
    off = torch.tensor([0, 128, 128, 640, 4096], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    calls = [
        lambda **k: fq.fp8q_rmsnorm_quant_act_1x128(x, w, residual=r, **k),
        lambda **k: tuple(fq.fp8q_rmsnorm_quant_act_1x128(x, w, **k)[i] for i in (0, 1, 3)),
        lambda **k: fq.fp8q_rmsnorm_backward(gy, x, w, rstd, gres=r, **k),
        lambda **k: fq.fp8q_rmsnorm_backward(gy[:100], x[:100], w, rstd[:100], **k),
        lambda **k: fq.fp8q_transpose_act_128x1(q, s, **k),
        lambda **k: fq.fp8q_transpose_act_128x1(q, s, row_token=tok, **k),
        lambda **k: fq.fp8q_quant_act_128x1(gy, **k),
        lambda **k: fq.fp8q_swiglu_backward_quant(q, s, gh, **k),
        lambda **k: fq.fp8q_gemm_wgrad(gs, es, xs, fs, **k),
        lambda **k: fq.fp8q_gemm_wgrad(gt, eg, xt, ex, **k),
        lambda **k: fq.fp8q_grouped_gemm_wgrad(gt, eg, xt, ex, off, **k),
    ]
    lib = fq.load_library()
    sizes = [lib.fp8q_rmsnorm_backward_workspace_bytes(M, K), lib.fp8q_gemm_wgrad_workspace_bytes(M, K, K, fq.OUT_F32)]
    assert min(sizes) > 0  # both forms that need a workspace are among the calls
    return calls, sizes


@pytest.mark.parametrize("which", range(len(NAMES)), ids=NAMES)
def test_memory_of_calls_on_a_given_stream(which, monkeypatch):
    calls, sizes = operands()
    f = calls[which]
    src = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    want = bytes_of(f())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    spy = Recorder(fq.load_library())
    monkeypatch.setattr(_binding, "load_library", lambda: spy)
    say(f"given stream: {NAMES[which]}")
    held = busy(side, src)
    got = f(stream=side)
    used = spy.seen
    mine = [torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda") for n in sizes + [t.numel() for t in want] for _ in range(3)]
    assert not overlap(mine, used)
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(bytes_of(got), want))
    made = {t.data_ptr() for t in (got if isinstance(got, tuple) else (got,))}
    del mine, got
    held.zero_()
    torch.cuda.synchronize()
    mine = [torch.empty(t.numel(), dtype=torch.uint8, device="cuda") for t in want for _ in range(3)]
    assert not overlap(mine, made)  # dropped outputs stay with the stream they were made on
    torch.cuda.synchronize()


def test_two_streams_at_once():
    """Every call on two streams at the same time, many times over: the results of calls alone."""
    calls, _ = operands()
    want = [bytes_of(f()) for f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for which, f in enumerate(calls):
        say(f"two streams: {NAMES[which]}")
        got = []
        for _ in range(8):
            for st in streams:
                with torch.cuda.stream(st):
                    got.append(f())
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for out in got for a, b in zip(bytes_of(out), want[which])), NAMES[which]


def test_calls_follow_their_stream():
    """Inputs that the same stream writes late, after milliseconds of copies."""
    g = torch.Generator(device="cuda").manual_seed(72)
    x, gy = (torch.randn((1000, 1024), device="cuda", generator=g).bfloat16() for _ in range(2))
    w = torch.ones(1024, device="cuda")

    def step(x, gy):
        q, s, h, rstd = fq.fp8q_rmsnorm_quant_act_1x128(x, w, pow2=True)
        gx, gw = fq.fp8q_rmsnorm_backward(gy, h, w, rstd)
        grads = fq.fp8q_swiglu_backward_quant(q, s, gy[:, :512])
        xt, ex = fq.fp8q_transpose_act_128x1(q, s)
        return (gx, gw, *grads, fq.fp8q_gemm_wgrad(*fq.fp8q_quant_act_128x1(gy), xt, ex),
                fq.fp8q_gemm_wgrad(grads[2], grads[3], xt, ex, out_dtype=torch.bfloat16))
    want = bytes_of(step(x, gy))
    src = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    late, late_g = torch.zeros_like(x), torch.zeros_like(gy)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    held = busy(side, src)
    with torch.cuda.stream(side):
        late.copy_(x)
        late_g.copy_(gy)
        got = step(late, late_g)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(bytes_of(got), want))
    del held
