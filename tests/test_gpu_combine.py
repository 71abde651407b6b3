"""Expert rows back to tokens, and the gradient, against float64.

A sum of k products in fp32 is within (k + 1) u of the sum of their magnitudes (u = 2^-24); a bf16 result may carry
its own rounding, 2^-9 of its magnitude (2^-8 is allowed for the pair).  The dot products add H / 256 terms per
lane, rounded up, then 10 levels of a tree."""
import numpy as np
import pytest
import torch

import fine_grained_quantization_amd as fq
import moe_int8_reference as ref
from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def problem(T, E, k, H, dt, seed, empty=0.0):
    rng = np.random.default_rng([21, seed, T, H])
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    idx[rng.random((T, k)) < empty] = -1
    rows = fq.fp8q_moe_route_capacity(T, E, k)
    offsets, row_of, row_token, _ = ref.layout(idx, E, rows)
    c = torch.from_numpy(rng.standard_normal((rows, H)).astype(np.float32)).to(DT[dt])
    w = rng.random((T, k)).astype(np.float32)
    return rng, offsets, row_of, row_token, c, w


def out_tol(want, mag, k, dt):
    return (k + 2) * ref.U * mag + (2.0 ** -8 * np.abs(want) if dt == "bf16" else 0.0) + 1e-37


SHAPES = [(1, 4, 1, 8, "bf16"), (3, 8, 2, 64, "f32"), (64, 64, 8, 7168, "bf16"), (37, 9, 8, 2056, "bf16"),
          (130, 16, 3, 1000, "f32"), (20, 24, 16, 4104, "bf16"), (5, 12, 9, 24, "f32"), (300, 6, 4, 128, "bf16")]


@pytest.mark.parametrize("T,E,k,H,dt", SHAPES)
@pytest.mark.parametrize("add,empty", [(False, 0.0), (True, 0.3)])
def test_combine(T, E, k, H, dt, add, empty):
    rng, offsets, row_of, row_token, c, w = problem(T, E, k, H, dt, 1, empty)
    base = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(DT[dt]) if add else None
    c[torch.from_numpy(row_token) < 0] = float("nan")  # rows of no token are not read
    say(f"combine T={T} k={k} H={H} {dt} add={add}")
    y = fq.fp8q_moe_combine(c.cuda(), torch.from_numpy(row_of).cuda(), torch.from_numpy(w).cuda(),
                            add=None if base is None else base.cuda())
    torch.cuda.synchronize()
    cd = c.double().numpy()
    want = np.zeros((T, H)) if base is None else base.double().numpy()
    mag = np.abs(want)
    for j in range(k):
        on = row_of[:, j] >= 0
        v = w[on, j:j + 1].astype(np.float64) * cd[row_of[on, j]]
        want[on] += v
        mag[on] += np.abs(v)
    got = y.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= out_tol(want, mag, k + 1, dt))


def test_combine_ignores_rows_out_of_range_and_keeps_nan_apart():
    c = torch.ones((4, 16), device="cuda")
    c[2] = float("nan")
    row_of = torch.tensor([[0, 7], [-9, 3], [2, 0], [4, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    w = torch.full((4, 2), 0.5, device="cuda")
    y = fq.fp8q_moe_combine(c, row_of, w).cpu()
    assert (y[0] == 0.5).all() and (y[1] == 0.5).all() and torch.isnan(y[2]).all() and (y[3] == 0).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_tokens_without_rows_keep_what_is_added(dt):
    """Bit for bit, signed zeros, infinities and NaN too."""
    add = torch.tensor([0.0, -0.0, 1.5, -2.0, float("inf"), float("-inf"), float("nan"), 1e-38], dtype=DT[dt]).repeat(3, 2)
    row_of = torch.full((3, 5), -1, dtype=torch.int32, device="cuda")
    y = fq.fp8q_moe_combine(torch.ones((2, 16), dtype=DT[dt], device="cuda"), row_of, torch.ones((3, 5), device="cuda"),
                            add=add.cuda()).cpu()
    bits = torch.int16 if dt == "bf16" else torch.int32
    assert torch.equal(torch.isnan(y), torch.isnan(add))
    assert torch.equal(y.view(bits)[~torch.isnan(y)], add.view(bits)[~torch.isnan(add)])
    y = fq.fp8q_moe_combine(torch.ones((2, 16), dtype=DT[dt], device="cuda"), row_of, torch.ones((3, 5), device="cuda"))
    assert (y.cpu().view(bits) == 0).all()


@pytest.mark.parametrize("T,E,k,H,dt", SHAPES)
@pytest.mark.parametrize("empty", [0.0, 0.3])
def test_combine_gradient(T, E, k, H, dt, empty):
    rng, offsets, row_of, row_token, c, w = problem(T, E, k, H, dt, 2, empty)
    gy = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(DT[dt])
    rows = len(row_token)
    gc = torch.full((rows, H), 77.0, dtype=DT[dt], device="cuda")
    say(f"combine backward T={T} k={k} H={H} {dt} empty={empty}")
    gc, gw = fq.fp8q_moe_combine_backward(gy.cuda(), c.cuda(), torch.from_numpy(row_of).cuda(),
                                          torch.from_numpy(w).cuda(), torch.from_numpy(row_token).cuda(),
                                          torch.from_numpy(offsets).cuda(), grad_c=gc)
    torch.cuda.synchronize()
    g, cd = gy.double().numpy(), c.double().numpy()
    want = np.full((rows, H), 77.0)
    want[:offsets[-1]] = 0.0
    wantw, magw = np.zeros((T, k)), np.zeros((T, k))
    for j in range(k):
        on = row_of[:, j] >= 0
        want[row_of[on, j]] = w[on, j:j + 1].astype(np.float64) * g[on]
        v = g[on] * cd[row_of[on, j]]
        wantw[on, j], magw[on, j] = v.sum(1), np.abs(v).sum(1)
    got = gc.double().cpu().numpy()
    tol = ref.U * np.abs(want) + (2.0 ** -8 * np.abs(want) if dt == "bf16" else 0.0)
    tol[offsets[-1]:] = 0.0
    assert np.all(np.abs(got - want) <= tol)
    assert np.all(np.abs(gw.double().cpu().numpy() - wantw) <= ((H + 255) // 256 + 10 + 8) * ref.U * magw)
    # Differences: y is linear in c and in the weights, so a whole step of one weight changes <grad_y, y> by the
    # gradient, up to what the two sums' rounding leaves (bounded by k + 2 roundings of each term).
    if dt == "f32" and not empty:
        t, j = T // 2, k - 1
        dev = [c.cuda(), torch.from_numpy(row_of).cuda()]
        w2 = w.copy()
        w2[t, j] += 1.0
        y0 = fq.fp8q_moe_combine(*dev, torch.from_numpy(w).cuda()).double().cpu().numpy()[t]
        y1 = fq.fp8q_moe_combine(*dev, torch.from_numpy(w2).cuda()).double().cpu().numpy()[t]
        step = float(w2[t, j]) - float(w[t, j])
        m = sum(np.abs(w2[t, i] * cd[row_of[t, i]]) for i in range(k))
        tol = 2 * (k + 2) * ref.U * float((np.abs(g[t]) * m).sum()) + 64 * ref.U * magw[t, j]
        assert abs(float((g[t] * (y1 - y0)).sum()) / step - float(gw[t, j])) <= tol


def test_empty_problems():
    i32 = dict(dtype=torch.int32, device="cuda")
    none = torch.empty((0, 2), **i32)
    assert fq.fp8q_moe_combine(torch.ones((128, 8), device="cuda"), none, torch.empty((0, 2), device="cuda")).shape == (0, 8)
    y = fq.fp8q_moe_combine(torch.empty((0, 8), device="cuda"), torch.zeros((3, 2), **i32), torch.ones((3, 2), device="cuda"))
    assert (y == 0).all()
    gc = torch.full((128, 8), 5.0, device="cuda")
    off = torch.tensor([0, 0], **i32)
    fq.fp8q_moe_combine_backward(torch.empty((0, 8), device="cuda"), torch.ones((128, 8), device="cuda"), none,
                                 torch.empty((0, 2), device="cuda"), torch.full((128,), -1, **i32), off, grad_c=gc)
    assert (gc == 5.0).all()
    _, gw = fq.fp8q_moe_combine_backward(torch.empty((3, 0), device="cuda"), torch.empty((128, 0), device="cuda"),
                                         torch.zeros((3, 2), **i32), torch.ones((3, 2), device="cuda"),
                                         torch.full((128,), -1, **i32), off)
    assert (gw == 0).all()


def test_rows_past_four_gigabytes():
    """600,000 expert rows of 4096 bf16 values are 4.9 GB."""
    rows, H, T = 600_064, 4096, 5
    c = torch.zeros((rows, H), dtype=torch.bfloat16, device="cuda")
    row_of = torch.tensor([[0, rows - 1], [rows - 2, 3], [300_000, 599_000], [524_288, 1], [rows - 5, -1]],
                          dtype=torch.int32, device="cuda")
    for t in range(T):
        for j in range(2):
            if int(row_of[t, j]) >= 0:
                c[int(row_of[t, j])] = 1.0 + t + 0.25 * j
    w = torch.tensor([[1.0, 2.0]], device="cuda").repeat(T, 1).contiguous()
    say("combine past 4 GiB")
    y = fq.fp8q_moe_combine(c, row_of, w).float().cpu()
    for t in range(T):
        assert (y[t] == (1.0 + t) + (2.0 * (1.25 + t) if t != 4 else 0.0)).all()
    row_token = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    for t in range(T):
        for j in range(2):
            if int(row_of[t, j]) >= 0:
                row_token[int(row_of[t, j])] = t
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    gy = torch.ones((T, H), dtype=torch.bfloat16, device="cuda")
    gc, gw = fq.fp8q_moe_combine_backward(gy, c, row_of, w, row_token, off)
    torch.cuda.synchronize()
    for t in range(T):
        for j in range(2):
            r = int(row_of[t, j])
            assert float(gw[t, j]) == (H * (1.0 + t + 0.25 * j) if r >= 0 else 0.0)
            if r >= 0:
                assert (gc[r].float() == 1.0 + j).all()
    assert float(gc.float().sum(dtype=torch.float64)) == H * (5 * 1.0 + 4 * 2.0)


def test_combine_wants_its_arguments_right():
    i = torch.zeros((3, 2), dtype=torch.int32, device="cuda")
    c, w = torch.zeros((128, 16), device="cuda"), torch.zeros((3, 2), device="cuda")
    bad = [lambda: fq.fp8q_moe_combine(c.half(), i, w), lambda: fq.fp8q_moe_combine(c, i.long(), w),
           lambda: fq.fp8q_moe_combine(c, i, w[:2]), lambda: fq.fp8q_moe_combine(c[:, :12].contiguous(), i, w),
           lambda: fq.fp8q_moe_combine(c[:, ::2], i, w), lambda: fq.fp8q_moe_combine(c, i, w, add=c[:2]),
           lambda: fq.fp8q_moe_combine(c, i, w, add=torch.zeros((3, 16), device="cuda").bfloat16()),
           lambda: fq.fp8q_moe_combine(c.view(-1)[1:129].view(8, 16), i, w),  # off 16-byte alignment
           lambda: fq.fp8q_moe_combine(c, torch.zeros((3, 17), dtype=torch.int32, device="cuda"), torch.zeros((3, 17), device="cuda")),
           lambda: fq.fp8q_moe_combine_backward(c[:2], c, i, w, torch.zeros(128, dtype=torch.int32, device="cuda"), i[0]),
           lambda: fq.fp8q_moe_combine_backward(c[:3], c, i, w, torch.zeros(127, dtype=torch.int32, device="cuda"), i[0])]
    for f in bad:
        with pytest.raises((ValueError, RuntimeError)):
            f()
