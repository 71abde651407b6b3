"""MoE gating with scores, bias, groups and weights, its layout and its gradient, against a plain 64-bit reference.

Experts, rows and loads have to be equal; logits are drawn so that no choice hangs on a relative difference under
1e-5 (tokens that do are drawn again), except where scores are equal outright.  Weights: exp to 2 units in the last
place of its argument's rounding (|x - max| u, at most 40 u here), the sum of E positive terms in a tree (at most 40
roundings), the sum of up to 16 scores and three quotients and products: together under 128 u relative, u = 2^-24.
Gradients: the same scores within sums of at most 16 terms, 256 u of the magnitudes that are added up."""
import numpy as np
import pytest
import torch

import fine_grained_quantization_amd as fq
import moe_int8_reference as ref
from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu

W_TOL = 128 * ref.U
G_TOL = 256 * ref.U
BF16_TOL = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def draw(rng, T, E, k, kind, bias, groups, dtype, off=()):
    """Logits [T, E] (float32 values, exact in dtype) of decided tokens."""
    x = np.zeros((T, E), np.float32)
    for t in range(T):
        for _ in range(100):
            row = rng.standard_normal(E).astype(np.float32) * 1.5
            if dtype == torch.bfloat16:
                row = torch.from_numpy(row).bfloat16().float().numpy()
            row[list(off)] = -np.inf
            if ref.gate_token(row, k, kind, bias, *groups, True, 1.0)[2] > 1e-5:
                break
        x[t] = row
    return x


def call(x, k, dtype=torch.float32, **kw):
    d = torch.from_numpy(x).to(dtype).cuda()
    if kw.get("bias") is not None:
        kw = dict(kw, bias=torch.from_numpy(np.asarray(kw["bias"], np.float32)).cuda())
    got = fq.fp8q_moe_gate_topk(d, k, **kw)
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in got]


def check(x, k, kind, bias, groups, renorm, scale, got, rows=None):
    T, E = x.shape
    idx, w, offsets, row_of, row_token, load = got
    exp = [ref.gate_token(x[t], k, kind, bias, *groups, renorm, scale) for t in range(T)]
    eidx = np.array([e[0] for e in exp], np.int32).reshape(T, k)
    ew = np.array([e[1] for e in exp]).reshape(T, k)
    assert np.array_equal(idx, eidx)
    assert np.all(np.abs(w - ew) <= W_TOL * np.abs(ew) + 1e-37)
    eo, er, et, el = ref.layout(eidx, E, len(row_token))
    assert np.array_equal(offsets, eo) and np.array_equal(load, el)
    assert np.array_equal(row_of, er) and np.array_equal(row_token, et)


CASES = [  # T, E, k, score, bias, (n_group, topk_group, group_top), renorm, scale, dtype, offline experts
    (1, 256, 8, "sigmoid", True, (8, 4, 2), True, 2.5, "f32", 0),
    (3, 1, 1, "sigmoid", False, (1, 1, 2), True, 1.0, "f32", 0),
    (5, 2, 2, "softmax", False, (1, 1, 1), False, 1.0, "bf16", 0),
    (31, 7, 3, "softmax", True, (1, 1, 1), True, 1.0, "f32", 0),
    (32, 64, 6, "sigmoid", False, (1, 1, 1), True, 1.0, "bf16", 3),
    (33, 65, 8, "softmax", True, (5, 2, 1), True, 2.5, "f32", 7),
    (64, 96, 4, "sigmoid", True, (3, 1, 2), False, 1.5, "f32", 0),
    (65, 128, 16, "softmax", False, (4, 4, 2), True, 1.0, "f32", 0),
    (100, 255, 8, "sigmoid", True, (1, 1, 2), True, 1.0, "bf16", 20),
    (130, 33 * 4, 6, "sigmoid", True, (33, 7, 2), True, 1.0, "f32", 0),
    (40, 64 * 16, 16, "softmax", True, (64, 9, 1), False, 1.0, "f32", 0),
    (70, 64, 2, "sigmoid", True, (64, 3, 2), True, 1.0, "f32", 0),
    (50, 1000, 9, "sigmoid", True, (1, 1, 1), True, 1.0, "f32", 0),
    (257, 320, 8, "softmax", False, (10, 3, 2), True, 1.0, "f32", 10),
    (34, 3 * 341, 12, "sigmoid", True, (3, 2, 2), True, 1.0, "f32", 0),
    (1500, 16, 2, "sigmoid", True, (4, 2, 1), True, 1.0, "bf16", 0),
]


@pytest.mark.parametrize("T,E,k,kind,bias,groups,renorm,scale,dt,off", CASES)
def test_gate_against_the_reference(T, E, k, kind, bias, groups, renorm, scale, dt, off):
    rng = np.random.default_rng([7, T, E, k])
    dtype = torch.bfloat16 if dt == "bf16" else torch.float32
    b = (0.05 * rng.standard_normal(E)).astype(np.float32) if bias else None
    gone = rng.choice(E, size=off, replace=False) if off else ()
    x = draw(rng, T, E, k, kind, b, groups, dtype, gone)
    say(f"gate T={T} E={E} k={k} {kind} groups={groups} {dt}")
    got = call(x, k, dtype, score=kind, bias=b, n_group=groups[0], topk_group=groups[1], group_top=groups[2],
               renormalize=renorm, scale=scale)
    check(x, k, kind, b, groups, renorm, scale, got)


def test_equal_scores_go_to_the_lower_index():
    x = np.zeros((70, 48), np.float32)
    x[1:30, 5] = -0.0
    x[30:, 40:] = 1.0
    for groups in ((1, 1, 2), (6, 2, 1), (6, 2, 2)):
        for kind in ("sigmoid", "softmax"):
            say(f"gate ties {groups} {kind}")
            got = call(x, 9, score=kind, n_group=groups[0], topk_group=groups[1], group_top=groups[2])
            check(x, 9, kind, None, groups, True, 1.0, got)


def test_masked_infinite_and_extreme_logits():
    big = np.finfo(np.float32).max
    E, k = 24, 4
    x = np.full((40, E), -np.inf, np.float32)
    x[0] = np.nan                                   # nothing left
    x[2, 7] = 1.0                                   # one expert left
    x[3, [1, 20]] = [-big, big]
    x[4] = np.linspace(-3, 3, E)
    x[4, 3:20] = np.nan
    x[5] = np.linspace(-3, 3, E)
    x[5, [2, 9]] = np.inf                           # counts as the largest finite value: equal, the lower first
    x[6] = -big                                     # the type's lowest value is not a mask
    x[7] = np.linspace(-90, -80, E)
    x[8] = np.linspace(80, 90, E)[::-1]
    x[33:] = np.linspace(2, -2, E)
    for kind, groups in (("softmax", (1, 1, 1)), ("sigmoid", (1, 1, 1)), ("softmax", (4, 2, 2))):
        for T in (9, 40):                           # one launch, and two
            sel = x[:T].copy()
            if kind == "sigmoid":
                sel[8] = 0.0                        # (1 / (1 + e^-80) is 1 for every expert in fp32, not in 64 bits)
            say(f"gate masks {kind} {groups} T={T}")
            got = call(sel, k, score=kind, n_group=groups[0], topk_group=groups[1], group_top=groups[2])
            assert not np.isnan(got[1]).any()
            check(sel, k, kind, None, groups, True, 1.0, got)


@pytest.mark.parametrize("T,E,k", [(8200, 12, 2), (20000, 40, 3), (9000, 1024, 1), (4096, 36, 5), (4097, 36, 5), (2000, 37, 4)])
def test_layout_of_many_tokens(T, E, k):
    """Past 256 chunks a workgroup places several of them."""
    rng = np.random.default_rng([8, T])
    x = np.argsort(rng.random((T, E)), axis=1).astype(np.float32) / np.float32(64.0)  # distinct in every row
    say(f"gate layout T={T} E={E}")
    # (softmax: neighbours differ by 1/64 of their value; the sigmoid of logits up to 16 is 1 for many in fp32)
    idx, w, offsets, row_of, row_token, load = call(x, k, score="softmax")
    eidx = np.argsort(-x, axis=1, kind="stable")[:, :k].astype(np.int32)
    assert np.array_equal(idx, eidx)
    eo, er, et, el = ref.layout(eidx, E, len(row_token))
    assert np.array_equal(offsets, eo) and np.array_equal(load, el)
    assert np.array_equal(row_of, er) and np.array_equal(row_token, et)


def test_no_tokens_strided_rows_and_spare_rows():
    got = call(np.zeros((0, 10), np.float32), 2)
    assert (got[2] == 0).all() and (got[4] == -1).all() and (got[5] == 0).all()
    rng = np.random.default_rng(9)
    x = draw(rng, 50, 30, 3, "sigmoid", None, (1, 1, 2), torch.float32)
    wide = torch.full((50, 47), float("nan"), device="cuda")
    wide[:, 5:35] = torch.from_numpy(x).cuda()
    view = wide[:, 5:35]
    assert view.stride(0) == 47
    rows = fq.fp8q_moe_route_capacity(50, 30, 3) + 130
    base = torch.full((rows + 1,), 77, dtype=torch.int32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    out = (torch.empty((50, 3), **i32), torch.empty((50, 3), device="cuda"), torch.empty(31, **i32),
           torch.empty((50, 3), **i32), base[1:], torch.empty(30, **i32))  # row_token off 16-byte alignment
    say("gate strided")
    fq.fp8q_moe_gate_topk(view, 3, rows=rows, out=out)
    torch.cuda.synchronize()
    check(x, 3, "sigmoid", None, (1, 1, 2), True, 1.0, [t.cpu().numpy() for t in out])
    assert int(base[0]) == 77


def test_gate_repeats_bit_for_bit_and_agrees_over_batch_sizes():
    """A token's choice and weights do not depend on the tokens beside it."""
    rng = np.random.default_rng(10)
    x = rng.standard_normal((300, 256)).astype(np.float32)
    kw = dict(score="softmax", n_group=8, topk_group=3, group_top=2)
    a, b = call(x, 8, **kw), call(x, 8, **kw)
    one = call(x[100:117], 8, **kw)
    assert all(np.array_equal(p, q) for p, q in zip(a, b))
    assert np.array_equal(a[0][100:117], one[0]) and np.array_equal(a[1][100:117], one[1])


MANY = [  # T, E, k, score, bias, groups, renorm, scale, dtype: past 4096 tokens with E % 4 == 0, 16 lanes a token
    (5000, 256, 8, "sigmoid", True, (8, 4, 2), True, 2.5, "f32"),    # 16 experts a lane, logits and bias as vectors
    (4200, 256, 8, "sigmoid", True, (8, 4, 2), True, 2.5, "bf16"),
    (4300, 512, 16, "softmax", True, (1, 1, 2), False, 1.0, "bf16"),  # 32
    (4097, 512, 8, "softmax", True, (8, 3, 1), True, 1.0, "f32"),
    (4500, 160, 6, "softmax", False, (8, 3, 1), True, 1.0, "f32"),   # 20 experts a group: 16 a lane, no vectors
    (4123, 64, 6, "softmax", True, (1, 1, 1), True, 1.0, "f32"),     # 4
    (4444, 12, 3, "sigmoid", True, (3, 2, 2), False, 1.5, "bf16"),   # 1
    (4100, 1024, 9, "sigmoid", True, (16, 5, 2), True, 1.0, "f32"),  # 64 experts a lane would be too many: 64 lanes a token
]


def many(T, E, k, kind, bias, groups, dt):
    """Logits of T tokens, the sampled ones (32 of them, the first and the last too) decided, and the bias."""
    rng = np.random.default_rng([14, T, E])
    dtype = torch.bfloat16 if dt == "bf16" else torch.float32
    b = (0.05 * rng.standard_normal(E)).astype(np.float32) if bias else None
    at = np.sort(np.concatenate([[0, T - 1], 1 + rng.choice(T - 2, 30, replace=False)]))
    x = 1.5 * rng.standard_normal((T, E)).astype(np.float32)
    x = torch.from_numpy(x).to(dtype).float().numpy()
    x[at] = draw(rng, len(at), E, k, kind, b, groups, dtype)
    return x, b, at, dtype


@pytest.mark.parametrize("T,E,k,kind,bias,groups,renorm,scale,dt", MANY)
def test_many_tokens_against_the_reference(T, E, k, kind, bias, groups, renorm, scale, dt):
    """Experts and weights of sampled tokens; the layout of all tokens from their experts."""
    x, b, at, dtype = many(T, E, k, kind, bias, groups, dt)
    say(f"gate many T={T} E={E} k={k} {kind} groups={groups} {dt}")
    idx, w, offsets, row_of, row_token, load = call(x, k, dtype, score=kind, bias=b, n_group=groups[0],
                                                    topk_group=groups[1], group_top=groups[2], renormalize=renorm,
                                                    scale=scale)
    for t in at:
        eidx, ew, _ = ref.gate_token(x[t], k, kind, b, *groups, renorm, scale)
        assert np.array_equal(idx[t], eidx)
        assert np.all(np.abs(w[t] - ew) <= W_TOL * np.abs(ew) + 1e-37)
    assert (idx >= 0).all() and (idx < E).all()
    eo, er, et, el = ref.layout(idx, E, len(row_token))
    assert np.array_equal(offsets, eo) and np.array_equal(load, el)
    assert np.array_equal(row_of, er) and np.array_equal(row_token, et)


@pytest.mark.parametrize("T,E,k,kind,bias,groups,renorm,scale,dt", MANY + [
    (4600, 256, 8, "softmax", True, (8, 4, 2), True, 1.0, "f32"), (4600, 256, 8, "softmax", False, (1, 1, 2), False, 1.0, "bf16")])
def test_a_tokens_answer_does_not_depend_on_its_batch(T, E, k, kind, bias, groups, renorm, scale, dt):
    """Bit for bit: many tokens (16 lanes each), batches of hundreds (64 lanes) and few tokens (one launch); masked experts
    and infinities among them."""
    x, b, at, dtype = many(T, E, k, kind, bias, groups, dt)
    x[5, ::3] = -np.inf
    x[6, 1] = np.inf
    x[7] = np.nan
    kw = dict(score=kind, bias=b, n_group=groups[0], topk_group=groups[1], group_top=groups[2], renormalize=renorm,
              scale=scale)
    say(f"gate batches T={T} E={E} k={k} {kind} groups={groups} {dt}")
    whole = call(x, k, dtype, **kw)
    for a, n in ((0, 1), (0, 32), (3, 33), (100, 700), (T - 50, 50), (T - 31, 31), (0, 4096)):
        part = call(x[a:a + n], k, dtype, **kw)
        assert np.array_equal(whole[0][a:a + n], part[0])
        assert np.array_equal(whole[1][a:a + n].view(np.uint32), part[1].view(np.uint32))


@pytest.mark.parametrize("most,E", [(6000, 256), (4097, 64), (33, 8), (5000, 36)])
def test_a_workspace_made_for_a_batch_does_for_smaller_ones(most, E):
    """Bit for bit the results of a call with a workspace of its own."""
    need = fq.load_library().fp8q_moe_gate_workspace_bytes
    rng = np.random.default_rng([13, most])
    x = torch.from_numpy(rng.standard_normal((most, E)).astype(np.float32)).cuda()
    for T in sorted({t for t in (1, 32, 33, 40, 2000, 3009, 4095, 4096, 4097, most) if t <= most}):
        ws = torch.full((need(most, E) + 64,), 0xA5, dtype=torch.uint8, device="cuda")
        say(f"gate workspace for {most} tokens, T={T} E={E}")
        for score in ("sigmoid", "softmax"):
            got = fq.fp8q_moe_gate_topk(x[:T], 4, score=score, n_group=4, topk_group=2, workspace=ws[:need(most, E)])
            want = fq.fp8q_moe_gate_topk(x[:T], 4, score=score, n_group=4, topk_group=2)
            assert all(torch.equal(a.view(torch.int32), b.view(torch.int32)) for a, b in zip(got, want))
        assert (ws[need(most, E):] == 0xA5).all()


GRADS = [  # T, E, k, score, renorm, scale, dtype
    (1, 256, 8, "sigmoid", True, 2.5, "f32"), (7, 5, 2, "softmax", True, 1.0, "f32"),
    (130, 64, 8, "softmax", False, 1.0, "bf16"), (33, 100, 3, "sigmoid", False, 1.5, "f32"),
    (9, 1024, 16, "softmax", True, 1.0, "f32"), (20, 513, 4, "softmax", False, 2.0, "f32"),
    (3, 1, 1, "sigmoid", False, 1.0, "f32"), (50, 96, 6, "sigmoid", True, 1.0, "bf16"),
]


def backward(x, idx, dw, dtype, **kw):
    d = torch.from_numpy(x).to(dtype).cuda()
    g = fq.fp8q_moe_gate_backward(d, torch.from_numpy(idx).cuda(), torch.from_numpy(dw).cuda(), **kw)
    torch.cuda.synchronize()
    assert g.dtype == dtype
    return g.float().cpu().numpy()


@pytest.mark.parametrize("T,E,k,kind,renorm,scale,dt", GRADS)
def test_gradient_against_formula_and_differences(T, E, k, kind, renorm, scale, dt):
    rng = np.random.default_rng([11, T, E])
    dtype = torch.bfloat16 if dt == "bf16" else torch.float32
    x = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).to(dtype).float().numpy()
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)  # any choice will do
    if k > 2:
        idx[0, 1] = -1
    dw = rng.standard_normal((T, k)).astype(np.float32)
    say(f"gate backward T={T} E={E} k={k} {kind} {dt}")
    g = backward(x, idx, dw, dtype, score=kind, renormalize=renorm, scale=scale)
    for t in range(T):
        want, mag = ref.gate_grad(x[t], idx[t], dw[t], kind, renorm, scale)
        tol = G_TOL * mag + (BF16_TOL * np.abs(want) if dt == "bf16" else 0.0) + 1e-37
        assert np.all(np.abs(g[t] - want) <= tol)
    # Differences of the 64-bit forward function: h^2 / 6 of third derivatives (below 4 |dw| scale per slot and
    # 1 / S^3 under renormalization) plus rounding 2^-52 / h.
    h = 1e-5
    t = 0
    S = sum(ref.scores(x[t], kind)[0][e] for e in idx[t] if e >= 0)
    slack = 1e-8 * scale * np.abs(dw[t]).sum() * (1.0 + 1.0 / min(S, 1.0) ** 3 if renorm else 1.0)
    want, mag = ref.gate_grad(x[t], idx[t], dw[t], kind, renorm, scale)
    for e in sorted(set(idx[t][idx[t] >= 0].tolist()) | set(range(min(E, 5)))):
        hi, lo = x[t].astype(np.float64), x[t].astype(np.float64)
        hi[e] += h
        lo[e] -= h
        diff = (ref.gate_weights(hi, idx[t], kind, renorm, scale) - ref.gate_weights(lo, idx[t], kind, renorm, scale))
        diff = float((dw[t] * diff).sum()) / (2 * h)
        tol = slack + G_TOL * mag[e] + (BF16_TOL * abs(want[e]) if dt == "bf16" else 0.0)
        assert abs(diff - g[t][e]) <= tol


def test_gradient_of_masked_and_strided_logits():
    rng = np.random.default_rng(12)
    x = rng.standard_normal((6, 20)).astype(np.float32)
    x[0] = -np.inf
    x[1, 3:9] = -np.inf
    x[2, 5] = np.nan
    x[3] = np.linspace(-95, 95, 20)
    idx = np.tile(np.array([[4, 1, 12]], np.int32), (6, 1))
    idx[0] = -1
    idx[4] = [20, -5, 7]  # outside [0, E): empty slots
    dw = rng.standard_normal((6, 3)).astype(np.float32)
    for kind in ("sigmoid", "softmax"):
        for renorm in (True, False):
            wide = torch.zeros((6, 31), device="cuda")
            wide[:, 4:24] = torch.from_numpy(x).cuda()
            say(f"gate backward masks {kind} {renorm}")
            g = fq.fp8q_moe_gate_backward(wide[:, 4:24], torch.from_numpy(idx).cuda(), torch.from_numpy(dw).cuda(),
                                          score=kind, renormalize=renorm)
            torch.cuda.synchronize()
            g = g.cpu().numpy()
            assert np.isfinite(g).all() and (g[0] == 0).all() and (g[1, 3:9] == 0).all() and g[2, 5] == 0
            for t in range(6):
                at = np.where((idx[t] >= 0) & (idx[t] < 20), idx[t], -1)
                want, mag = ref.gate_grad(x[t], at, dw[t], kind, renorm, 1.0)
                assert np.all(np.abs(g[t] - want) <= G_TOL * mag + 1e-30)


def test_gate_wants_its_arguments_right():
    d = torch.zeros((4, 12), device="cuda")
    i = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    w = torch.zeros((4, 2), device="cuda")
    bad = [lambda: fq.fp8q_moe_gate_topk(d.double(), 2), lambda: fq.fp8q_moe_gate_topk(d.cpu(), 2),
           lambda: fq.fp8q_moe_gate_topk(d.t(), 2), lambda: fq.fp8q_moe_gate_topk(d[0], 2),
           lambda: fq.fp8q_moe_gate_topk(d, 2, score="relu"), lambda: fq.fp8q_moe_gate_topk(d, 2, group_top=3),
           lambda: fq.fp8q_moe_gate_topk(d, 13), lambda: fq.fp8q_moe_gate_topk(d, 0),
           lambda: fq.fp8q_moe_gate_topk(d, 2, bias=torch.zeros(11, device="cuda")),
           lambda: fq.fp8q_moe_gate_topk(d, 2, bias=torch.zeros(12, device="cuda").bfloat16()),
           lambda: fq.fp8q_moe_gate_topk(d, 2, rows=128), lambda: fq.fp8q_moe_gate_topk(d, 2, n_group=5),
           lambda: fq.fp8q_moe_gate_topk(d, 2, n_group=3, topk_group=4),
           lambda: fq.fp8q_moe_gate_topk(d, 5, n_group=3, topk_group=1),
           lambda: fq.fp8q_moe_gate_topk(torch.zeros((40, 12), device="cuda"), 2, workspace=torch.zeros(8, dtype=torch.uint8, device="cuda")),
           lambda: fq.fp8q_moe_gate_backward(d, i.long(), w), lambda: fq.fp8q_moe_gate_backward(d, i[:3], w),
           lambda: fq.fp8q_moe_gate_backward(d, i, w[:, :1].contiguous()),
           lambda: fq.fp8q_moe_gate_backward(d, i, w, grad_logits=torch.zeros((4, 12), device="cuda").bfloat16())]
    for f in bad:
        with pytest.raises((ValueError, RuntimeError, TypeError)):
            f()
