"""The norm's, the checkpoints' and the weight gradients' entry points refuse bad arguments before touching a device (CPU-only;
the addresses are never dereferenced: every call fails validation, or has nothing to do)."""
import ctypes
import os

import pytest
import torch

import fine_grained_quantization_amd as fq
from fine_grained_quantization_amd import _binding

A, B, MIS, MIS8 = ctypes.c_void_p(4096), ctypes.c_void_p(8192), ctypes.c_void_p(4098), ctypes.c_void_p(4104)
OK, NULL, SHAPE, ALIGN, DTYPE, WORKSPACE, OPTION = 0, -1, -2, -3, -4, -8, -9


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fq.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return fq.load_library()


NORM = dict(x=A, ldx=256, res=A, ldr=256, w=A, dtype=0, eps=1e-6, pow2=0, M=4, K=256, h=B, y=None, q=B, s=B, rstd=B, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(M=-1), SHAPE), (dict(K=-128), SHAPE), (dict(K=200), SHAPE), (dict(ldx=255), SHAPE), (dict(ldx=260), SHAPE),
    (dict(ldr=248), SHAPE), (dict(ldr=257), SHAPE), (dict(M=1 << 22), SHAPE), (dict(K=1 << 31, ldx=1 << 31, ldr=1 << 31), SHAPE),
    (dict(dtype=2), DTYPE), (dict(eps=0.0), OPTION), (dict(eps=-1.0), OPTION), (dict(eps=float("nan")), OPTION),
    (dict(eps=float("inf")), OPTION), (dict(pow2=2), OPTION), (dict(pow2=-1), OPTION), (dict(res=None), OPTION),
    (dict(M=0, x=None, w=None), OK), (dict(K=0, x=None), OK), (dict(x=None), NULL), (dict(w=None), NULL), (dict(q=None), NULL),
    (dict(s=None), NULL), (dict(h=None), NULL), (dict(res=None, h=None, q=None, s=None, rstd=None), NULL), (dict(x=MIS8), ALIGN),
    (dict(res=MIS8), ALIGN), (dict(w=MIS8), ALIGN), (dict(h=MIS8), ALIGN), (dict(y=MIS8), ALIGN), (dict(q=MIS8), ALIGN),
    (dict(s=MIS), ALIGN), (dict(rstd=MIS), ALIGN),
])
def test_norm(lib, change, want):
    assert set(change) <= set(NORM)
    assert lib.fp8q_rmsnorm_quant_act_1x128(*{**NORM, **change}.values()) == want


@pytest.mark.parametrize("out", ["h", "y"])
@pytest.mark.parametrize("which", ["x", "res"])
def test_norm_over_rows_that_others_read(lib, which, out):
    """h or y in place of an array whose rows are further apart than theirs, or sharing part of its memory: each row's workgroup
    would write over rows of others.  (4 rows of 256 elements: 2048 bytes of h or y from 1 << 20 on.)"""
    base, ld = 1 << 20, "ldx" if which == "x" else "ldr"
    other = "res" if which == "x" else "x"

    def call(**change):
        c = {**NORM, other: ctypes.c_void_p(1 << 30), "h": ctypes.c_void_p(1 << 31), out: ctypes.c_void_p(base), **change}
        return lib.fp8q_rmsnorm_quant_act_1x128(*c.values())

    for at, stride in ((base, 264), (base, 512), (base + 16, 256), (base - 16, 256), (base + 512, 256), (base - 512, 256),
                       (base + 2032, 256), (base - 2032, 256), (base - 2560, 1024), (base - 3 * 8192 + 2032, 4096)):
        assert call(**{which: ctypes.c_void_p(at), ld: stride}) == OPTION, (at - base, stride)
    # fine: the array itself, one row of any stride, memory before and behind, and between two rows; they pass to the next
    # check (of the device), which a machine without one fails
    if not torch.cuda.is_available():
        for at, stride, M in ((base, 256, 4), (base, 512, 1), (base - 2048, 256, 4), (base + 2048, 256, 4), (base - 512, 2048, 4),
                              (base + (1 << 25), 512, 4), (base - 4096, (1 << 63) - 8, 4)):
            assert call(**{which: ctypes.c_void_p(at), ld: stride, "M": M}) not in (OK, NULL, SHAPE, ALIGN, OPTION), (at - base, stride)


def test_norm_outputs_apart(lib):
    for y in (8192, 8192 + 2032, 8192 - 2032):
        c = {**NORM, "h": ctypes.c_void_p(8192), "y": ctypes.c_void_p(y), "x": ctypes.c_void_p(1 << 20), "res": ctypes.c_void_p(1 << 21)}
        assert lib.fp8q_rmsnorm_quant_act_1x128(*c.values()) == OPTION


GRAD = dict(gy=A, ldg=256, h=A, ldh=256, w=A, dtype=1, rstd=A, gres=None, M=200, K=256, gx=B, gw=B, ws=B, wsb=1 << 20, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(M=-1), SHAPE), (dict(M=1 << 22), SHAPE), (dict(K=100), SHAPE), (dict(K=20480 + 128, ldg=1 << 15, ldh=1 << 15), SHAPE),
    (dict(ldg=128), SHAPE), (dict(ldg=260), SHAPE), (dict(ldh=255), SHAPE), (dict(ldh=257), SHAPE), (dict(dtype=-1), DTYPE),
    (dict(M=0, gw=None, gy=None), OK), (dict(K=0, gy=None), OK), (dict(gy=None), NULL), (dict(h=None), NULL), (dict(w=None), NULL),
    (dict(rstd=None), NULL), (dict(gx=None), NULL), (dict(ws=None), NULL), (dict(gy=MIS8), ALIGN), (dict(h=MIS8), ALIGN),
    (dict(w=MIS8), ALIGN), (dict(rstd=MIS), ALIGN), (dict(gres=MIS8), ALIGN), (dict(gx=MIS8), ALIGN), (dict(gw=MIS8), ALIGN),
    (dict(gx=A), OPTION), (dict(h=B), OPTION), (dict(gres=B, wsb=0), WORKSPACE), (dict(ws=MIS8), ALIGN), (dict(wsb=-1), WORKSPACE), (dict(wsb=200 * 256 * 4 - 1), WORKSPACE),
])
def test_norm_gradient(lib, change, want):
    assert set(change) <= set(GRAD)
    assert lib.fp8q_rmsnorm_backward(*{**GRAD, **change}.values()) == want


@pytest.mark.parametrize("which,ld", [("gy", "ldg"), ("h", "ldh"), ("gres", None)])
def test_norm_gradient_over_rows_that_others_read(lib, which, ld):
    """gx sharing part of the memory of gy, h or gres (4 rows of 256 elements, 2048 bytes of gx)."""
    base = 1 << 20
    c = {**GRAD, "M": 4, "gy": ctypes.c_void_p(1 << 30), "h": ctypes.c_void_p(1 << 31), "gres": ctypes.c_void_p(1 << 32),
         "gx": ctypes.c_void_p(base)}
    for at, stride in ((16, 256), (-16, 256), (512, 256), (-512, 256), (2032, 256), (-2032, 256), (-2560, 1024), (0, 512)):
        if ld is not None or (stride == 256):
            change = {which: ctypes.c_void_p(base + at), **({ld: stride} if ld else {})}
            assert lib.fp8q_rmsnorm_backward(*{**c, **change}.values()) == OPTION, (at, stride)
    if not torch.cuda.is_available():  # fine, up to the check of the device
        for at in (-2048, 2048) if ld else (-2048, 0, 2048):
            assert lib.fp8q_rmsnorm_backward(*{**c, which: ctypes.c_void_p(base + at)}.values()) not in (OK, NULL, SHAPE, ALIGN, OPTION)


def test_norm_gradient_workspace(lib):
    need = lib.fp8q_rmsnorm_backward_workspace_bytes
    assert need(0, 256) == 0 and need(128, 7168) == 0 and need(129, 256) == 129 * 256 * 4
    assert need(-1, 256) == -1 and need(4, 100) == -1 and need(4, 20608) == -1 and need(1 << 22, 128) == -1
    for K in (128, 7168, 20480):
        sizes = [need(M, K) for M in list(range(0, 1200)) + [5000, 1 << 20]]
        assert sizes == sorted(sizes)


TRANS = dict(q=A, s=A, T=4, K=256, row_token=None, rows=4, qt=B, et=B, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(T=-1), SHAPE), (dict(T=1 << 31), SHAPE), (dict(rows=3), SHAPE), (dict(rows=-1), SHAPE), (dict(K=100), SHAPE),
    (dict(row_token=A, rows=1 << 31), SHAPE), (dict(row_token=A, rows=1 << 30, K=256), SHAPE), (dict(K=1 << 40), SHAPE),
    (dict(T=0, rows=0, q=None), OK), (dict(rows=0, qt=None), OK), (dict(K=0), OK), (dict(q=None), NULL), (dict(s=None), NULL),
    (dict(qt=None), NULL), (dict(et=None), NULL), (dict(q=MIS8), ALIGN), (dict(s=MIS), ALIGN), (dict(row_token=MIS), ALIGN),
    (dict(qt=MIS8), ALIGN), (dict(et=MIS8), ALIGN),
])
def test_transpose(lib, change, want):
    assert set(change) <= set(TRANS)
    assert lib.fp8q_transpose_act_128x1(*{**TRANS, **change}.values()) == want
    if "s" not in change and "q" not in change:
        c = {**TRANS, **change}
        assert lib.fp8q_quant_act_128x1(c["q"], max(c["K"], 0), c["T"], c["K"], c["row_token"], c["rows"], c["qt"], c["et"],
                                        None) == want


def test_weight_gradients_with_too_many_scale_bytes(lib):
    need = lib.fp8q_gemm_wgrad_workspace_bytes
    assert need(1 << 23, 16384, 16, 1) >= 0 and need(1 << 23, 16400, 16, 1) == -1 and need(1 << 23, 16, 16400, 1) == -1
    c = {**WG, "M": 1 << 23, "N": 16, "K": 16400}
    assert lib.fp8q_gemm_wgrad(*c.values()) == SHAPE
    assert lib.fp8q_grouped_gemm_wgrad(*{**GWG, "M": 1 << 23, "N": 16400, "K": 16}.values()) == SHAPE


def test_bf16_rows(lib):
    f = lib.fp8q_quant_act_128x1
    assert f(A, 255, 4, 256, None, 4, B, B, None) == SHAPE and f(A, 260, 4, 256, None, 4, B, B, None) == SHAPE
    assert f(None, 256, 4, 256, None, 4, B, B, None) == NULL and f(MIS8, 256, 4, 256, None, 4, B, B, None) == ALIGN


SWI = dict(q=A, s=A, gh=A, ldg=256, M=4, F=256, gq=B, gs=B, gqt=B, get=B, hqt=B, het=B, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(M=-1), SHAPE), (dict(F=100), SHAPE), (dict(F=-128), SHAPE), (dict(ldg=128), SHAPE), (dict(ldg=260), SHAPE),
    (dict(M=1 << 30), SHAPE), (dict(M=0, q=None), OK), (dict(F=0, q=None), OK), (dict(q=None), NULL), (dict(s=None), NULL),
    (dict(gh=None), NULL), (dict(gq=None), NULL), (dict(gs=None), NULL), (dict(gqt=None), NULL), (dict(get=None), NULL),
    (dict(hqt=None), NULL), (dict(het=None), NULL), (dict(q=MIS8), ALIGN), (dict(s=MIS), ALIGN), (dict(gh=MIS8), ALIGN),
    (dict(gq=MIS8), ALIGN), (dict(gs=MIS), ALIGN), (dict(gqt=MIS8), ALIGN), (dict(get=MIS8), ALIGN), (dict(hqt=MIS8), ALIGN),
    (dict(het=MIS8), ALIGN),
])
def test_swiglu(lib, change, want):
    assert set(change) <= set(SWI)
    assert lib.fp8q_swiglu_backward_quant(*{**SWI, **change}.values()) == want


WG = dict(gt=A, eg=A, xt=A, ex=A, dw=B, dtype=1, acc=0, M=256, N=64, K=80, ws=B, wsb=1 << 30, stream=None)
GWG = dict(gt=A, eg=A, xt=A, ex=A, dw=B, dtype=1, acc=0, off=A, E=3, M=256, N=64, K=80, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(M=-128), SHAPE), (dict(M=100), SHAPE), (dict(M=(1 << 23) + 128), SHAPE), (dict(N=-16), SHAPE), (dict(N=24), SHAPE),
    (dict(K=40), SHAPE), (dict(N=1 << 30, K=1 << 30), SHAPE), (dict(dtype=2), DTYPE), (dict(acc=2), OPTION), (dict(acc=-1), OPTION),
    (dict(N=0, gt=None), OK), (dict(K=0, gt=None), OK), (dict(M=0, acc=1, gt=None, dw=None), OK), (dict(dw=None), NULL),
    (dict(gt=None), NULL), (dict(eg=None), NULL), (dict(xt=None), NULL), (dict(ex=None), NULL), (dict(gt=MIS8), ALIGN),
    (dict(eg=MIS8), ALIGN), (dict(xt=MIS8), ALIGN), (dict(ex=MIS8), ALIGN), (dict(dw=MIS8), ALIGN),
])
def test_wgrad(lib, change, want):
    assert set(change) <= set(WG)
    assert lib.fp8q_gemm_wgrad(*{**WG, **change}.values()) == want
    assert lib.fp8q_grouped_gemm_wgrad(*{**GWG, **change}.values()) == want


def test_experts_wgrad(lib):
    f = lib.fp8q_grouped_gemm_wgrad
    for change, want in ((dict(E=0), SHAPE), (dict(E=1 << 31), SHAPE), (dict(off=None), NULL), (dict(off=MIS), ALIGN),
                         (dict(E=(1 << 31) - 1, N=4096, K=4096), SHAPE)):
        assert f(*{**GWG, **change}.values()) == want


def test_wgrad_workspace(lib):
    need = lib.fp8q_gemm_wgrad_workspace_bytes
    assert need(-128, 64, 64, 1) == -1 and need(100, 64, 64, 1) == -1 and need(128, 60, 64, 1) == -1 and need(128, 64, 64, 2) == -1
    assert need(0, 64, 64, 1) == 0 and need(128, 64, 64, 0) == 0
    for M, N, K in ((8192, 64, 64), (1 << 16, 256, 256), (4096, 576, 7168), (4096, 18432, 7168)):
        for code in (0, 1):
            n = need(M, N, K, code)
            assert n >= 0 and n % 16 == 0
            if n > 0:
                c = {**WG, "M": M, "N": N, "K": K, "dtype": code}
                assert lib.fp8q_gemm_wgrad(*{**c, "wsb": n - 1}.values()) == WORKSPACE
                assert lib.fp8q_gemm_wgrad(*{**c, "ws": None}.values()) == NULL
                assert lib.fp8q_gemm_wgrad(*{**c, "ws": MIS8}.values()) == ALIGN


def test_tensors_elsewhere_are_refused(monkeypatch):
    """The binding refuses tensors that are not on the current device (here: on none), before the library is called."""
    monkeypatch.setattr(_binding, "_GET_DEVICE", lambda: 0)
    monkeypatch.setattr(_binding, "load_library", lambda: pytest.fail("the library was called"))
    x, w, v = torch.zeros((4, 256), dtype=torch.bfloat16), torch.ones(256), torch.zeros(4)
    q, s = torch.zeros((4, 256), dtype=torch.uint8), torch.zeros((2, 4))
    t, e = torch.zeros((16, 128), dtype=torch.uint8), torch.zeros((1, 16), dtype=torch.uint8)
    for call in (lambda: fq.fp8q_rmsnorm_quant_act_1x128(x, w), lambda: fq.fp8q_rmsnorm_backward(x, x, w, v),
                 lambda: fq.fp8q_transpose_act_128x1(q, s), lambda: fq.fp8q_quant_act_128x1(x),
                 lambda: fq.fp8q_swiglu_backward_quant(q, s, x[:, :128]), lambda: fq.fp8q_gemm_wgrad(t, e, t, e),
                 lambda: fq.fp8q_grouped_gemm_wgrad(t, e, t, e, torch.zeros(3, dtype=torch.int32))):
        with pytest.raises(ValueError, match="device"):
            call()
