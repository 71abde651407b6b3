"""The gating, combination and INT8 entry points refuse bad arguments before touching a device (CPU-only; the
addresses are never dereferenced: every call fails validation, or has nothing to do)."""
import ctypes
import os

import pytest

import fine_grained_quantization_amd as fq

A, B, MIS = ctypes.c_void_p(4096), ctypes.c_void_p(8192), ctypes.c_void_p(4098)
OK, NULL, SHAPE, ALIGN, DTYPE, WORKSPACE, OPTION = 0, -1, -2, -3, -4, -8, -9


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fq.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return fq.load_library()


GATE = dict(logits=A, dtype=1, ld=64, T=40, E=64, k=4, score=0, bias=None, n_group=8, topk_group=4, group_top=2,
            renorm=1, scale=1.0, idx=A, weight=A, off=A, row_of=A, row_token=A, rows=1 << 20, load=None, ws=A,
            wsb=1 << 20, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(T=-1), SHAPE), (dict(E=0), SHAPE), (dict(E=1025, ld=1025), SHAPE), (dict(k=0), SHAPE), (dict(k=17), SHAPE),
    (dict(ld=63), SHAPE), (dict(rows=100), SHAPE), (dict(rows=1 << 31), SHAPE), (dict(n_group=0), SHAPE),
    (dict(n_group=7), SHAPE), (dict(n_group=65), SHAPE), (dict(topk_group=0), SHAPE), (dict(topk_group=9), SHAPE),
    (dict(k=16, topk_group=1), SHAPE), (dict(T=1 << 31, rows=(1 << 31) - 1), SHAPE),
    (dict(T=1 << 26, rows=(1 << 31) - 1), SHAPE), (dict(dtype=2), DTYPE),
    (dict(score=2), OPTION), (dict(group_top=0), OPTION), (dict(group_top=3), OPTION), (dict(renorm=2), OPTION),
    (dict(off=None), NULL), (dict(row_token=None), NULL), (dict(logits=None), NULL), (dict(idx=None), NULL),
    (dict(weight=None), NULL), (dict(row_of=None), NULL), (dict(ws=None), NULL), (dict(logits=MIS), ALIGN),
    (dict(bias=MIS), ALIGN), (dict(load=MIS), ALIGN), (dict(ws=MIS), ALIGN), (dict(weight=MIS), ALIGN),
    (dict(dtype=0, logits=ctypes.c_void_p(4097)), ALIGN), (dict(wsb=127), WORKSPACE), (dict(wsb=-1), WORKSPACE),
])
def test_gate(lib, change, want):
    assert set(change) <= set(GATE)
    assert lib.fp8q_moe_gate_topk(*{**GATE, **change}.values()) == want


def test_gate_workspace(lib):
    need = lib.fp8q_moe_gate_workspace_bytes
    assert need(0, 5) == 0 and need(32, 256) == 0 and need(33, 256) == 768 and need(65, 5) == 24 and need(4097, 8) == 129 * 8
    assert need(-1, 5) == -1 and need(5, 0) == -1 and need(5, 1025) == -1


@pytest.mark.parametrize("E", [1, 5, 8, 64, 255, 256, 1024])
def test_gate_refuses_only_less_than_the_counts_of_32_token_chunks(lib, E):
    for T in (33, 64, 65, 3009, 4096, 4097, 6000):
        least = (T + 31) // 32 * ((E + 3) // 4 * 4)
        assert least <= lib.fp8q_moe_gate_workspace_bytes(T, E)
        change = dict(T=T, E=E, ld=E, k=1, n_group=1, topk_group=1)
        assert lib.fp8q_moe_gate_topk(*{**GATE, **change, "wsb": least - 1}.values()) == WORKSPACE
    needs = [lib.fp8q_moe_gate_workspace_bytes(T, E) for T in range(1, 9000)]
    assert all((t + 31) // 32 * ((E + 3) // 4 * 4) <= min(needs[t - 1:]) for t in range(33, 9000))


BACK = dict(logits=A, dtype=1, ld=64, T=4, E=64, k=4, score=0, renorm=1, scale=1.0, idx=A, gw=A, out=B, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(T=-1), SHAPE), (dict(E=0), SHAPE), (dict(k=65), SHAPE), (dict(k=17), SHAPE), (dict(ld=63), SHAPE),
    (dict(T=1 << 26), SHAPE),
    (dict(dtype=-1), DTYPE), (dict(score=-1), OPTION), (dict(renorm=-1), OPTION), (dict(T=0, logits=None), OK),
    (dict(logits=None), NULL), (dict(idx=None), NULL), (dict(gw=None), NULL), (dict(out=None), NULL),
    (dict(out=MIS), ALIGN), (dict(gw=MIS), ALIGN),
])
def test_gate_backward(lib, change, want):
    assert lib.fp8q_moe_gate_backward(*{**BACK, **change}.values()) == want


COMB = dict(c=A, dtype=0, rows=128, H=16, row_of=A, w=A, T=3, k=2, add=None, y=B, stream=None)
CBACK = dict(gy=A, c=A, dtype=0, rows=128, H=16, row_of=A, w=A, T=3, k=2, row_token=A, off=A, E=2, gc=B, gw=B,
             stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(T=-1), SHAPE), (dict(H=12), SHAPE), (dict(H=-8), SHAPE), (dict(rows=-1), SHAPE), (dict(k=0), SHAPE),
    (dict(k=17), SHAPE), (dict(T=1 << 31), SHAPE), (dict(T=(1 << 31) - 1, H=4096), SHAPE), (dict(T=1 << 24), SHAPE),
    (dict(dtype=3), DTYPE),
    (dict(T=0, c=None), OK), (dict(H=0, c=None), OK), (dict(c=None), NULL), (dict(row_of=None), NULL),
    (dict(w=None), NULL), (dict(y=None), NULL), (dict(c=ctypes.c_void_p(4104)), ALIGN), (dict(add=MIS), ALIGN),
    (dict(y=MIS), ALIGN), (dict(w=MIS), ALIGN),
])
def test_combine(lib, change, want):
    assert lib.fp8q_moe_combine(*{**COMB, **change}.values()) == want


@pytest.mark.parametrize("change,want", [
    (dict(T=-1), SHAPE), (dict(H=12), SHAPE), (dict(E=0), SHAPE), (dict(k=17), SHAPE), (dict(dtype=3), DTYPE),
    (dict(T=1 << 24), SHAPE), (dict(T=0, rows=0), OK), (dict(gy=None), NULL), (dict(c=None), NULL), (dict(gw=None), NULL), (dict(gc=None), NULL),
    (dict(row_token=None), NULL), (dict(off=None), NULL), (dict(gc=MIS), ALIGN), (dict(off=MIS), ALIGN),
])
def test_combine_backward(lib, change, want):
    assert lib.fp8q_moe_combine_backward(*{**CBACK, **change}.values()) == want


def test_int8(lib):
    q = lib.fp8q_quant_int8
    assert q(A, 32, 4, 24, B, B, None) == SHAPE and q(A, 31, 4, 32, B, B, None) == SHAPE
    assert q(A, 36, 4, 32, B, B, None) == SHAPE and q(A, 32, -1, 32, B, B, None) == SHAPE
    assert q(None, 32, 0, 32, None, None, None) == OK and q(None, 32, 4, 32, B, B, None) == NULL
    assert q(A, 0, 4, 0, None, None, None) == NULL and q(MIS, 32, 4, 32, B, B, None) == ALIGN
    assert q(A, 32, 4, 32, B, MIS, None) == ALIGN and q(A, 32, 1 << 24, 32, B, B, None) == SHAPE
    g = lib.fp8q_gemm_int8
    assert g(A, A, A, A, B, 0, 4, 12, 32, None) == SHAPE and g(A, A, A, A, B, 0, 4, 8, 24, None) == SHAPE
    assert g(A, A, A, A, B, 0, 4, 8, 0, None) == SHAPE and g(A, A, A, A, B, 0, 4, 8, 131072, None) == SHAPE
    assert g(A, A, A, A, B, 0, -1, 8, 32, None) == SHAPE and g(A, A, A, A, B, 2, 4, 8, 32, None) == DTYPE
    assert g(A, A, A, A, B, 0, 1 << 40, 1 << 20, 32, None) == SHAPE
    assert g(None, None, None, None, None, 0, 0, 8, 32, None) == OK
    assert g(A, None, A, A, B, 0, 4, 8, 32, None) == NULL and g(A, A, A, A, MIS, 0, 4, 8, 32, None) == ALIGN
    assert g(A, MIS, A, A, B, 0, 4, 8, 32, None) == ALIGN
    gg = lib.fp8q_grouped_gemm_int8
    assert gg(A, A, A, A, B, 0, A, 0, 128, 8, 32, None) == SHAPE and gg(A, A, A, A, B, 0, A, 2, 100, 8, 32, None) == SHAPE
    assert gg(A, A, A, A, B, 0, A, 2, 0, 8, 32, None) == OK and gg(A, A, A, A, B, 0, None, 2, 128, 8, 32, None) == NULL
    assert gg(A, A, A, A, B, 0, MIS, 2, 128, 8, 32, None) == ALIGN
    ga = lib.fp8q_grouped_gemm_int8_gather
    assert ga(A, A, -1, A, A, A, B, 0, A, 2, 128, 8, 32, None) == SHAPE
    assert ga(A, A, 1 << 26, A, A, A, B, 0, A, 2, 128, 8, 32, None) == SHAPE  # T * K = 2^31
    assert ga(A, A, 4, None, A, A, B, 0, A, 2, 128, 8, 32, None) == NULL
    assert ga(None, None, 4, A, A, A, B, 0, A, 2, 128, 8, 32, None) == NULL
    assert ga(A, A, 4, A, A, A, B, 9, A, 2, 128, 8, 32, None) == DTYPE
    assert lib.fp8q_status_string(OPTION).startswith(b"FP8Q_ERR_OPTION")
