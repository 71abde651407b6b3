"""INT8 quantization and products.  Codes and scales equal the fp32 reference bit for bit; the products' sums are
exact integers, so every fp32 output equals fl32(sum) * fl32(sa * sw) bit for bit, and every bf16 output is that
value rounded to nearest even: no tolerance anywhere."""
import numpy as np
import pytest
import torch

import fine_grained_quantization_amd as fq
import moe_int8_reference as ref
from gpu_util import every_amax_groups, host, require_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def bf16(rng, shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).bfloat16()


@pytest.mark.parametrize("M,K", [(1, 16), (3, 48), (5, 2064), (64, 7168), (2, 8208), (3, 16384), (2, 18432), (1, 40000)])
def test_quantizer(M, K):
    rng = np.random.default_rng([31, M, K])
    x = bf16(rng, (M, K))
    x[0, K // 2] = 50.0
    if M > 2:
        x[2] = 0.0
    say(f"quant int8 {M}x{K}")
    q, s = fq.fp8q_quant_int8(x.cuda())
    eq, es = ref.quant_int8(x.float().numpy())
    assert np.array_equal(host(q), eq) and np.array_equal(host(s).view(np.uint32), es.view(np.uint32))


def test_quantizer_every_amax():
    """One row of 128 for every positive finite bf16 amax (denormals too: there the rounding of the scale lets a quotient
    reach 127.008, which is still code 127)."""
    bits = every_amax_groups(33).reshape(-1, 128)
    x = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16)
    say("quant int8 every amax")
    q, s = fq.fp8q_quant_int8(x.cuda())
    eq, es = ref.quant_int8(x.float().numpy())
    assert np.array_equal(host(s).view(np.uint32), es.view(np.uint32))
    assert np.array_equal(host(q), eq)


def test_quantizer_strided_rows_and_no_columns():
    rng = np.random.default_rng(34)
    wide = bf16(rng, (9, 400)).cuda()
    q, s = fq.fp8q_quant_int8(wide[:, 16:352])
    eq, es = ref.quant_int8(wide[:, 16:352].float().cpu().numpy())
    assert np.array_equal(host(q), eq) and np.array_equal(host(s), es)
    q, s = fq.fp8q_quant_int8(torch.empty((4, 0), dtype=torch.bfloat16, device="cuda"), s=torch.ones(4, device="cuda"))
    assert (host(s) == 0).all()


def operands(rng, M, N, K):
    qa = rng.integers(-127, 128, (M, K), dtype=np.int8)
    qw = rng.integers(-127, 128, (N, K), dtype=np.int8)
    return qa, (rng.random(M) * 0.01 + 1e-4).astype(np.float32), qw, (rng.random(N) * 0.01 + 1e-4).astype(np.float32)


def dev(*arrays):
    return [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in arrays]


def check_out(c, want, what):
    got = host(c)
    if c.dtype == torch.float32:
        assert np.array_equal(got.view(np.uint32), want.view(np.uint32)), what
    else:
        assert np.array_equal(got, ref.bf16_round(want)), what


DENSE = [(1, 8, 16), (1, 18432, 256), (2, 24, 48), (7, 136, 112), (15, 520, 128), (16, 2048, 144), (17, 1000, 1040),
         (33, 72, 7168), (63, 264, 256), (64, 128, 400), (65, 256, 272), (100, 4104, 528), (128, 640, 1024),
         (129, 136, 2064), (200, 384, 640), (255, 248, 384), (256, 512, 128), (257, 256, 176), (300, 776, 896),
         (513, 1032, 1168), (1037, 4104, 400), (2049, 264, 272), (3, 8, 131056),
         (520, 4104, 4112), (500, 16376, 912), (801, 8216, 400), (1800, 4104, 400), (600, 16392, 144), (1290, 13000, 272)]


@pytest.mark.parametrize("M,N,K", DENSE)
def test_dense(M, N, K):
    rng = np.random.default_rng([41, M, N, K])
    ops = operands(rng, M, N, K)
    want = ref.gemm_int8(*ops)
    for dt in (torch.bfloat16, torch.float32):
        say(f"int8 {M}x{N}x{K} {dt}")
        c = fq.fp8q_gemm_int8(*dev(*ops), out_dtype=dt)
        check_out(c, want, f"{M}x{N}x{K}")


@pytest.mark.parametrize("M", [1, 40, 150, 300])
def test_largest_sums(M):
    """Every code -128 or 127 at the longest K: sums up to 2^31 - 2^18 and down to -2^31 + ..."""
    K, N = 131056, 24
    qa = np.full((M, K), -128, np.int8)
    qw = np.full((N, K), -128, np.int8)
    qw[1::2] = 127
    sa, sw = np.full(M, 1.0, np.float32), np.full(N, 1.0, np.float32)
    say(f"int8 largest sums M={M}")
    c = fq.fp8q_gemm_int8(*dev(qa, sa, qw, sw), out_dtype=torch.float32)
    want = np.where(np.arange(N) % 2, -128.0 * 127 * K, 128.0 * 128 * K).astype(np.float32)
    assert (host(c) == want[None, :]).all()


def test_buffers_beside_the_operands_are_not_read_or_written():
    """Operands and result end inside larger buffers whose other bytes would change the result."""
    for M, N, K in ((3, 24, 48), (70, 136, 176), (300, 264, 144)):
        rng = np.random.default_rng([42, M])
        qa, sa, qw, sw = operands(rng, M, N, K)
        A = torch.full((M * K + 4096,), 127, dtype=torch.int8, device="cuda")
        W = torch.full((N * K + 4096,), 127, dtype=torch.int8, device="cuda")
        C = torch.full((M * N + 4096,), 7.0, device="cuda")
        A[:M * K] = torch.from_numpy(qa.reshape(-1)).cuda()
        W[:N * K] = torch.from_numpy(qw.reshape(-1)).cuda()
        say(f"int8 guard {M}x{N}x{K}")
        dsa, dsw = dev(sa, sw)
        fq.fp8q_gemm_int8(A[:M * K].view(M, K), dsa, W[:N * K].view(N, K), dsw, out_dtype=torch.float32,
                          c=C[:M * N].view(M, N))
        check_out(C[:M * N].view(M, N), ref.gemm_int8(qa, sa, qw, sw), "guard")
        assert (C[M * N:] == 7.0).all()


@pytest.mark.parametrize("M", [2, 100, 200, 300])
def test_weight_past_two_gigabytes(M):
    """N * K = 2.3e9 bytes; a sample of channels against the reference."""
    N, K = 17600, 131056
    g = torch.Generator(device="cuda")
    g.manual_seed(43)
    qw = torch.randint(-127, 128, (N, K), device="cuda", dtype=torch.int8, generator=g)
    qa = torch.randint(-127, 128, (M, K), device="cuda", dtype=torch.int8, generator=g)
    sa, sw = torch.rand(M, device="cuda", generator=g), torch.rand(N, device="cuda", generator=g)
    say(f"int8 weight past 2 GiB M={M}")
    c = fq.fp8q_gemm_int8(qa, sa, qw, sw, out_dtype=torch.float32)
    at = torch.tensor([0, 1, 8000, 16383, 16384, 16400, 17000, N - 1], device="cuda")
    m = torch.tensor([0, M // 2, M - 1], device="cuda")
    want = ref.gemm_int8(host(qa[m]), host(sa[m]), host(qw[at]), host(sw[at]))
    assert np.array_equal(host(c[m][:, at]), want)


def test_many_rows_and_outputs_past_two_gigabytes():
    M, N, K = 33000, 32768, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(44)
    qw = torch.randint(-127, 128, (N, K), device="cuda", dtype=torch.int8, generator=g)
    qa = torch.randint(-127, 128, (M, K), device="cuda", dtype=torch.int8, generator=g)
    sa, sw = torch.rand(M, device="cuda", generator=g), torch.rand(N, device="cuda", generator=g)
    say("int8 output past 2 GiB")
    c = fq.fp8q_gemm_int8(qa, sa, qw, sw, out_dtype=torch.float32)
    m = torch.tensor([0, 5, 16383, 16384, 32767, 32768, M - 1], device="cuda")
    want = ref.gemm_int8(host(qa[m]), host(sa[m]), host(qw), host(sw))
    assert np.array_equal(host(c[m]), want)


def grouped_problem(T, E, k, N, K, seed, empty=()):
    rng = np.random.default_rng([51, seed, T, E])
    keep = np.array([e for e in range(E) if e not in empty])
    idx = keep[np.argsort(rng.random((T, len(keep))), axis=1)[:, :k]].astype(np.int32)
    rows = fq.fp8q_moe_route_capacity(T, E, k)
    offsets, row_of, row_token, _ = ref.layout(idx, E, rows)
    q = rng.integers(-127, 128, (T, K), dtype=np.int8)
    s = (rng.random(T) * 0.01 + 1e-4).astype(np.float32)
    qw = rng.integers(-127, 128, (E, N, K), dtype=np.int8)
    sw = (rng.random((E, N)) * 0.01 + 1e-4).astype(np.float32)
    want = np.zeros((rows, N), np.float32)
    for e in range(E):
        r = np.arange(offsets[e], offsets[e + 1])
        r = r[row_token[r] >= 0]
        if len(r):
            want[r] = ref.gemm_int8(q[row_token[r]], s[row_token[r]], qw[e], sw[e])
    return offsets, row_token, q, s, qw, sw, want


GROUPED = [(1, 4, 2, 24, 48), (5, 8, 3, 136, 144), (20, 6, 2, 264, 400), (90, 5, 4, 128, 256), (64, 40, 8, 72, 272),
           (200, 2, 1, 520, 176), (700, 3, 2, 256, 1040), (33, 300, 2, 8, 16), (513, 2, 2, 1032, 128), (16, 4, 4, 2048, 528),
           (3000, 5, 2, 2056, 272)]


@pytest.mark.parametrize("T,E,k,N,K", GROUPED)
def test_grouped_and_gather(T, E, k, N, K):
    empty = (1,) if E > k + 1 else ()
    offsets, row_token, q, s, qw, sw, want = grouped_problem(T, E, k, N, K, 1, empty)
    rows, used = len(row_token), offsets[-1]
    pad = row_token[:, None] < 0
    qa = np.where(pad, 0, q[row_token]).astype(np.int8)
    sa = np.where(pad[:, 0], 0, s[row_token]).astype(np.float32)
    for dt in (torch.bfloat16, torch.float32):
        for gather in (False, True):
            c = torch.full((rows, N), 77.0, dtype=dt, device="cuda")
            say(f"int8 grouped T={T} E={E} k={k} N={N} K={K} {dt} gather={gather}")
            if gather:
                fq.fp8q_grouped_gemm_int8_gather(*dev(q, s, row_token, qw, sw, offsets), out_dtype=dt, c=c)
            else:
                fq.fp8q_grouped_gemm_int8(*dev(qa, sa, qw, sw, offsets), out_dtype=dt, c=c)
            check_out(c[:used], want[:used], "grouped")
            assert (c[used:] == 77.0).all()  # rows from offsets[E] on are not written


def call_time(f, n=10):
    """Median over 7 loops of n calls."""
    times = []
    for _ in range(8):
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        for _ in range(n):
            f()
        end.record()
        torch.cuda.synchronize()
        times.append(begin.elapsed_time(end))
    return sorted(times[1:])[3]


@pytest.mark.parametrize("T,E,N,K", [(1, 64, 2048, 7168), (16, 64, 2048, 7168), (4, 64, 7168, 2048)])
def test_rows_in_place_read_the_weights_about_once(T, E, N, K):
    """A decode batch's product with rows in place takes at most 2.5 times as long as the form that reads the tokens through
    the layout (it has the padding to multiply too, but not the weights to read for every few rows of it)."""
    offsets, row_token, q, s, qw, sw, _ = (dev(a)[0] for a in grouped_layout(T, E, 8, N, K))
    rows, pad = row_token.numel(), row_token[:, None] < 0
    qa = torch.where(pad, 0, q[row_token.clamp(min=0).long()])
    sa = torch.where(pad[:, 0], 0.0, s[row_token.clamp(min=0).long()])
    c = torch.zeros((rows, N), dtype=torch.bfloat16, device="cuda")
    say(f"int8 grouped, rows in place and gathered, T={T} E={E} N={N} K={K}")
    place = call_time(lambda: fq.fp8q_grouped_gemm_int8(qa, sa, qw, sw, offsets, c=c))
    gather = call_time(lambda: fq.fp8q_grouped_gemm_int8_gather(q, s, row_token, qw, sw, offsets, c=c))
    assert place < 2.5 * gather


def test_gathered_full_segments_read_the_weights_about_once():
    """A layout cut to the rows in use, every one with a token: the gathered product is the one with rows in place, bit for
    bit, and takes at most 2.5 times as long."""
    E, N, K, T = 64, 2048, 2064, 1024
    g = torch.Generator(device="cuda").manual_seed(46)
    row_token = torch.cat([torch.randperm(T, device="cuda", generator=g)[:128] for _ in range(E)]).int()
    off = torch.arange(E + 1, dtype=torch.int32, device="cuda") * 128
    q = torch.randint(-127, 128, (T, K), device="cuda", dtype=torch.int8, generator=g)
    qw = torch.randint(-127, 128, (E, N, K), device="cuda", dtype=torch.int8, generator=g)
    s, sw = torch.rand(T, device="cuda", generator=g), torch.rand((E, N), device="cuda", generator=g)
    qa, sa = q[row_token.long()], s[row_token.long()]
    say("int8 gather, full segments")
    a = fq.fp8q_grouped_gemm_int8(qa, sa, qw, sw, off)
    b = fq.fp8q_grouped_gemm_int8_gather(q, s, row_token, qw, sw, off)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    place = call_time(lambda: fq.fp8q_grouped_gemm_int8(qa, sa, qw, sw, off, c=a))
    gather = call_time(lambda: fq.fp8q_grouped_gemm_int8_gather(q, s, row_token, qw, sw, off, c=b))
    assert gather < 2.5 * place


def grouped_layout(T, E, k, N, K):
    """Layout, tokens and weights without the expected result (sizes at which the host would take long)."""
    rng = np.random.default_rng([55, T, E])
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    offsets, row_of, row_token, _ = ref.layout(idx, E, fq.fp8q_moe_route_capacity(T, E, k))
    return (offsets, row_token, rng.integers(-127, 128, (T, K), dtype=np.int8), rng.random(T).astype(np.float32),
            rng.integers(-127, 128, (E, N, K), dtype=np.int8), rng.random((E, N)).astype(np.float32), row_of)


def test_grouped_offsets_that_break_the_rules():
    """Offsets off the 128-row grid, starting past 0 and ending past the buffer are cut to it."""
    E, N, K, M = 3, 40, 64, 256
    rng = np.random.default_rng(52)
    qa, sa, _, _ = operands(rng, M, 8, K)
    qw = rng.integers(-127, 128, (E, N, K), dtype=np.int8)
    sw = rng.random((E, N)).astype(np.float32)
    off = np.array([10, 77, 200, 5000], np.int32)
    c = torch.full((M, N), 77.0, device="cuda")
    say("int8 grouped odd offsets")
    fq.fp8q_grouped_gemm_int8(*dev(qa, sa, qw, sw, off), out_dtype=torch.float32, c=c)
    want = np.full((M, N), 77.0, np.float32)
    for e, (a, b) in enumerate(((10, 77), (77, 200), (200, 256))):
        want[a:b] = ref.gemm_int8(qa[a:b], sa[a:b], qw[e], sw[e])
    assert np.array_equal(host(c), want)


def test_gather_tokens_out_of_range_are_empty_rows():
    E, N, K, T = 2, 24, 32, 5
    rng = np.random.default_rng(53)
    q, s, _, _ = operands(rng, T, 8, K)
    qw = rng.integers(-127, 128, (E, N, K), dtype=np.int8)
    sw = rng.random((E, N)).astype(np.float32)
    row_token = np.full(256, -1, np.int32)
    row_token[[0, 1, 2, 3, 130, 131]] = [4, 5, -7, 2 ** 31 - 1, 0, 3]
    off = np.array([0, 128, 256], np.int32)
    say("int8 gather out of range")
    c = fq.fp8q_grouped_gemm_int8_gather(*dev(q, s, row_token, qw, sw, off), out_dtype=torch.float32)
    want = np.zeros((256, N), np.float32)
    for r, e in ((0, 0), (130, 1), (131, 1)):
        want[r] = ref.gemm_int8(q[row_token[r]][None], s[row_token[r]][None], qw[e], sw[e])[0]
    assert np.array_equal(host(c), want)
    c.fill_(7.0)
    fq.fp8q_grouped_gemm_int8_gather(torch.empty((0, K), dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda"),
                                     *dev(row_token, qw, sw, off), out_dtype=torch.float32, c=c)  # no tokens at all
    assert (host(c) == 0).all()


@pytest.mark.parametrize("T,E,rows,N,K", [(6, 16, 2048, 264, 144), (60, 2, 512, 264, 144), (1600, 2, 4096, 4104, 272)])
def test_gathered_rows_of_no_token_are_zero_whatever_the_scales(T, E, rows, N, K):
    """+0 beside tokens in the same tile too, by the kernel of few rows, the small tiles and the large ones; channel
    scales negative, infinite and NaN."""
    rng = np.random.default_rng([54, T])
    q, s, _, _ = operands(rng, T, 8, K)
    qw = rng.integers(-127, 128, (E, N, K), dtype=np.int8)
    sw = rng.standard_normal((E, N)).astype(np.float32)
    sw[:, ::5], sw[:, 1::7], sw[:, 2::9] = np.inf, -np.inf, np.nan
    row_token = np.where(rng.random(rows) < 0.5, rng.integers(0, T, rows), -1).astype(np.int32)
    row_token[rows // 2:rows // 2 + 20] = -1
    off = (np.arange(E + 1) * (rows // E)).astype(np.int32)
    for dt in (torch.bfloat16, torch.float32):
        say(f"int8 gather, empty rows beside tokens T={T} rows={rows} {dt}")
        c = fq.fp8q_grouped_gemm_int8_gather(*dev(q, s, row_token, qw, sw, off), out_dtype=dt)
        bits = host(c.view(torch.int16 if dt == torch.bfloat16 else torch.int32))
        assert (bits[row_token < 0] == 0).all()
        fine = np.isfinite(sw[0])
        r = np.nonzero(row_token[:rows // E] >= 0)[0]
        want = ref.gemm_int8(q[row_token[r]], s[row_token[r]], qw[0][fine], sw[0][fine])
        check_out(c[:rows // E][torch.from_numpy(r).cuda()][:, torch.from_numpy(fine).cuda()].contiguous(), want, "tokens")


@pytest.mark.parametrize("used", [3, 300])
def test_gather_from_the_largest_token_array(used):
    """T * K = 2^31 - 2048, the last tokens among the rows, by the kernel of few rows and by the tiles."""
    T, K, N, E = 131200, 16368, 24, 1
    g = torch.Generator(device="cuda")
    g.manual_seed(45)
    q = torch.randint(-127, 128, (T, K), device="cuda", dtype=torch.int8, generator=g)
    s, sw = torch.rand(T, device="cuda", generator=g), torch.rand((E, N), device="cuda", generator=g)
    qw = torch.randint(-127, 128, (E, N, K), device="cuda", dtype=torch.int8, generator=g)
    rows = (used + 127) // 128 * 128
    row_token = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    row_token[:used] = T - 1 - torch.arange(used, device="cuda") * 400
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    say(f"int8 gather at T * K = {T * K}, {used} rows")
    c = fq.fp8q_grouped_gemm_int8_gather(q, s, row_token, qw, sw, off, out_dtype=torch.float32)
    at = row_token[:used].long()
    want = ref.gemm_int8(host(q[at]), host(s[at]), host(qw[0]), host(sw[0]))
    assert np.array_equal(host(c[:used]), want) and (host(c[used:]) == 0).all()


def test_gather_of_few_rows_from_the_largest_token_array():
    """The same by the kernel of few rows, which more experts than half the tokens make the choice: 8200 experts, three of
    them with tokens, T * K = 2^31 - 131088, K at its largest."""
    T, K, N, E = 16385, 131056, 8, 8200
    g = torch.Generator(device="cuda")
    g.manual_seed(47)
    q = torch.randint(-127, 128, (T, K), device="cuda", dtype=torch.int8, generator=g)
    s, sw = torch.rand(T, device="cuda", generator=g), torch.rand((E, N), device="cuda", generator=g)
    qw = torch.randint(-127, 128, (E, N, K), device="cuda", dtype=torch.int8, generator=g)  # 8.6 GB
    row_token = torch.full((384,), -1, dtype=torch.int32, device="cuda")
    used = {0: (0, [T - 1, 0, 8192]), 4321: (128, [T - 2] * 17), E - 1: (256, [12345, T - 1])}
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    for e, (r, tokens) in used.items():
        row_token[r:r + len(tokens)] = torch.tensor(tokens, dtype=torch.int32, device="cuda")
        off[e + 1:] = r + 128
    say(f"int8 gather of few rows at T * K = {T * K}")
    c = fq.fp8q_grouped_gemm_int8_gather(q, s, row_token, qw, sw, off, out_dtype=torch.float32)
    for e, (r, tokens) in used.items():
        want = ref.gemm_int8(host(q[tokens]), host(s[tokens]), host(qw[e]), host(sw[e]))
        assert np.array_equal(host(c[r:r + len(tokens)]), want)
    assert (host(c)[host(row_token) < 0] == 0).all()


def test_int8_wants_its_arguments_right():
    a = torch.zeros((4, 32), dtype=torch.int8, device="cuda")
    w = torch.zeros((16, 32), dtype=torch.int8, device="cuda")
    sa, sw = torch.zeros(4, device="cuda"), torch.zeros(16, device="cuda")
    x = torch.zeros((4, 32), dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(2, dtype=torch.int32, device="cuda")
    bad = [lambda: fq.fp8q_gemm_int8(a.view(torch.uint8), sa, w, sw), lambda: fq.fp8q_gemm_int8(a, sa[:3], w, sw),
           lambda: fq.fp8q_gemm_int8(a, sa, w[:12], sw[:12]), lambda: fq.fp8q_gemm_int8(a[:, :24].contiguous(), sa, w, sw),
           lambda: fq.fp8q_gemm_int8(a[:, :24].contiguous(), sa, w[:, :24].contiguous(), sw),
           lambda: fq.fp8q_gemm_int8(a, sa, w, sw, out_dtype=torch.float16), lambda: fq.fp8q_gemm_int8(a.t(), sa, w, sw),
           lambda: fq.fp8q_gemm_int8(a, sa, w.view(-1)[8:264].view(8, 32), sw[:8]),
           lambda: fq.fp8q_quant_int8(x.float()), lambda: fq.fp8q_quant_int8(x[:, :24].contiguous()),
           lambda: fq.fp8q_quant_int8(x[:, 1:17]), lambda: fq.fp8q_quant_int8(x.t()),
           lambda: fq.fp8q_grouped_gemm_int8(a, sa, w.view(1, 16, 32), sw, off),  # 4 rows: not a multiple of 128
           lambda: fq.fp8q_grouped_gemm_int8(a, sa, w, sw, off),
           lambda: fq.fp8q_grouped_gemm_int8_gather(a, sa, off, w.view(1, 16, 32), sw, off[:1])]
    for f in bad:
        with pytest.raises((ValueError, RuntimeError, TypeError)):
            f()
