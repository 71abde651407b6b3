// The backward pass's operands from 8-bit checkpoints: transposed copies in groups of 128 tokens of one channel, whose scales
// are powers of two (an E8M0 byte each), and SwiGLU's gradient recomputed from its 8-bit inputs.
//   transposed copy:  v[m][k] = fl32(code * s) (or bf16),  e[mb][k] = least e with max_{m in mb} |v| <= 448 * 2^e,
//                     qt[k][m] = E4M3(v 2^-e), exact but for E4M3's rounding; columns past the last token hold zeros.
// (Where the checkpoint's own scales are powers of two, no code changes unless it leaves E4M3's range below.)
//   SwiGLU:  p = 1 / (1 + exp(-x)),  h = x p u,  du = g x p,  dx = g u (p + x p (1 - p)).
// Every kernel takes tiles of 128 tokens x 128 channels: one read and one write of everything, bound by memory.
#include "fp8q_device.h"
#include "fp8q_kernels.h"

namespace fp8q {
namespace {

constexpr int kThreads = 512;

typedef float f32x2 __attribute__((ext_vector_type(2)));

// 8 codes to fp32 values times s.
__device__ __forceinline__ void decode8(const uint2 &d, float s, float *v) {
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)d.x, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)d.x, true);
    const f32x2 c = __builtin_amdgcn_cvt_pk_f32_fp8((int)d.y, false), e = __builtin_amdgcn_cvt_pk_f32_fp8((int)d.y, true);
    v[0] = a[0] * s; v[1] = a[1] * s; v[2] = b[0] * s; v[3] = b[1] * s;
    v[4] = c[0] * s; v[5] = c[1] * s; v[6] = e[0] * s; v[7] = e[1] * s;
}

__device__ __forceinline__ void widen8(const u32x4 &d, float *v) {
    v[0] = bf16_lo(d.x); v[1] = bf16_hi(d.x); v[2] = bf16_lo(d.y); v[3] = bf16_hi(d.y);
    v[4] = bf16_lo(d.z); v[5] = bf16_hi(d.z); v[6] = bf16_lo(d.w); v[7] = bf16_hi(d.w);
}

// The scale bytes of 8 channels are maxima of the bytes of their values (pow2_byte grows with its argument), two to a dword; until
// the last maximum they are 8 more than the bytes, and not yet cut off below.
typedef u16x2 Bytes8[4];

template <int R>
__device__ __forceinline__ void column_bytes(const float (&v)[R][8], Bytes8 &e) {
    uint32_t t[8];
#pragma unroll
    for (int c = 0; c < 8; c++) {
        float a = __builtin_fabsf(v[0][c]);
#pragma unroll
        for (int j = 1; j < R; j++) a = __builtin_fmaxf(a, __builtin_fabsf(v[j][c]));
        t[c] = (__float_as_uint(a) + kPow2Round) >> 23;
    }
#pragma unroll
    for (int d = 0; d < 4; d++) e[d] = __builtin_bit_cast(u16x2, t[2 * d] | t[2 * d + 1] << 16);
}

// Maxima over the lanes whose numbers differ in bits [log2 FROM, 6).
template <int FROM>
__device__ __forceinline__ void lanes_max(Bytes8 &e) {
#pragma unroll
    for (int o = FROM; o < 64; o <<= 1)
#pragma unroll
        for (int d = 0; d < 4; d++)
            e[d] = __builtin_elementwise_max(e[d], __builtin_bit_cast(u16x2, __shfl_xor(__builtin_bit_cast(int, e[d]), o, 64)));
}

__device__ __forceinline__ u32x4 as_dwords(const Bytes8 &e) {
    return (u32x4){__builtin_bit_cast(uint32_t, e[0]), __builtin_bit_cast(uint32_t, e[1]), __builtin_bit_cast(uint32_t, e[2]),
                   __builtin_bit_cast(uint32_t, e[3])};
}

// The channels' bytes of all 8 waves' tokens.
template <int CHUNKS>
__device__ __forceinline__ void waves_max(const u32x4 (&all)[8][CHUNKS], int chunk, Bytes8 &e) {
#pragma unroll
    for (int d = 0; d < 4; d++) e[d] = (u16x2){0, 0};
#pragma unroll
    for (int w = 0; w < 8; w++) {
        const u32x4 o = all[w][chunk];
#pragma unroll
        for (int d = 0; d < 4; d++) {
            const uint32_t x = o[d];  // (a bit cast of a vector's element would be one of its first)
            e[d] = __builtin_elementwise_max(e[d], __builtin_bit_cast(u16x2, x));
        }
    }
#pragma unroll
    for (int d = 0; d < 4; d++) e[d] = __builtin_elementwise_max(e[d], (u16x2){8, 8}) - (u16x2){8, 8};
}

__device__ __forceinline__ uint2 packed_bytes(const Bytes8 &e) {
    return (uint2){(uint32_t)e[0].x | (uint32_t)e[0].y << 8 | (uint32_t)e[1].x << 16 | (uint32_t)e[1].y << 24,
                   (uint32_t)e[2].x | (uint32_t)e[2].y << 8 | (uint32_t)e[3].x << 16 | (uint32_t)e[3].y << 24};
}

// 4 codes of values times 2^-e, e a scale byte; the conversion applies the power.
__device__ __forceinline__ uint32_t encode4_pow2(float a, float b, float c, float d, uint32_t byte) {
    typedef short s16x2 __attribute__((ext_vector_type(2)));
    const float p = pow2_value(byte);
    s16x2 r = {0, 0};
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, a, b, p, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, c, d, p, true);
    return __builtin_bit_cast(uint32_t, r);
}

// Streaming store: the copies are larger than any cache where their time matters.
__device__ __forceinline__ void store_stream16(void *p, const u32x4 &v) {
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4 *>(p));
}

// A tile of transposed codes: a row of 128 bytes a channel, 8 pieces of 16 bytes; piece p of channel c sits at p ^ ((c / 8) & 7),
// which spreads one store instruction's writes (channels 8 apart) over the banks.
template <int CHANNELS>
__device__ __forceinline__ void column_store(const uint32_t (&tile)[CHANNELS * 32], uint8_t *qt, int64_t ld, int t) {
#pragma unroll
    for (int i = 0; i < CHANNELS * 8 / kThreads; i++) {
        const int p = t + i * kThreads, row = p >> 3, piece = p & 7;
        store_stream16(qt + row * ld + piece * 16,
                       *reinterpret_cast<const u32x4 *>(&tile[row * 32 + ((piece ^ ((row >> 3) & 7)) << 2)]));
    }
}

struct TransposeArgs {
    const void *x;
    const float *s;
    int64_t ld, T, K, rows, cols;  // cols: rows rounded up to 128
    const int32_t *row_token;
    uint8_t *qt, *et;
};

// A workgroup takes 128 tokens x 256 channels (the last may have 128): a thread 8 tokens x 8 channels, 64 values in registers
// between the maxima and the codes, which go through LDS to leave as rows of 128 bytes.  8192 x 7168: 22 us from codes (5.35
// TB/s), 28 from bf16 (6.3).  Routed to 64 experts (73,000 rows of 7168): 124-143 us for 523 MB written (with a branch around
// each load 149-160); 470 vector instructions a wave keep the SIMDs busy for 0.86 of that.
template <bool CODES, bool ROUTED>
__global__ __launch_bounds__(kThreads) void transpose_kernel(TransposeArgs p) {
    __shared__ __align__(16) uint32_t tile[256 * 32];
    __shared__ u32x4 all[8][32];
    const int t = threadIdx.x, lane = t & 63, chunk = t & 31, g = t >> 5;
    // Rows in place: neighbours share rows.  Routed rows: each XCD (workgroups b with the same b % 8) takes an eighth of all
    // tiles, channels by channels, so that a token's 256 channels come from its L2 after the first of the token's rows.
    const uint32_t KQ = (uint32_t)((p.K + 255) >> 8), MB = (uint32_t)(p.cols >> 7), tiles = KQ * MB;  // (fewer than 2^23)
    uint32_t kq, mb32;
    if constexpr (!ROUTED) {
        if (blockIdx.x >= tiles) return;
        kq = blockIdx.x % KQ;
        mb32 = blockIdx.x / KQ;
    } else {
        const uint32_t i = (blockIdx.x % 8) * ((tiles + 7) / 8) + blockIdx.x / 8;
        if (i >= tiles) return;
        kq = i / MB;
        mb32 = i % MB;
    }
    const int64_t k0 = kq * 256, mb = mb32;
    const bool in = k0 + chunk * 8 < p.K;
    const int c0 = (in ? chunk : chunk & 15) * 8;
    // Rows without a token, and channels past the last, read token 0 and are made zeros: no branch stands between the loads.
    int tok[8];
    const int64_t m0 = mb * 128 + g * 8;
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const bool there = m0 + j < p.rows;
        tok[j] = ROUTED ? p.row_token[there ? m0 + j : 0] : (int)(m0 + j);
        if (!(there && in && (uint32_t)tok[j] < (uint32_t)p.T)) tok[j] = -1;
    }
    float v[8][8];
    if constexpr (CODES) {
        const uint8_t *x = static_cast<const uint8_t *>(p.x) + k0 + c0;
        const float *s = p.s + (k0 / 128 + (c0 >> 7)) * p.T;
        uint2 d[8];
        float sc[8];
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const uint32_t r = max(tok[j], 0);
            d[j] = *reinterpret_cast<const uint2 *>(x + r * (uint64_t)(uint32_t)p.K);
            sc[j] = s[r];
        }
#pragma unroll
        for (int j = 0; j < 8; j++) {
            if (tok[j] < 0) d[j] = (uint2){0u, 0u};
            if (tok[j] < 0) sc[j] = 0.0f;
            decode8(d[j], sc[j], v[j]);
        }
    } else {
        const uint16_t *x = static_cast<const uint16_t *>(p.x) + k0 + c0;
        u32x4 d[8];
#pragma unroll
        for (int j = 0; j < 8; j++) d[j] = *reinterpret_cast<const u32x4 *>(x + (int64_t)max(tok[j], 0) * p.ld);
#pragma unroll
        for (int j = 0; j < 8; j++) {
            if (tok[j] < 0) d[j] = (u32x4){0u, 0u, 0u, 0u};
            widen8(d[j], v[j]);
        }
    }
    Bytes8 e;
    column_bytes(v, e);
    lanes_max<32>(e);
    if (lane < 32) all[t >> 6][chunk] = as_dwords(e);
    __syncthreads();
    waves_max(all, chunk, e);
    if (t < 32 && in) *reinterpret_cast<uint2 *>(p.et + mb * p.K + k0 + chunk * 8) = packed_bytes(e);
#pragma unroll
    for (int c = 0; c < 8; c++) {
        const uint32_t byte = e[c / 2][c % 2];
        const uint2 w = {encode4_pow2(v[0][c], v[1][c], v[2][c], v[3][c], byte),
                         encode4_pow2(v[4][c], v[5][c], v[6][c], v[7][c], byte)};
        *reinterpret_cast<uint2 *>(&tile[(chunk * 8 + c) * 32 + (((g >> 1) ^ (chunk & 7)) << 2) + (g & 1) * 2]) = w;
    }
    __syncthreads();
    uint8_t *qt = p.qt + k0 * p.cols + mb * 128;
    if (k0 + 256 <= p.K) {
        column_store<256>(tile, qt, p.cols, t);
    } else {
        column_store<128>(reinterpret_cast<const uint32_t(&)[128 * 32]>(tile), qt, p.cols, t);
    }
}

struct SwigluArgs {
    const uint8_t *q;
    const float *s;
    const uint16_t *gh;
    int64_t ldg, M, F, cols;
    uint8_t *gq;
    float *gs;
    uint8_t *gqt, *get, *hqt, *het;
};

// 1 / (1 + e^-x): the hardware's exponential (an ulp, and |x| / 2 for its argument) and its reciprocal with a Newton step.  Up
// to 2^126 the sum has a reciprocal that is a normal number; it is held there for gates below kFarGate, whose results still
// lack far_factor.
constexpr float kLog2e = 1.44269504088896340736f, kFarGate = -87.0f;
__device__ __forceinline__ float sigmoid(float x) {
    const float d = 1.0f + __builtin_amdgcn_exp2f(__builtin_fminf(x * -kLog2e, 126.0f));
    const float r = __builtin_amdgcn_rcpf(d);
    return __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r);
}
// e^x / 2^-126 for gates beyond that, which takes p through the subnormal numbers to zero; else exactly 1.
__device__ __forceinline__ float far_factor(float x) {
    return __builtin_amdgcn_exp2f(__builtin_fminf(126.0f + x * kLog2e, 0.0f));
}

// Codes of a token's 128 channels (the 16 lanes of a DPP row) and their scale.
__device__ __forceinline__ float row_codes(const float (&v)[8], uint8_t *q) {
    float a = __builtin_fabsf(v[0]);
#pragma unroll
    for (int i = 1; i < 8; i++) a = __builtin_fmaxf(a, __builtin_fabsf(v[i]));
    const float top = __uint_as_float(row16_max(__float_as_uint(a)));
    uint2 o = {0u, 0u};
    if (top > 0x1p-110f && top < 0x1p110f) {  // 448 / top with a Newton step, far from where reciprocals are no normal numbers
        const float r = __builtin_amdgcn_rcpf(top), inv0 = 448.0f * r;
        const float inv = __builtin_fmaf(__builtin_fmaf(-top, inv0, 448.0f), r, inv0);
        o.x = encode4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
        o.y = encode4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
    } else if (top > 0.0f) {
        const double inv = 448.0 / (double)top;
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; i++) w[i] = (float)((double)v[i] * inv);
        o.x = encode4(w[0], w[1], w[2], w[3]);
        o.y = encode4(w[4], w[5], w[6], w[7]);
    }
    *reinterpret_cast<uint2 *>(q) = o;
    return group_scale(top);
}

// Tiles of 128 tokens x 128 channels, a thread 4 tokens x 8 channels of each of the three results: 96 registers of them.  Two
// workgroups to a CU would leave 128 registers and spill (235-268 us at 4096 x 18432), 1024 threads of 4 x 4 take 215; so one
// walks tiles b, b + G, ..., with the next tile's inputs on the way (40 more registers) while it computes: 170 us, 4.1 TB/s.
// What keeps it from a copy's 138: one tile at a time between three barriers, vector instructions for 0.52 of the time.
__global__ __launch_bounds__(kThreads, 2) void swiglu_backward_kernel(SwigluArgs p) {
    __shared__ __align__(16) uint32_t tile[3][128 * 32];
    __shared__ __align__(16) uint32_t top[3][128];  // the channels' bytes, as in column_bytes
    const int t = threadIdx.x, lane = t & 63, chunk = t & 15, g = t >> 4;
    const uint32_t FB = (uint32_t)(p.F >> 7), MB = (uint32_t)(p.cols >> 7), tiles = FB * MB;  // (fewer than 2^23)
    // The tiles under way are neighbours along the shorter side first, so that both the rows' and the columns' pieces that
    // are written together are long: 4096 x 18432 takes 170 us along the tokens and 184 along the channels, 8192 x 2048 41.2
    // and 39.9.
    auto place = [&](uint32_t i, int64_t &fb, int64_t &mb) __attribute__((always_inline)) {
        const uint32_t n = MB < FB ? MB : FB, far = i / n, near = i % n;
        fb = MB < FB ? far : near;
        mb = MB < FB ? near : far;
    };
    const int ldq = (int)(2 * p.F), ldg = (int)p.ldg;  // (offsets within a tile's 128 rows are 32 bits)
    uint2 xq[4], uq[4];
    u32x4 gq[4];
    float sx[4], su[4];
    auto load = [&](uint32_t i) __attribute__((always_inline)) {
        int64_t fb, mb;
        place(i, fb, mb);
        const int rows = (int)(p.M - mb * 128 < 128 ? p.M - mb * 128 : 128);
        const uint8_t *q0 = p.q + mb * 128 * 2 * p.F + fb * 128;
        const uint16_t *g0 = p.gh + mb * 128 * p.ldg + fb * 128;
        const float *sx0 = p.s + fb * p.M + mb * 128, *su0 = sx0 + FB * p.M;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const int m = g * 4 + j, r = m < rows ? m : rows - 1;
            xq[j] = *reinterpret_cast<const uint2 *>(q0 + (r * ldq + chunk * 8));
            uq[j] = *reinterpret_cast<const uint2 *>(q0 + p.F + (r * ldq + chunk * 8));
            gq[j] = load_stream16(g0 + (r * ldg + chunk * 8));
            sx[j] = sx0[r];
            su[j] = su0[r];
        }
    };
    load(blockIdx.x);
    for (uint32_t i = blockIdx.x; i < tiles; i += gridDim.x) {
        int64_t fb, mb;
        place(i, fb, mb);
        const int rows = (int)(p.M - mb * 128 < 128 ? p.M - mb * 128 : 128);
        uint8_t *oq = p.gq + mb * 128 * 2 * p.F + fb * 128;
        float *osx = p.gs + fb * p.M + mb * 128, *osu = osx + FB * p.M;
        if (t < 384) top[t >> 7][t & 127] = 0;
        uint2 x0[4], u0[4];
        u32x4 g0[4];
        float sx0[4], su0[4];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const bool in = g * 4 + j < rows;  // (rows past the last one: zeros)
            x0[j] = xq[j];
            u0[j] = uq[j];
            g0[j] = gq[j];
            sx0[j] = in ? sx[j] : 0.f;
            su0[j] = in ? su[j] : 0.f;
        }
        if (i + gridDim.x < tiles) load(i + gridDim.x);
        float v[3][4][8];  // dx, du, h
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const int m = g * 4 + j;
            float x[8], u[8], gr[8];
            decode8(x0[j], sx0[j], x);
            decode8(u0[j], su0[j], u);
            widen8(g0[j], gr);
            float p1[8], least = x[0];
#pragma unroll
            for (int c = 0; c < 8; c++) {
                p1[c] = sigmoid(x[c]);
                least = __builtin_fminf(least, x[c]);
            }
            if (__any(least < kFarGate)) {  // (rare, and the same for the whole wave)
#pragma unroll
                for (int c = 0; c < 8; c++) p1[c] *= far_factor(x[c]);
            }
#pragma unroll
            for (int c = 0; c < 8; c++) {
                const float sg = p1[c];
                const float silu = x[c] * sg;
                v[1][j][c] = gr[c] * silu;
                v[2][j][c] = silu * u[c];
                // p + x p (1 - p) = p + silu (1 - p)
                v[0][j][c] = gr[c] * u[c] * __builtin_fmaf(silu, 1.0f - sg, sg);
            }
            if (m < rows) {
                const float s0 = row_codes(v[0][j], oq + (m * ldq + chunk * 8));
                const float s1 = row_codes(v[1][j], oq + p.F + (m * ldq + chunk * 8));
                if (chunk == 0) {
                    osx[m] = s0;
                    osu[m] = s1;
                }
            }
        }
        lds_barrier();
#pragma unroll
        for (int k = 0; k < 3; k++) {
            Bytes8 e;
            column_bytes(v[k], e);
            lanes_max<16>(e);
            if (lane < 16) {
#pragma unroll
                for (int c = 0; c < 8; c++) atomicMax(&top[k][chunk * 8 + c], (uint32_t)e[c / 2][c % 2]);
            }
        }
        lds_barrier();
#pragma unroll
        for (int k = 0; k < 3; k++) {
            uint32_t byte[8];
#pragma unroll
            for (int c = 0; c < 8; c++) byte[c] = max(top[k][chunk * 8 + c], 8u) - 8u;
            uint8_t *et = k == 2 ? p.het + mb * p.F : p.get + mb * 2 * p.F + k * p.F;
            if (t >> 4 == k)
                *reinterpret_cast<uint2 *>(et + fb * 128 + chunk * 8) =
                    (uint2){byte[0] | byte[1] << 8 | byte[2] << 16 | byte[3] << 24,
                            byte[4] | byte[5] << 8 | byte[6] << 16 | byte[7] << 24};
#pragma unroll
            for (int c = 0; c < 8; c++)
                tile[k][(chunk * 8 + c) * 32 + (((g >> 2) ^ (chunk & 7)) << 2) + (g & 3)] =
                    encode4_pow2(v[k][0][c], v[k][1][c], v[k][2][c], v[k][3][c], byte[c]);
        }
        lds_barrier();
        column_store<128>(tile[0], p.gqt + fb * 128 * p.cols + mb * 128, p.cols, t);
        column_store<128>(tile[1], p.gqt + (p.F + fb * 128) * p.cols + mb * 128, p.cols, t);
        column_store<128>(tile[2], p.hqt + fb * 128 * p.cols + mb * 128, p.cols, t);
    }
}

}  // namespace

hipError_t launch_transpose_128x1(const void *x, const float *s, bool codes, int64_t ld, int64_t T, int64_t K,
                                  const int32_t *row_token, int64_t rows, uint8_t *qt, uint8_t *et,
                                  hipStream_t stream) {
    const int64_t cols = (rows + 127) / 128 * 128;
    if (T == 0) {  // (all rows are zeros; what they read does not matter, and the copy's first 128 rows are there)
        x = qt;
        s = reinterpret_cast<const float *>(qt);
    }
    const TransposeArgs p = {x, s, ld, T, K, rows, cols, row_token, qt, et};
    const dim3 grid((unsigned)((cols / 128 * ((K + 255) / 256) + 7) / 8 * 8));
    if (codes && row_token != nullptr)
        transpose_kernel<true, true><<<grid, kThreads, 0, stream>>>(p);
    else if (codes)
        transpose_kernel<true, false><<<grid, kThreads, 0, stream>>>(p);
    else if (row_token != nullptr)
        transpose_kernel<false, true><<<grid, kThreads, 0, stream>>>(p);
    else
        transpose_kernel<false, false><<<grid, kThreads, 0, stream>>>(p);
    return hipGetLastError();
}

hipError_t launch_swiglu_backward_quant(const uint8_t *q, const float *s, const uint16_t *gh, int64_t ldg, int64_t M,
                                        int64_t F, uint8_t *gq, float *gs, uint8_t *gqt, uint8_t *get, uint8_t *hqt,
                                        uint8_t *het, hipStream_t stream) {
    const int64_t cols = (M + 127) / 128 * 128;
    const SwigluArgs p = {q, s, gh, ldg, M, F, cols, gq, gs, gqt, get, hqt, het};
    const int64_t tiles = cols / 128 * (F / 128), wgs = cu_count();
    swiglu_backward_kernel<<<dim3((unsigned)(tiles < wgs ? tiles : wgs)), kThreads, 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace fp8q
