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

constexpr int kThreads = 512;        // a thread holds 4 tokens x 8 channels of a tile
constexpr int kR = 4, kG = kThreads / 16;

// Column maxima by token group, then (dead by then) the transposed codes: tile row = channel, 128 code bytes = 8 pieces of
// 16 bytes; piece p of row r sits at p ^ ((r / 8) & 7), which spreads one store instruction's 4-byte writes over the banks.
union ColumnTile {
    uint32_t top[kG][128];
    uint32_t tile[128 * 32];
};

// 8 codes to fp32 values times s.
__device__ __forceinline__ void decode8(const uint2 &d, float s, float *v) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    const f2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)d.x, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)d.x, true);
    const f2 c = __builtin_amdgcn_cvt_pk_f32_fp8((int)d.y, false), e = __builtin_amdgcn_cvt_pk_f32_fp8((int)d.y, true);
    v[0] = a[0] * s; v[1] = a[1] * s; v[2] = b[0] * s; v[3] = b[1] * s;
    v[4] = c[0] * s; v[5] = c[1] * s; v[6] = e[0] * s; v[7] = e[1] * s;
}

__device__ __forceinline__ void widen8(const u32x4 &d, float *v) {
    v[0] = bf16_lo(d.x); v[1] = bf16_hi(d.x); v[2] = bf16_lo(d.y); v[3] = bf16_hi(d.y);
    v[4] = bf16_lo(d.z); v[5] = bf16_hi(d.z); v[6] = bf16_lo(d.w); v[7] = bf16_hi(d.w);
}

__device__ __forceinline__ void column_tops(const float (&v)[kR][8], ColumnTile &sh, int g, int chunk) {
#pragma unroll
    for (int c = 0; c < 8; c++) {
        uint32_t a = 0;
#pragma unroll
        for (int j = 0; j < kR; j++) a = max(a, __float_as_uint(v[j][c]) & 0x7FFFFFFFu);
        sh.top[g][chunk * 8 + c] = a;
    }
}

// After column_tops and a barrier: threads [t0, t0 + 128) form the channels' scale bytes.
__device__ __forceinline__ void column_scales(const ColumnTile &sh, uint8_t *bytes, uint8_t *et, int i) {
    uint32_t a = 0;
#pragma unroll
    for (int g = 0; g < kG; g++) a = max(a, sh.top[g][i]);
    const uint32_t e = pow2_byte(a);
    bytes[i] = (uint8_t)e;
    et[i] = (uint8_t)e;
}

// After the scales and a barrier: the thread's codes into the tile.
__device__ __forceinline__ void column_codes(const float (&v)[kR][8], ColumnTile &sh, const uint8_t *bytes, int g,
                                             int chunk) {
    const uint2 b = *reinterpret_cast<const uint2 *>(bytes + chunk * 8);
#pragma unroll
    for (int c = 0; c < 8; c++) {
        const float inv = pow2_inverse(((c < 4 ? b.x : b.y) >> (8 * (c & 3))) & 255u);
        const uint32_t w = encode4(v[0][c] * inv, v[1][c] * inv, v[2][c] * inv, v[3][c] * inv);
        sh.tile[(chunk * 8 + c) * 32 + (((g >> 2) ^ (chunk & 7)) << 2) + (g & 3)] = w;
    }
}

// After another barrier: the tile's rows to the channel-major copy (rows ld bytes apart).
__device__ __forceinline__ void column_store(const ColumnTile &sh, uint8_t *qt, int64_t ld, int t) {
#pragma unroll
    for (int i = 0; i < 1024 / kThreads; i++) {
        const int p = t + i * kThreads, row = p >> 3, piece = p & 7;
        *reinterpret_cast<u32x4 *>(qt + row * ld + piece * 16) =
            *reinterpret_cast<const u32x4 *>(&sh.tile[row * 32 + ((piece ^ ((row >> 3) & 7)) << 2)]);
    }
}

struct TransposeArgs {
    const void *x;
    const float *s;
    int64_t ld, T, K, rows, cols;  // cols: rows rounded up to 128
    const int32_t *row_token;
    uint8_t *qt, *et;
};

template <bool CODES>
__global__ __launch_bounds__(kThreads) void transpose_kernel(TransposeArgs p) {
    __shared__ __align__(16) ColumnTile sh;
    __shared__ __align__(8) uint8_t bytes[128];
    const int t = threadIdx.x, chunk = t & 15, g = t >> 4;
    const int64_t KB = p.K >> 7, kb = blockIdx.x % KB, mb = blockIdx.x / KB;
    float v[kR][8];
#pragma unroll
    for (int j = 0; j < kR; j++) {
        const int64_t m = mb * 128 + g * kR + j;
        int64_t tok = m < p.rows ? m : -1;
        if (p.row_token != nullptr && tok >= 0) tok = p.row_token[m];
        if (tok >= p.T) tok = -1;
        if constexpr (CODES) {
            uint2 d = {0u, 0u};
            float s = 0.f;
            if (tok >= 0) {
                d = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(p.x) + tok * p.K + kb * 128 + chunk * 8);
                s = p.s[kb * p.T + tok];
            }
            decode8(d, s, v[j]);
        } else {
            u32x4 d = {0u, 0u, 0u, 0u};
            if (tok >= 0)
                d = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(p.x) + tok * p.ld + kb * 128 + chunk * 8);
            widen8(d, v[j]);
        }
    }
    column_tops(v, sh, g, chunk);
    __syncthreads();
    if (t < 128) column_scales(sh, bytes, p.et + mb * p.K + kb * 128, t);
    __syncthreads();
    column_codes(v, sh, bytes, g, chunk);
    __syncthreads();
    column_store(sh, p.qt + kb * 128 * p.cols + mb * 128, p.cols, t);
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

// Codes of a token's 128 channels (the 16 lanes of a DPP row) and their scale.
__device__ __forceinline__ void row_codes(const float (&v)[8], uint8_t *q, float *s, bool first) {
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) a = max(a, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    const float top = __uint_as_float(row16_max(a));
    const float inv = top > 0.0f ? 448.0f / top : 0.0f;
    uint2 o;
    o.x = encode4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    o.y = encode4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
    *reinterpret_cast<uint2 *>(q) = o;
    if (first) *s = top / 448.0f;
}

__global__ __launch_bounds__(kThreads) void swiglu_backward_kernel(SwigluArgs p) {
    __shared__ __align__(16) ColumnTile sh[3];
    __shared__ __align__(8) uint8_t bytes[3][128];
    const int t = threadIdx.x, chunk = t & 15, g = t >> 4;
    const int64_t FB = p.F >> 7, fb = blockIdx.x % FB, mb = blockIdx.x / FB;
    float dx[kR][8], du[kR][8], h[kR][8];
#pragma unroll
    for (int j = 0; j < kR; j++) {
        const int64_t m = mb * 128 + g * kR + j;
        uint2 a = {0u, 0u}, b = {0u, 0u};
        u32x4 d = {0u, 0u, 0u, 0u};
        float sa = 0.f, sb = 0.f;
        if (m < p.M) {
            const uint8_t *row = p.q + m * 2 * p.F + fb * 128 + chunk * 8;
            a = *reinterpret_cast<const uint2 *>(row);
            b = *reinterpret_cast<const uint2 *>(row + p.F);
            d = *reinterpret_cast<const u32x4 *>(p.gh + m * p.ldg + fb * 128 + chunk * 8);
            sa = p.s[fb * p.M + m];
            sb = p.s[(fb + FB) * p.M + m];
        }
        float x[8], u[8], gr[8];
        decode8(a, sa, x);
        decode8(b, sb, u);
        widen8(d, gr);
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float e = __expf(-x[i]);
            const float sg = 1.0f / (1.0f + e);
            const float silu = x[i] * sg;
            du[j][i] = gr[i] * silu;
            dx[j][i] = gr[i] * u[i] * (sg * (1.0f + x[i] * (1.0f - sg)));
            h[j][i] = silu * u[i];
        }
        if (m < p.M) {
            uint8_t *q = p.gq + m * 2 * p.F + fb * 128 + chunk * 8;
            row_codes(dx[j], q, p.gs + fb * p.M + m, chunk == 0);
            row_codes(du[j], q + p.F, p.gs + (fb + FB) * p.M + m, chunk == 0);
        }
    }
    column_tops(dx, sh[0], g, chunk);
    column_tops(du, sh[1], g, chunk);
    column_tops(h, sh[2], g, chunk);
    __syncthreads();
    if (t < 384) {
        const int k = t >> 7;
        uint8_t *et = k == 0 ? p.get + mb * 2 * p.F + fb * 128 : k == 1 ? p.get + mb * 2 * p.F + p.F + fb * 128
                                                                      : p.het + mb * p.F + fb * 128;
        column_scales(sh[k], bytes[k], et, t & 127);
    }
    __syncthreads();
    column_codes(dx, sh[0], bytes[0], g, chunk);
    column_codes(du, sh[1], bytes[1], g, chunk);
    column_codes(h, sh[2], bytes[2], g, chunk);
    __syncthreads();
    column_store(sh[0], p.gqt + fb * 128 * p.cols + mb * 128, p.cols, t);
    column_store(sh[1], p.gqt + (p.F + fb * 128) * p.cols + mb * 128, p.cols, t);
    column_store(sh[2], p.hqt + fb * 128 * p.cols + mb * 128, p.cols, t);
}

}  // namespace

hipError_t launch_transpose_128x1(const void *x, const float *s, bool codes, int64_t ld, int64_t T, int64_t K,
                                  const int32_t *row_token, int64_t rows, uint8_t *qt, uint8_t *et,
                                  hipStream_t stream) {
    const int64_t cols = (rows + 127) / 128 * 128;
    const TransposeArgs p = {x, s, ld, T, K, rows, cols, row_token, qt, et};
    const dim3 grid((unsigned)(cols / 128 * (K / 128)));
    if (codes)
        transpose_kernel<true><<<grid, kThreads, 0, stream>>>(p);
    else
        transpose_kernel<false><<<grid, kThreads, 0, stream>>>(p);
    return hipGetLastError();
}

hipError_t launch_swiglu_backward_quant(const uint8_t *q, const float *s, const uint16_t *gh, int64_t ldg, int64_t M,
                                        int64_t F, uint8_t *gq, float *gs, uint8_t *gqt, uint8_t *get, uint8_t *hqt,
                                        uint8_t *het, hipStream_t stream) {
    const int64_t cols = (M + 127) / 128 * 128;
    const SwigluArgs p = {q, s, gh, ldg, M, F, cols, gq, gs, gqt, get, hqt, het};
    swiglu_backward_kernel<<<dim3((unsigned)(cols / 128 * (F / 128))), kThreads, 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace fp8q
