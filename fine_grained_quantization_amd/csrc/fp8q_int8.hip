// INT8 quantization with one scale per row (a token, or an output channel) and the INT8 matrix product, dense
// and per expert:
//   s[m] = fl32(max_k |x[m,k]| / 127),  q[m,k] = rne(fl32(x[m,k] / s[m])) in [-127, 127] (0 where s is 0)
//   C[m,n] = round( fl32(acc) * (sa[m] * sw[n]) ),  acc = sum_k qa[m,k] qw[n,k], exact in 32-bit integers
// (|code| <= 128 and K <= 131056, so |acc| < 2^31).
#include "fp8q_device.h"
#include "fp8q_kernels.h"
#include "fp8q_tiles.h"

namespace fp8q {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));

// RN64(1/127).  For every bf16 amax, fl32((double)amax * kInv127) is the fp32 quotient amax / 127: the product is
// within 2^-52 (relative) of it, and a quotient of an 8-bit significand by 127 is at least 2^-32 (relative) away
// from every fp32 rounding midpoint.
constexpr double kInv127 = 1.0 / 127.0;

__device__ __forceinline__ uint32_t int8x4(uint32_t d0, uint32_t d1, double inv) {
    const int a = (int)rintf(quotient(bf16_lo(d0), inv)), b = (int)rintf(quotient(bf16_hi(d0), inv));
    const int c = (int)rintf(quotient(bf16_lo(d1), inv)), d = (int)rintf(quotient(bf16_hi(d1), inv));
    return (uint32_t)(a & 255) | ((uint32_t)(b & 255) << 8) | ((uint32_t)(c & 255) << 16) | ((uint32_t)d << 24);
}

// One workgroup per row, the row's first CH * 2048 elements kept in registers between the two passes.  |x| <= amax
// and s = fl32(amax / 127) give |x / s| <= 127.008 (the most over every bf16 amax, reached where s is subnormal),
// which rounds to at most 127: no clamp.
template <int CH>
__global__ __launch_bounds__(256) void quant_int8_kernel(const uint16_t *__restrict__ x, int64_t ld, int64_t K,
                                                         uint8_t *__restrict__ q, float *__restrict__ s) {
    __shared__ uint32_t wmax[4];
    const int t = threadIdx.x;
    const int64_t m = blockIdx.x;
    const int64_t chunks = K >> 3;
    const uint16_t *row = x + m * ld;
    uint8_t *dst = q + m * K;
    u32x4 v[CH];
#pragma unroll
    for (int j = 0; j < CH; j++) {
        const int64_t c = t + 256 * j;
        v[j] = c < chunks ? load_stream16(row + c * 8) : (u32x4){0u, 0u, 0u, 0u};
    }
    u16x2 mh = absmax_halves(v[0]);
#pragma unroll
    for (int j = 1; j < CH; j++) mh = __builtin_elementwise_max(mh, absmax_halves(v[j]));
    for (int64_t c = t + 256 * CH; c < chunks; c += 256)
        mh = __builtin_elementwise_max(mh, absmax_halves(*reinterpret_cast<const u32x4 *>(row + c * 8)));
    const uint32_t wm = wave_max(halves_max(mh));
    if ((t & 63) == 0) wmax[t >> 6] = wm;
    __syncthreads();
    const float amax = bf16_mag_f32(max(max(wmax[0], wmax[1]), max(wmax[2], wmax[3])));
    const float sc = (float)((double)amax * kInv127);
    const double inv = scale_reciprocal(sc);
#pragma unroll
    for (int j = 0; j < CH; j++) {
        const int64_t c = t + 256 * j;
        if (c < chunks)
            *reinterpret_cast<uint2 *>(dst + c * 8) = (uint2){int8x4(v[j].x, v[j].y, inv), int8x4(v[j].z, v[j].w, inv)};
    }
    for (int64_t c = t + 256 * CH; c < chunks; c += 256) {
        const u32x4 u = load_stream16(row + c * 8);
        *reinterpret_cast<uint2 *>(dst + c * 8) = (uint2){int8x4(u.x, u.y, inv), int8x4(u.z, u.w, inv)};
    }
    if (t == 0) s[m] = sc;
}

// ---------------------------------------------------------------------------------------------------------
// Matrix product.  A workgroup of 4 waves computes 128 rows x 128 channels, a wave 64 x 64 of them, K in blocks
// of 128 codes through one LDS stage.
// ---------------------------------------------------------------------------------------------------------

constexpr int kTile = 128;

struct Int8Args {
    const uint8_t *qa;
    const float *sa;
    const uint8_t *qw;
    const float *sw;
    void *c;
    int64_t M, N, K;  // M: rows of c
    const int32_t *off, *rtok;
    int64_t E, T;     // T: rows of qa when rtok picks them
    int64_t n_mtiles, n_ntiles;
};

template <bool OUT_BF16, bool GROUPED, bool GATHER>
__global__ __launch_bounds__(256) void gemm_int8_kernel(Int8Args p) {
    __shared__ __attribute__((aligned(1024))) uint8_t tA[kTile * 128], tW[kTile * 128];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int64_t m0, mend = p.M, n0, e = 0;
    if constexpr (GROUPED) {
        if (!grouped_tile<kTile>(blockIdx.x, p.off, p.E, p.M, p.n_mtiles, p.n_ntiles, kTile, lane, m0, mend, n0, e))
            return;
    } else {
        int64_t mt, nt;
        if (!dense_tile_at(xcd_order(blockIdx.x), p.n_mtiles, p.n_ntiles, mt, nt)) return;
        m0 = mt * kTile;
        n0 = nt * kTile;
    }
    const uint8_t *W = p.qw + e * p.N * p.K;
    const float *SW = p.sw + e * p.N;
    const int wm = (wave & 1) * 64, wn = (wave >> 1) * 64;
    // Copies: thread t moves chunk t % 8 of rows t / 8, t / 8 + 32, ... of both tiles.
    const int cr = tid >> 3, cc = tid & 7;
    int64_t arow[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const int64_t r = m0 + cr + 32 * j;
        int64_t src = r < mend ? r : -1;
        if constexpr (GATHER) {
            src = src >= 0 ? p.rtok[src] : -1;
            if (src >= p.T) src = -1;
        }
        arow[j] = src;
    }
    v4i acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) acc[i][j] = (v4i){0, 0, 0, 0};
    const u32x4 zero = {0u, 0u, 0u, 0u};
    for (int64_t k0 = 0; k0 < p.K; k0 += 128) {
        u32x4 va[4], vw[4];
        const int64_t k = k0 + cc * 16;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const int64_t n = n0 + cr + 32 * j;
            va[j] = k < p.K && arow[j] >= 0 ? *reinterpret_cast<const u32x4 *>(p.qa + arow[j] * p.K + k) : zero;
            vw[j] = k < p.K && n < p.N ? *reinterpret_cast<const u32x4 *>(W + n * p.K + k) : zero;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; j++) {
            *reinterpret_cast<u32x4 *>(tA + swz(cr + 32 * j, cc)) = va[j];
            *reinterpret_cast<u32x4 *>(tW + swz(cr + 32 * j, cc)) = vw[j];
        }
        __syncthreads();
#pragma unroll
        for (int h = 0; h < 2; h++) {
            v4i fa[4], fw[4];
            const int ch = 4 * h + (lane >> 4);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                fa[i] = *reinterpret_cast<const v4i *>(tA + swz(wm + 16 * i + (lane & 15), ch));
                fw[i] = *reinterpret_cast<const v4i *>(tW + swz(wn + 16 * i + (lane & 15), ch));
            }
#pragma unroll
            for (int ni = 0; ni < 4; ni++)
#pragma unroll
                for (int mi = 0; mi < 4; mi++)
                    acc[ni][mi] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[ni], fa[mi], acc[ni][mi], 0, 0, 0);
        }
    }
    // A lane holds channels n .. n + 3 of one row.
#pragma unroll
    for (int mi = 0; mi < 4; mi++) {
        const int64_t m = m0 + wm + 16 * mi + (lane & 15);
        if (m >= mend) continue;
        int64_t src = m;
        if constexpr (GATHER) {
            src = p.rtok[m];
            if (src >= p.T) src = -1;
        }
        const float sa = src >= 0 ? p.sa[src] : 0.0f;
#pragma unroll
        for (int ni = 0; ni < 4; ni++) {
            const int64_t n = n0 + wn + 16 * ni + 4 * (lane >> 4);
            if (n >= p.N) continue;
            v4f v;
#pragma unroll
            for (int r = 0; r < 4; r++) v[r] = (float)acc[ni][mi][r] * (sa * SW[n + r]);
            store4<OUT_BF16>(p.c, m * p.N + n, v);
        }
    }
}

template <bool GROUPED, bool GATHER>
hipError_t launch_int8(Int8Args p, bool out_bf16, hipStream_t stream) {
    p.n_mtiles = GROUPED ? p.M / kTile + p.E : (p.M + kTile - 1) / kTile;
    p.n_ntiles = (p.N + kTile - 1) / kTile;
    const dim3 grid((unsigned)((p.n_mtiles * p.n_ntiles + 255) / 256 * 256));
    if (out_bf16)
        gemm_int8_kernel<true, GROUPED, GATHER><<<grid, 256, 0, stream>>>(p);
    else
        gemm_int8_kernel<false, GROUPED, GATHER><<<grid, 256, 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace

int64_t gemm_int8_blocks(int64_t M, int64_t N, int64_t E) {
    // an upper bound: 128 x 128 tiles; -1 past 2^40
    const int64_t mt = M / kTile + (E > 0 ? E : 1), nt = (N + kTile - 1) / kTile;
    if (nt > 0 && mt > (int64_t(1) << 40) / nt) return -1;
    return mt * nt + 256;
}

hipError_t launch_quant_int8(const uint16_t *x, int64_t ld, int64_t M, int64_t K, uint8_t *q, float *s,
                             hipStream_t stream) {
    const dim3 grid((unsigned)M);
    if (K <= 256 * 4 * 8)
        quant_int8_kernel<4><<<grid, 256, 0, stream>>>(x, ld, K, q, s);
    else
        quant_int8_kernel<8><<<grid, 256, 0, stream>>>(x, ld, K, q, s);
    return hipGetLastError();
}

hipError_t launch_gemm_int8(const uint8_t *qa, const float *sa, const uint8_t *qw, const float *sw, void *c,
                            bool out_bf16, int64_t M, int64_t N, int64_t K, hipStream_t stream) {
    const Int8Args p = {qa, sa, qw, sw, c, M, N, K, nullptr, nullptr, 0, M, 0, 0};
    return launch_int8<false, false>(p, out_bf16, stream);
}

hipError_t launch_grouped_gemm_int8(const uint8_t *qa, const float *sa, int64_t T, const int32_t *row_token,
                                    const uint8_t *qw, const float *sw, void *c, bool out_bf16, const int32_t *off,
                                    int64_t E, int64_t M_total, int64_t N, int64_t K, hipStream_t stream) {
    const Int8Args p = {qa, sa, qw, sw, c, M_total, N, K, off, row_token, E, T, 0, 0};
    return row_token != nullptr ? launch_int8<true, true>(p, out_bf16, stream)
                                : launch_int8<true, false>(p, out_bf16, stream);
}

}  // namespace fp8q
