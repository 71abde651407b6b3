// Root-mean-square norm in front of an FP8 Linear, and its gradients:
//   h = bf16(x + residual),  rstd = 1 / sqrt(mean_k h^2 + eps),  y = rstd * (h * w),
//   y in 1x128 groups: E4M3 codes and one fp32 scale each, either amax / 448 or the least power of two p with amax <= 448 p;
//   gx = gres + rstd (g w - h rstd^2 mean_k(g w h)),  gw = sum_m g h rstd.
// One read of each input and one write of each output: bound by memory, or for few rows by the latency of a load, the
// row's sum over its workgroup and a store.
#include "fp8q_device.h"
#include "fp8q_kernels.h"

namespace fp8q {
namespace {

__device__ __forceinline__ float elem(const u32x4 &v, int i) {
    const uint32_t d = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    return i & 1 ? bf16_hi(d) : bf16_lo(d);
}

// 8 weights from element k on, as they are (bf16) or widened to fp32.
template <bool W_BF16>
struct W8 {
    u32x4 v[W_BF16 ? 1 : 2];
    __device__ __forceinline__ void load(const void *w, int64_t k) {
        if constexpr (W_BF16) {
            v[0] = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(w) + k);
        } else {
            v[0] = *reinterpret_cast<const u32x4 *>(static_cast<const float *>(w) + k);
            v[1] = *reinterpret_cast<const u32x4 *>(static_cast<const float *>(w) + k + 4);
        }
    }
    __device__ __forceinline__ void zero() { v[0] = v[W_BF16 ? 0 : 1] = (u32x4){0u, 0u, 0u, 0u}; }
    __device__ __forceinline__ float at(int i) const {
        if constexpr (W_BF16) return elem(v[0], i);
        const u32x4 &u = v[i < 4 ? 0 : 1];
        return __uint_as_float((i & 3) == 0 ? u.x : (i & 3) == 1 ? u.y : (i & 3) == 2 ? u.z : u.w);
    }
};

template <bool W_BF16>
__device__ __forceinline__ void load_w8(const void *w, int64_t k, float *f) {
    if constexpr (W_BF16) {
        const u32x4 v = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(w) + k);
#pragma unroll
        for (int i = 0; i < 8; i++) f[i] = elem(v, i);
    } else {
        const float4 a = *reinterpret_cast<const float4 *>(static_cast<const float *>(w) + k);
        const float4 b = *reinterpret_cast<const float4 *>(static_cast<const float *>(w) + k + 4);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
}

__device__ __forceinline__ u32x4 add8(const u32x4 &a, const u32x4 &b) {
    u32x4 o;
    o.x = pack_bf16x2(bf16_lo(a.x) + bf16_lo(b.x), bf16_hi(a.x) + bf16_hi(b.x));
    o.y = pack_bf16x2(bf16_lo(a.y) + bf16_lo(b.y), bf16_hi(a.y) + bf16_hi(b.y));
    o.z = pack_bf16x2(bf16_lo(a.z) + bf16_lo(b.z), bf16_hi(a.z) + bf16_hi(b.z));
    o.w = pack_bf16x2(bf16_lo(a.w) + bf16_lo(b.w), bf16_hi(a.w) + bf16_hi(b.w));
    return o;
}

// Sum over the workgroup's threads; every thread gets it.  The order is fixed.  T: the type in which the waves' sums are added.
template <int THREADS, typename T = float>
__device__ __forceinline__ T block_sum(float v, float *part) {
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    T s = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 64; i++) s += part[i];
    return s;
}

// 1 / sqrt(a): the hardware's fp32 result and a Newton step in double, where a and the result are normal numbers by far.
__device__ __forceinline__ double inverse_root(double a) {
    if (!(a > 0x1p-100 && a < 0x1p120)) return 1.0f / sqrtf((float)a);
    const double r = __builtin_amdgcn_rsqf((float)a);
    return fma(r * 0.5, fma(-a * r, r, 1.0), r);
}

struct NormArgs {
    const uint16_t *x, *res;
    int64_t ldx, ldr, K;
    const void *w;
    float eps;
    double inv_k;
    uint16_t *h, *y;
    uint8_t *q;
    float *s, *rstd;
    int64_t M;
    bool stream;
};

// A row's first chunks, CH a thread.
template <int THREADS, int CH>
__device__ __forceinline__ void load_row(const uint16_t *x, int64_t chunks, bool stream, u32x4 (&v)[CH]) {
    if (stream) {
#pragma unroll
        for (int j = 0; j < CH; j++) {
            const int64_t c = threadIdx.x + THREADS * j;
            v[j] = c < chunks ? load_stream16(x + c * 8) : (u32x4){0u, 0u, 0u, 0u};
        }
    } else {
#pragma unroll
        for (int j = 0; j < CH; j++) {
            const int64_t c = threadIdx.x + THREADS * j;
            v[j] = c < chunks ? *reinterpret_cast<const u32x4 *>(x + c * 8) : (u32x4){0u, 0u, 0u, 0u};
        }
    }
}

// Codes of one 8-element chunk of h: t = h w, exact in fp32 where w is bf16.  A group's 16 chunks lie in the 16 lanes of a
// DPP row.  With scale amax / 448 the row's factor cancels, y / (amax_y / 448) = t 448 / amax_t; products of two bf16
// values often lie right between two codes, and the quotient (in double, as the other quantizers form it) is then that
// tie, which a rounded factor would decide at random.
template <bool W_BF16, bool POW2>
__device__ __forceinline__ void norm_chunk(const NormArgs &p, const u32x4 &v, int64_t m, int64_t c, float r) {
    float t[8];
    load_w8<W_BF16>(p.w, c * 8, t);
#pragma unroll
    for (int i = 0; i < 8; i++) t[i] *= elem(v, i);
    if (p.y != nullptr || POW2) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; i++) y[i] = t[i] * r;
        if (p.y != nullptr) {
            const u32x4 o = {pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                             pack_bf16x2(y[6], y[7])};
            *reinterpret_cast<u32x4 *>(p.y + m * p.K + c * 8) = o;
        }
        if constexpr (POW2) {
#pragma unroll
            for (int i = 0; i < 8; i++) t[i] = y[i];
        }
    }
    if (p.q == nullptr) return;
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) a = max(a, __float_as_uint(t[i]) & 0x7FFFFFFFu);
    a = row16_max(a);
    uint2 o;
    float sc;
    if constexpr (POW2) {
        const uint32_t e = pow2_byte(a);
        const float inv = pow2_inverse(e);
        o.x = encode4(t[0] * inv, t[1] * inv, t[2] * inv, t[3] * inv);
        o.y = encode4(t[4] * inv, t[5] * inv, t[6] * inv, t[7] * inv);
        sc = a > 0 ? pow2_value(e) : 0.0f;
    } else {
        const float top = __uint_as_float(a);
        const double inv = top > 0.0f ? 448.0 / (double)top : 0.0;
        o.x = encode4(quotient(t[0], inv), quotient(t[1], inv), quotient(t[2], inv), quotient(t[3], inv));
        o.y = encode4(quotient(t[4], inv), quotient(t[5], inv), quotient(t[6], inv), quotient(t[7], inv));
        sc = (float)((double)top * (double)r * kInv448);
    }
    *reinterpret_cast<uint2 *>(p.q + m * p.K + c * 8) = o;
    if ((c & 15) == 0) p.s[(c >> 4) * p.M + m] = sc;
}

// One workgroup per row, its first CH * THREADS chunks of 8 elements kept in registers between the sum and the codes; the
// chunks past them are read again.  (x, residual and h may be one array: a thread reads its elements before it writes them.)
// Threads by K, so that a row fits their registers: 256 x 1 chunk, 256 x 4, 1024 x 3.  Bound by memory: 4096 x 7168 with a
// residual 41 us, 5.0 TB/s (as a large copy); 8192 x 2048 21.5 us, 5.4.  One row 4.2 us: a load, the sum, a store.
template <bool W_BF16, bool POW2, int THREADS, int CH>
__global__ __launch_bounds__(THREADS) void rmsnorm_quant_kernel(NormArgs p) {
    __shared__ float part[THREADS / 64];
    const int64_t m = blockIdx.x;
    const int t = threadIdx.x;
    const int64_t chunks = p.K >> 3;
    const uint16_t *x = p.x + m * p.ldx;
    const uint16_t *res = p.res != nullptr ? p.res + m * p.ldr : nullptr;
    uint16_t *h = p.res != nullptr ? p.h + m * p.K : nullptr;
    u32x4 v[CH];
    load_row<THREADS>(x, chunks, p.stream, v);
    if (res != nullptr) {
        u32x4 u[CH];
        load_row<THREADS>(res, chunks, p.stream, u);
#pragma unroll
        for (int j = 0; j < CH; j++) {
            const int64_t c = t + THREADS * j;
            v[j] = add8(v[j], u[j]);
            if (c < chunks) *reinterpret_cast<u32x4 *>(h + c * 8) = v[j];
        }
    }
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < CH; j++)
#pragma unroll
        for (int i = 0; i < 8; i++) ss = __builtin_fmaf(elem(v[j], i), elem(v[j], i), ss);
    for (int64_t c = t + THREADS * CH; c < chunks; c += THREADS) {
        u32x4 a = *reinterpret_cast<const u32x4 *>(x + c * 8);
        if (res != nullptr) {
            a = add8(a, *reinterpret_cast<const u32x4 *>(res + c * 8));
            *reinterpret_cast<u32x4 *>(h + c * 8) = a;
        }
#pragma unroll
        for (int i = 0; i < 8; i++) ss = __builtin_fmaf(elem(a, i), elem(a, i), ss);
    }
    const float r = (float)inverse_root(block_sum<THREADS, double>(ss, part) * p.inv_k + (double)p.eps);
    if (t == 0 && p.rstd != nullptr) p.rstd[m] = r;
    if (p.q == nullptr && p.y == nullptr) return;
#pragma unroll
    for (int j = 0; j < CH; j++) {
        const int64_t c = t + THREADS * j;
        if (c < chunks) norm_chunk<W_BF16, POW2>(p, v[j], m, c, r);
    }
    for (int64_t c = t + THREADS * CH; c < chunks; c += THREADS)
        norm_chunk<W_BF16, POW2>(p, *reinterpret_cast<const u32x4 *>((res != nullptr ? h : x) + c * 8), m, c, r);
}

template <bool W_BF16, bool POW2>
hipError_t launch_norm(const NormArgs &p, hipStream_t stream) {
    const dim3 grid((unsigned)p.M);
    if (p.K <= 2048)
        rmsnorm_quant_kernel<W_BF16, POW2, 256, 1><<<grid, 256, 0, stream>>>(p);
    else if (p.K <= 8192)
        rmsnorm_quant_kernel<W_BF16, POW2, 256, 4><<<grid, 256, 0, stream>>>(p);
    else
        rmsnorm_quant_kernel<W_BF16, POW2, 1024, 3><<<grid, 1024, 0, stream>>>(p);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------------------------------------
// Gradients.  A workgroup takes rows b, b + G, ..., the next row on the way while one is summed up (K up to 8192), and keeps its columns'
// weights and parts of gw in registers; the parts [G][K] meet in the workspace and a second launch adds them in order.
// Up to kFewRows rows gw needs no parts: in the same launch further workgroups read g and h again (from the caches) and sum
// up 64 columns each (128 x 7168: 8.5 us a call; 129 x 7168, with parts, 12.2).  Bound by memory: 4096 x 7168 42 us, 5.6 TB/s,
// and 4.6 for the second launch, which has 7 MB of parts to read.
// ---------------------------------------------------------------------------------------------------------

struct NormGradArgs {
    const uint16_t *g, *h, *gres;
    int64_t ldg, ldh, M, K;
    const void *w;
    const float *rstd;
    uint16_t *gx;
    float *part;  // [G][K], or null
    float *gw;    // for the further workgroups, from number G on
    int64_t G;
};

constexpr int64_t kFewRows = 128;
constexpr float kMaxF32 = 3.402823466e38f;

template <bool W_BF16, int THREADS, int CH>
__global__ __launch_bounds__(THREADS) void rmsnorm_backward_kernel(NormGradArgs p) {
    __shared__ float part[2][THREADS / 64];
    __shared__ float sums[THREADS / 8][64];
    const int t = threadIdx.x;
    if (blockIdx.x >= p.G) {  // gw of 64 columns: 8 threads a row, 8 columns each
        const int64_t k0 = (blockIdx.x - p.G) * 64 + (t & 7) * 8;
        float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int64_t m = t >> 3; m < p.M; m += THREADS / 8) {
            const u32x4 g = *reinterpret_cast<const u32x4 *>(p.g + m * p.ldg + k0);
            const u32x4 h = *reinterpret_cast<const u32x4 *>(p.h + m * p.ldh + k0);
            const float r = p.rstd[m];
#pragma unroll
            for (int i = 0; i < 8; i++) s[i] = __builtin_fmaf(elem(g, i) * elem(h, i), r, s[i]);
        }
#pragma unroll
        for (int i = 0; i < 8; i++) sums[t >> 3][(t & 7) * 8 + i] = s[i];
        __syncthreads();
        if (t < 64) {
            float sum = 0.f;
            for (int i = 0; i < THREADS / 8; i++) sum += sums[i][t];
            p.gw[(blockIdx.x - p.G) * 64 + t] = sum;
        }
        return;
    }
    const int64_t chunks = p.K >> 3;
    float gw[CH][8];
    W8<W_BF16> w[CH];
    u32x4 g[CH], h[CH], a[CH];
    auto load = [&](int64_t m) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < CH; j++) {
            const int64_t c = t + THREADS * j;
            const bool in = m < p.M && c < chunks;
            g[j] = in ? load_stream16(p.g + m * p.ldg + c * 8) : (u32x4){0u, 0u, 0u, 0u};
            h[j] = in ? load_stream16(p.h + m * p.ldh + c * 8) : (u32x4){0u, 0u, 0u, 0u};
            a[j] = in && p.gres != nullptr ? *reinterpret_cast<const u32x4 *>(p.gres + m * p.K + c * 8) : (u32x4){0u, 0u, 0u, 0u};
        }
    };
    constexpr bool kAhead = CH == 1;  // (else the registers would not suffice for two rows)
    if constexpr (kAhead) load(blockIdx.x);
#pragma unroll
    for (int j = 0; j < CH; j++) {
        const int64_t c = t + THREADS * j;
#pragma unroll
        for (int i = 0; i < 8; i++) gw[j][i] = 0.f;
        w[j].zero();
        if (c < chunks) w[j].load(p.w, c * 8);
    }
    int flip = 0;
    for (int64_t m = blockIdx.x; m < p.M; m += p.G, flip ^= 1) {
        const float r = p.rstd[m];
        if constexpr (!kAhead) load(m);
        u32x4 g0[CH], h0[CH], a0[CH];
#pragma unroll
        for (int j = 0; j < CH; j++) {
            g0[j] = g[j];
            h0[j] = h[j];
            a0[j] = a[j];
        }
        if constexpr (kAhead) load(m + p.G);
        float dot = 0.f;
#pragma unroll
        for (int j = 0; j < CH; j++)
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const float gh = elem(g0[j], i) * elem(h0[j], i);
                gw[j][i] = __builtin_fmaf(gh, r, gw[j][i]);
                dot = __builtin_fmaf(gh, w[j].at(i), dot);
            }
        // (two buffers in turn: a wave may reach the next row's sum while others still read this one)
        const float sum = block_sum<THREADS>(dot, part[flip]);
        // (r is past 2^64, and its square past fp32, where eps is below 3e-39 and the row small: f itself need not be)
        const float r2 = r * r, f = r2 <= kMaxF32 ? r2 * sum / (float)p.K : r * (r * (sum / (float)p.K));
#pragma unroll
        for (int j = 0; j < CH; j++) {
            const int64_t c = t + THREADS * j;
            if (c >= chunks) continue;
            // (not to be kept in fp32 since the sum: those registers would be missing)
            asm volatile("" : "+v"(g0[j]), "+v"(h0[j]));
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; i++)
                o[i] = elem(a0[j], i) + r * (elem(g0[j], i) * w[j].at(i) - elem(h0[j], i) * f);
            const u32x4 v = {pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]),
                             pack_bf16x2(o[6], o[7])};
            *reinterpret_cast<u32x4 *>(p.gx + m * p.K + c * 8) = v;
        }
    }
    if (p.part != nullptr) {
#pragma unroll
        for (int j = 0; j < CH; j++) {
            const int64_t c = t + THREADS * j;
            if (c < chunks) {
                float *o = p.part + blockIdx.x * p.K + c * 8;
                *reinterpret_cast<float4 *>(o) = make_float4(gw[j][0], gw[j][1], gw[j][2], gw[j][3]);
                *reinterpret_cast<float4 *>(o + 4) = make_float4(gw[j][4], gw[j][5], gw[j][6], gw[j][7]);
            }
        }
    }
}

// gw[k] = sum over the G parts: 32 threads a column, each its parts in order, then those sums in order.
__global__ __launch_bounds__(1024) void rmsnorm_gw_kernel(const float *__restrict__ part, int64_t G, int64_t K,
                                                          float *__restrict__ gw) {
    __shared__ float sum[32][32];
    const int64_t k = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31);
    const int slice = threadIdx.x >> 5;
    float s = 0.f;
#pragma unroll 8
    for (int64_t g = slice; g < G; g += 32) s += part[g * K + k];
    sum[slice][threadIdx.x & 31] = s;
    __syncthreads();
    if (slice == 0) {
        for (int i = 1; i < 32; i++) s += sum[i][threadIdx.x];
        gw[k] = s;
    }
}

// As many workgroups as the CUs hold at once: four of 256 threads, two of 1024, or one of those with three chunks a thread.
int64_t norm_groups(int64_t M, int64_t K) {
    const int64_t most = (K <= 2048 ? 4 : K <= 8192 ? 2 : 1) * cu_count();
    return M < most ? M : most;
}

template <bool W_BF16>
void launch_norm_backward(const NormGradArgs &p, hipStream_t stream) {
    const dim3 grid((unsigned)(p.G + (p.gw != nullptr ? p.K / 64 : 0)));
    if (p.K <= 2048) rmsnorm_backward_kernel<W_BF16, 256, 1><<<grid, 256, 0, stream>>>(p);
    else if (p.K <= 8192) rmsnorm_backward_kernel<W_BF16, 1024, 1><<<grid, 1024, 0, stream>>>(p);
    else rmsnorm_backward_kernel<W_BF16, 1024, 3><<<grid, 1024, 0, stream>>>(p);
}

}  // namespace

int64_t rmsnorm_backward_workspace_bytes(int64_t M, int64_t K) { return M <= kFewRows ? 0 : norm_groups(M, K) * K * 4; }

hipError_t launch_rmsnorm_quant_act_1x128(const uint16_t *x, int64_t ldx, const uint16_t *residual, int64_t ldr,
                                          const void *w, bool w_bf16, float eps, bool pow2, int64_t M, int64_t K,
                                          uint16_t *h, uint16_t *y, uint8_t *q, float *s, float *rstd,
                                          hipStream_t stream) {
    // Streaming loads for inputs of 96 to 256 MB, which the last cache cannot keep beside the outputs, but would try to.  us with
    // them and without: 4096 x 4096 and a residual (67 MB) 24.9, 22.9; 4096 x 5120 (84 MB) 29.5, 29.2; 4096 x 7168 (117 MB) 41.2,
    // 46.7; 8192 x 5120 (168 MB) 51.4, 57.1; 8192 x 7168 (235 MB) 78.0, 79.2, and 82, 85 where x has just been written;
    // 16384 x 7168 149 both, and then 170, 150.
    const int64_t in = M * K * (residual != nullptr ? 4 : 2);
    const bool stream_loads = in > (int64_t(96) << 20) && in <= (int64_t(256) << 20);
    const NormArgs p = {x, residual, ldx, ldr, K, w, eps, K > 0 ? 1.0 / (double)K : 0.0, h, y, q, s, rstd, M, stream_loads};
    if (w_bf16) return pow2 ? launch_norm<true, true>(p, stream) : launch_norm<true, false>(p, stream);
    return pow2 ? launch_norm<false, true>(p, stream) : launch_norm<false, false>(p, stream);
}

hipError_t launch_rmsnorm_backward(const uint16_t *gy, int64_t ldg, const uint16_t *h, int64_t ldh, const void *w,
                                   bool w_bf16, const float *rstd, const uint16_t *gres, int64_t M, int64_t K,
                                   uint16_t *gx, float *gw, float *workspace, hipStream_t stream) {
    const int64_t G = norm_groups(M, K);
    const bool few = M <= kFewRows;
    const NormGradArgs p = {gy, h, gres, ldg, ldh, M, K, w, rstd, gx, gw != nullptr && !few ? workspace : nullptr,
                            few ? gw : nullptr, G};
    if (M > 0 || gw != nullptr) {
        if (w_bf16) launch_norm_backward<true>(p, stream);
        else launch_norm_backward<false>(p, stream);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (p.part != nullptr) rmsnorm_gw_kernel<<<dim3((unsigned)(K / 32)), 1024, 0, stream>>>(workspace, G, K, gw);
    return hipGetLastError();
}

}  // namespace fp8q
