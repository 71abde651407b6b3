// Combination of the experts' output rows back into tokens, and its gradient.
//   y[t] = add[t] + sum_j weight[t][j] * c[row_of[t][j]]
//   grad_c[row_of[t][j]] = weight[t][j] * grad_y[t],   grad_weight[t][j] = <grad_y[t], c[row_of[t][j]]>
// with sums in fp32 (slots in order j = 0, 1, ...) and one rounding at the end.  A slot whose row is outside
// [0, rows) is empty: it adds nothing, its gradient is 0 and no row is read or written for it.
// Both are bound by memory: each expert row is read (and its gradient written) once, with loads and stores that do not
// stay in the caches.  8192 tokens x 8 rows of 7168 bf16: 1.17 GB in 221 us, 5.3 TB/s (a device copy: 5.2; with cached
// loads 230 us).  The gradient of 4093 tokens x 6 rows of 2048: 218 MB and 16 MB of zeros in 44 us, 5.3 TB/s (with
// cached loads and stores 53 us).  64 tokens: 3.8 us, a launch and two round trips to memory.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8q_device.h"
#include "fp8q_kernels.h"

namespace fp8q {
namespace {

// A 16-byte chunk of a row as fp32 values: 8 of bf16, 4 of fp32.
template <bool BF16>
struct Chunk {
    static constexpr int N = BF16 ? 8 : 4;
    float f[N];
    __device__ __forceinline__ void set(const u32x4 &v) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            if constexpr (BF16) {
                f[2 * i] = bf16_lo(v[i]);
                f[2 * i + 1] = bf16_hi(v[i]);
            } else {
                f[i] = __uint_as_float(v[i]);
            }
        }
    }
    __device__ __forceinline__ u32x4 pack() const {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            if constexpr (BF16)
                v[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
            else
                v[i] = __float_as_uint(f[i]);
        }
        return v;
    }
};

constexpr int kSlots = 8;  // expert rows in flight per lane
constexpr int kZeroRows = 16;

// One workgroup of 256 lanes per (token, 256 chunks of its row): a lane owns one 16-byte chunk of y, so that a few tokens
// spread over many CUs too.
template <bool BF16>
__global__ __launch_bounds__(256) void moe_combine_kernel(const void *__restrict__ c, int64_t rows, int64_t chunks,
                                                          int64_t spans, const int32_t *__restrict__ row_of,
                                                          const float *__restrict__ weight, int k,
                                                          const void *__restrict__ add, void *__restrict__ y) {
    const int64_t t = blockIdx.x / spans;
    const int64_t ch = (blockIdx.x - t * spans) * 256 + threadIdx.x;
    if (ch >= chunks) return;
    const u32x4 *src = static_cast<const u32x4 *>(c) + ch;
    const u32x4 zero = {0u, 0u, 0u, 0u};
    Chunk<BF16> acc;
    acc.set(add != nullptr ? static_cast<const u32x4 *>(add)[t * chunks + ch] : zero);
    for (int j0 = 0; j0 < k; j0 += kSlots) {
        u32x4 v[kSlots];
        float w[kSlots];
#pragma unroll
        for (int u = 0; u < kSlots; u++) {
            const int64_t r = j0 + u < k ? row_of[t * k + j0 + u] : -1;  // the same in every lane
            const bool in = r >= 0 && r < rows;
            w[u] = in ? weight[t * k + j0 + u] : -0.0f;  // (-0 * 0 leaves every sum as it is, -0 too)
            v[u] = in ? load_stream16(src + r * chunks) : zero;
        }
#pragma unroll
        for (int u = 0; u < kSlots; u++) {
            Chunk<BF16> x;
            x.set(v[u]);
#pragma unroll
            for (int i = 0; i < Chunk<BF16>::N; i++) acc.f[i] = __builtin_fmaf(w[u], x.f[i], acc.f[i]);
        }
    }
    static_cast<u32x4 *>(y)[t * chunks + ch] = acc.pack();
}

// The first T workgroups take one token each: a lane walks the row in 16-byte chunks, keeps one partial sum per
// slot, and the workgroup adds the partials up in a fixed order.  The workgroups after them write zeros into the
// rows below offsets[E] that no token has, kZeroRows rows each.
template <bool BF16>
__global__ __launch_bounds__(256) void moe_combine_backward_kernel(
    const void *__restrict__ grad_y, const void *__restrict__ c, int64_t rows, int64_t chunks,
    const int32_t *__restrict__ row_of, const float *__restrict__ weight, int64_t T, int k,
    const int32_t *__restrict__ row_token, const int32_t *__restrict__ offsets, int64_t E, void *__restrict__ grad_c,
    float *__restrict__ grad_weight) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const u32x4 zero = {0u, 0u, 0u, 0u};
    if ((int64_t)blockIdx.x >= T) {
        const int64_t used = offsets[E] < rows ? offsets[E] : rows;
        const int64_t r0 = ((int64_t)blockIdx.x - T) * kZeroRows;
        for (int i = wave; i < kZeroRows; i += 4) {
            const int64_t r = r0 + i;
            if (r >= used) break;
            const int64_t t = __builtin_amdgcn_readfirstlane(row_token[r]);
            if (t >= 0 && t < T) continue;
            u32x4 *to = static_cast<u32x4 *>(grad_c) + r * chunks;
            for (int64_t ch = lane; ch < chunks; ch += 64) to[ch] = zero;
        }
        return;
    }
    __shared__ float part[4][kSlots];
    const int64_t t = blockIdx.x;
    const u32x4 *g = static_cast<const u32x4 *>(grad_y) + t * chunks;
    for (int j0 = 0; j0 < k; j0 += kSlots) {
        int64_t row[kSlots];
        float w[kSlots], dot[kSlots];
#pragma unroll
        for (int u = 0; u < kSlots; u++) {
            const int64_t r = j0 + u < k ? row_of[t * k + j0 + u] : -1;  // the same in every lane
            row[u] = r >= 0 && r < rows ? r : -1;
            w[u] = row[u] >= 0 ? weight[t * k + j0 + u] : 0.0f;
            dot[u] = 0.0f;
        }
        for (int64_t ch = tid; ch < chunks; ch += 256) {
            Chunk<BF16> dy;
            dy.set(g[ch]);
            u32x4 v[kSlots];
#pragma unroll
            for (int u = 0; u < kSlots; u++)
                v[u] = row[u] >= 0 ? load_stream16(static_cast<const u32x4 *>(c) + row[u] * chunks + ch) : zero;
#pragma unroll
            for (int u = 0; u < kSlots; u++) {
                if (row[u] < 0) continue;  // the same in every lane
                Chunk<BF16> x, dc;
                x.set(v[u]);
#pragma unroll
                for (int i = 0; i < Chunk<BF16>::N; i++) {
                    dot[u] = __builtin_fmaf(x.f[i], dy.f[i], dot[u]);
                    dc.f[i] = w[u] * dy.f[i];
                }
                __builtin_nontemporal_store(dc.pack(), static_cast<u32x4 *>(grad_c) + row[u] * chunks + ch);
            }
        }
#pragma unroll
        for (int u = 0; u < kSlots; u++) {
            for (int d = 32; d > 0; d >>= 1) dot[u] += __shfl_xor(dot[u], d, 64);
            if (lane == 0) part[wave][u] = dot[u];
        }
        __syncthreads();
        if (tid < kSlots && j0 + tid < k)
            grad_weight[t * k + j0 + tid] = (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
        __syncthreads();
    }
}

}  // namespace

int64_t moe_combine_blocks(int64_t T, int64_t H, bool bf16) {
    const int64_t chunks = H / (bf16 ? 8 : 4);
    return T * ((chunks + 255) / 256);
}

hipError_t launch_moe_combine(const void *c, bool bf16, int64_t rows, int64_t H, const int32_t *row_of,
                              const float *weight, int64_t T, int k, const void *add, void *y, hipStream_t stream) {
    const int64_t chunks = H / (bf16 ? 8 : 4), spans = (chunks + 255) / 256;
    const dim3 grid((unsigned)(T * spans));
    if (bf16)
        moe_combine_kernel<true><<<grid, 256, 0, stream>>>(c, rows, chunks, spans, row_of, weight, k, add, y);
    else
        moe_combine_kernel<false><<<grid, 256, 0, stream>>>(c, rows, chunks, spans, row_of, weight, k, add, y);
    return hipGetLastError();
}

hipError_t launch_moe_combine_backward(const void *grad_y, const void *c, bool bf16, int64_t rows, int64_t H,
                                       const int32_t *row_of, const float *weight, int64_t T, int k,
                                       const int32_t *row_token, const int32_t *offsets, int64_t E, void *grad_c,
                                       float *grad_weight, hipStream_t stream) {
    const int64_t chunks = H / (bf16 ? 8 : 4);
    const dim3 grid((unsigned)(T + (rows + kZeroRows - 1) / kZeroRows));
    if (bf16)
        moe_combine_backward_kernel<true><<<grid, 256, 0, stream>>>(grad_y, c, rows, chunks, row_of, weight, T, k,
                                                                    row_token, offsets, E, grad_c, grad_weight);
    else
        moe_combine_backward_kernel<false><<<grid, 256, 0, stream>>>(grad_y, c, rows, chunks, row_of, weight, T, k,
                                                                     row_token, offsets, E, grad_c, grad_weight);
    return hipGetLastError();
}

}  // namespace fp8q
