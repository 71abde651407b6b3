// MoE gating: scores, group-limited top-k, weights, the expert-sorted layout, and the gradient of the weights.
//
// For token t with logits x_e (bf16 or fp32), clamped to the largest finite fp32:
//   s_e = 1 / (1 + exp(-x_e))                       (sigmoid), or
//   s_e = exp(x_e - max_e x) / sum_e exp(x_e - max) (softmax),
//   key_e = s_e + bias_e;  an expert whose logit is -inf or NaN is masked and never chosen.
// The E experts form n_group equal groups of consecutive experts; a group's value is the sum of its best
// group_top keys, and only the topk_group groups of largest value keep their experts.  The token takes the k
// largest remaining keys, best first, lower index first between equal keys (groups too); where fewer than k
// experts remain, the last slots are empty (expert -1, weight 0, row -1).  Its weights are
//   w_j = scale * s_j / (sum_i s_i + 1e-20)  (renormalized)   or   scale * s_j.
// What it moves is small (8192 x 256 fp32 logits: 8 MB, 2 us); it is bound by instructions and latency: the scores, then
// k rounds of a maximum over the token's lanes.  8192 tokens, 256 experts in 8 groups, k = 8: 11 us for the choice (1880
// VALU instructions a wave of 4 tokens, 2 waves a SIMD: the SIMDs issue them for 0.6 of the time, a wave waits for half of
// its time), 7.4 for the layout; 160 experts in 8 groups, 20 a group and so no vector loads, 12.8; one token 7.5 us in one
// launch (the latency of one wave, up to three round trips to memory in a row: logits, bias, the chosen logits again).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8q_device.h"
#include "fp8q_kernels.h"

namespace fp8q {
namespace {

constexpr int kGateChunk = 32;      // tokens per workgroup of the gating kernel, at most (a bit each in 32-bit masks)
constexpr int kGateThreads = 1024;  // of the kernels that build the layout
constexpr int kGateWaves = kGateThreads / 64;
constexpr float kWeightEps = 1e-20f;

__device__ __forceinline__ float bf16_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

// One DPP step over 32-bit values; lanes whose row is not in `rmask` keep `old`.
template <int CTRL, int RMASK>
__device__ __forceinline__ uint32_t dpp(uint32_t old, uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)old, (int)v, CTRL, RMASK, 0xF, false);
}

// Reductions over the LT lanes (16, a DPP row, or the whole wave) that share a token; every lane gets the result.  The sum
// is formed in one fixed order.
template <int LT>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
    v = row16_max(v);
    if constexpr (LT == 64) {
        v = max(v, dpp<0x142, 0xA>(v, v));  // lane 15 of a row to the next row
        v = max(v, dpp<0x143, 0xC>(v, v));  // lane 31 to rows 2 and 3
        v = (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
    }
    return v;
}
__device__ __forceinline__ uint32_t lanes_min16(uint32_t v) {
    v = min(v, dpp<0x128, 0xF>(v, v));
    v = min(v, dpp<0x124, 0xF>(v, v));
    v = min(v, dpp<0x122, 0xF>(v, v));
    return min(v, dpp<0x121, 0xF>(v, v));
}
template <int CTRL, int RMASK>
__device__ __forceinline__ float dpp_add(float f) {
    return f + __uint_as_float(dpp<CTRL, RMASK>(0, __float_as_uint(f)));
}
template <int LT>
__device__ __forceinline__ float lanes_sum(float f) {
    f = dpp_add<0x128, 0xF>(f);
    f = dpp_add<0x124, 0xF>(f);
    f = dpp_add<0x122, 0xF>(f);
    f = dpp_add<0x121, 0xF>(f);
    if constexpr (LT == 64) {
        f = dpp_add<0x142, 0xA>(f);
        f = dpp_add<0x143, 0xC>(f);
        f = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(f), 63));
    }
    return f;
}

// Sum of numbers in [0, 1] that does not depend on their order: each is rounded to a multiple of 2^-42 (1536 has the last
// bit 2^-42 in 53 bits), and up to 1024 such multiples add up exactly in 64-bit floats.  So a token's softmax is the same
// whatever lanes it is spread over.
__device__ __forceinline__ double multiple(float f) { return ((double)f + 1536.0) - 1536.0; }
template <int CTRL, int RMASK>
__device__ __forceinline__ double dpp_add(double d) {
    const uint64_t v = __builtin_bit_cast(uint64_t, d);
    const uint64_t o = (uint64_t)dpp<CTRL, RMASK>(0, (uint32_t)v) | (uint64_t)dpp<CTRL, RMASK>(0, (uint32_t)(v >> 32)) << 32;
    return d + __builtin_bit_cast(double, o);
}
template <int LT>
__device__ __forceinline__ float lanes_sum_exact(double d) {
    d = dpp_add<0x128, 0xF>(d);
    d = dpp_add<0x124, 0xF>(d);
    d = dpp_add<0x122, 0xF>(d);
    d = dpp_add<0x121, 0xF>(d);
    float f;
    if constexpr (LT == 64) {
        d = dpp_add<0x142, 0xA>(d);
        d = dpp_add<0x143, 0xC>(d);
        f = (float)d;
        f = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(f), 63));
    } else {
        f = (float)d;
    }
    return f;
}

// e^x for x <= 0 to about 2 units in the last place: 2^(x log2 e) with the product's rounding error carried along (log2 e
// as a sum of two floats), scaled so that results below the normal range keep their bits.
__device__ __forceinline__ float exp_neg(float x) {
    x = fmaxf(x, -150.0f);  // e^-150 is 0 in fp32
    const float hi = x * 1.44269502f;
    const float lo = __builtin_fmaf(x, 1.44269502f, -hi) + x * 1.92596299e-8f;
    const bool small = hi < -120.0f;
    const float e = __builtin_amdgcn_exp2f(small ? hi + 64.0f : hi);
    const float y = __builtin_fmaf(e * lo, 0.693147182f, e);
    return small ? y * 5.42101086e-20f : y;  // 2^-64
}
// 1 / d for d in [1, 2], or any d whose reciprocal and itself are normal.
__device__ __forceinline__ float reciprocal(float d) {
    const float r = __builtin_amdgcn_rcpf(d);
    return __builtin_fmaf(r, __builtin_fmaf(-d, r, 1.0f), r);
}
// 1 / (1 + e^-x), from e^-|x| so that nothing overflows.
__device__ __forceinline__ float sigmoid(float x) {
    const float e = exp_neg(-fabsf(x));
    const float r = reciprocal(1.0f + e);
    return x >= 0.0f ? r : e * r;
}

// Keys as unsigned integers in the order of the floats (-0 equals +0); 0 is below every key: a masked expert.
__device__ __forceinline__ uint32_t sort_key(float f) {
    const uint32_t b = __float_as_uint(f + 0.0f);
    return b ^ (((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unsort_key(uint32_t u) {
    return __uint_as_float(u ^ (((int32_t)~u >> 31) | 0x80000000u));
}

__device__ __forceinline__ float load_logit(const void *p, int64_t i, bool bf16) {
    return bf16 ? bf16_f32(static_cast<const uint16_t *>(p)[i]) : static_cast<const float *>(p)[i];
}

// Clamped logit; -inf for a masked expert (NaN, -inf).
__device__ __forceinline__ float clean_logit(float x) {
    return x > -__builtin_inff() ? fminf(x, 3.4028234663852886e38f) : -__builtin_inff();
}

struct GateArgs {
    const void *logits;
    const float *bias;
    int64_t ld, T;
    int E, k, G, topk_group, group_top;
    int lanes_per_group;  // LT / (n_group rounded up to a power of two)
    float scale;
    bool bf16, softmax, renorm;
    // Lanes hold R experts or none, and their logits (biases) lie at multiples of their size, or of 16 bytes.
    bool vec, vec_bias;
};

// SIZE bytes in pieces of at most 16, each aligned to its size.
template <int SIZE>
__device__ __forceinline__ void copy_aligned(void *to, const void *from) {
    constexpr int A = SIZE < 16 ? SIZE : 16;
#pragma unroll
    for (int i = 0; i < SIZE; i += A)
        __builtin_memcpy(static_cast<char *>(to) + i,
                         __builtin_assume_aligned(static_cast<const char *>(from) + i, A), A);
}

// R consecutive logits from element `at` on, `n` of them valid (with a.vec: all or none); -inf for the others.
template <int R>
__device__ __forceinline__ void load_logits(const GateArgs &a, int64_t at, int n, float (&x)[R]) {
    const float ninf = -__builtin_inff();
    if (!a.vec) {
#pragma unroll
        for (int r = 0; r < R; r++) x[r] = r < n ? clean_logit(load_logit(a.logits, at + r, a.bf16)) : ninf;
        return;
    }
#pragma unroll
    for (int r = 0; r < R; r++) x[r] = ninf;
    if (n <= 0) return;
    if (a.bf16) {
        uint16_t h[R];
        copy_aligned<2 * R>(h, static_cast<const uint16_t *>(a.logits) + at);
#pragma unroll
        for (int r = 0; r < R; r++) x[r] = clean_logit(bf16_f32(h[r]));
    } else {
        float f[R];
        copy_aligned<4 * R>(f, static_cast<const float *>(a.logits) + at);
#pragma unroll
        for (int r = 0; r < R; r++) x[r] = clean_logit(f[r]);
    }
}

// LT lanes choose the experts of one token, so a wave those of 64 / LT tokens.  Lane `in` of them holds up to R
// consecutive experts of group in / lanes_per_group, so (lane, register) order is expert order.  Lane j < k returns slot
// j's expert and weight.  Every lane of the wave takes part; `valid` is false in the lanes of tokens past the last.
template <int LT, int R>
__device__ __forceinline__ void gate_token(const GateArgs &a, int64_t t, bool valid, int lane, int &idx, float &weight) {
    const int in = lane % LT;
    const int L = a.lanes_per_group;
    const int gs = a.E / a.G;
    const int g = in / L;
    const int in0 = (in % L) * R;  // first expert of the lane within its group
    const int e0 = g * gs + in0;
    const float ninf = -__builtin_inff();
    float x[R];
    load_logits<R>(a, t * a.ld + e0, valid && g < a.G ? gs - in0 : 0, x);
    float m = 0.0f, inv = 1.0f;
    if (a.softmax) {
        m = ninf;
#pragma unroll
        for (int r = 0; r < R; r++) m = fmaxf(m, x[r]);
        m = fmaxf(unsort_key(lanes_max<LT>(sort_key(m))), -3.4028234663852886e38f);
    }
    uint32_t key[R];
    uint32_t gone = 0;
    double sum = 0.0;
#pragma unroll
    for (int r = 0; r < R; r++) {
        gone |= x[r] == ninf ? 1u << r : 0u;
        if (a.softmax) {
            x[r] = x[r] == ninf ? 0.0f : exp_neg(x[r] - m);
            sum += multiple(x[r]);
        } else {
            x[r] = sigmoid(x[r]);
        }
    }
    if (a.softmax) inv = reciprocal(fmaxf(lanes_sum_exact<LT>(sum), 1e-30f));
    float b[R];
#pragma unroll
    for (int r = 0; r < R; r++) b[r] = 0.0f;
    if (a.bias != nullptr && g < a.G) {
        if (a.vec_bias) {
            if (in0 < gs) copy_aligned<4 * R>(b, a.bias + e0);
        } else {
#pragma unroll
            for (int r = 0; r < R; r++)
                if (in0 + r < gs) b[r] = a.bias[e0 + r];
        }
    }
#pragma unroll
    for (int r = 0; r < R; r++) key[r] = (gone >> r) & 1u ? 0u : sort_key(__builtin_fmaf(x[r], inv, b[r]));
    if (a.topk_group < a.G) {
        // The group's two largest keys, over the lane's registers and then over its lanes (which are an aligned power of
        // two: once the quads agree, mirrored lanes are in the other half).
        uint32_t k1 = 0, k2 = 0;
#pragma unroll
        for (int r = 0; r < R; r++) {
            k2 = max(k2, min(k1, key[r]));
            k1 = max(k1, key[r]);
        }
        auto merge = [&](uint32_t o1, uint32_t o2) {
            k2 = max(max(k2, o2), min(k1, o1));
            k1 = max(k1, o1);
        };
        if (L > 1) merge(dpp<0xB1, 0xF>(0, k1), dpp<0xB1, 0xF>(0, k2));    // lane ^ 1
        if (L > 2) merge(dpp<0x4E, 0xF>(0, k1), dpp<0x4E, 0xF>(0, k2));    // lane ^ 2
        if (L > 4) merge(dpp<0x141, 0xF>(0, k1), dpp<0x141, 0xF>(0, k2));  // mirrored within 8
        if (L > 8) merge(dpp<0x140, 0xF>(0, k1), dpp<0x140, 0xF>(0, k2));  // mirrored within 16
        if (LT > 16 && L > 16) merge((uint32_t)__shfl_xor((int)k1, 16, 64), (uint32_t)__shfl_xor((int)k2, 16, 64));
        float v = k1 ? unsort_key(k1) : ninf;
        if (a.group_top == 2 && k2) v += unsort_key(k2);
        int before = 0;  // groups ahead of this lane's
        for (int h = 0; h < a.G; h++) {
            const float o = LT == 64 ? __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), h * L))
                                     : __shfl(v, (lane - in) + h * L, 64);
            before += o > v || (o == v && h < g) ? 1 : 0;
        }
        if (before >= a.topk_group) {
#pragma unroll
            for (int r = 0; r < R; r++) key[r] = 0;
        }
    }
    // k rounds: the largest key over the lanes, then the lowest expert that has it; its lane takes it out.
    idx = -1;
    uint32_t best = 0;
    int at = 0;
#pragma unroll
    for (int r = 0; r < R; r++) {
        at = key[r] > best ? r : at;
        best = max(best, key[r]);
    }
    for (int j = 0; j < a.k; j++) {
        const uint32_t top = lanes_max<LT>(best);
        uint32_t e;
        if constexpr (LT == 64) {
            const uint64_t have = __ballot(best == top && top != 0);  // the first lane's expert is the lowest
            e = have ? (uint32_t)__builtin_amdgcn_readlane(e0 + at, __builtin_ctzll(have)) : 0xFFFFFFFFu;
        } else {
            e = lanes_min16(best == top && top != 0 ? (uint32_t)(e0 + at) : 0xFFFFFFFFu);
        }
        idx = in == j ? (int)e : idx;  // -1 when no expert is left
        if (best != 0 && e == (uint32_t)(e0 + at)) {
            uint32_t nb = 0;
            int na = 0;
#pragma unroll
            for (int r = 0; r < R; r++) {
                key[r] = r == at ? 0u : key[r];
                na = key[r] > nb ? r : na;
                nb = max(nb, key[r]);
            }
            best = nb;
            at = na;
        }
    }
    // Slot j's score once more from its logit (the keys hold score plus bias), the same arithmetic as above.
    float score = 0.0f;
    if (idx >= 0) {
        const float y = clean_logit(load_logit(a.logits, t * a.ld + idx, a.bf16));
        score = a.softmax ? exp_neg(y - m) * inv : sigmoid(y);
    }
    // (the slots are lanes 0 .. 15 of the token's: one DPP row)
    weight = a.renorm ? a.scale * (score * reciprocal(lanes_sum<16>(score) + kWeightEps)) : a.scale * score;
}

struct LayoutArgs {
    int32_t *topk_idx;
    float *topk_weight;
    int32_t *offsets, *row_of, *row_token, *load;
    uint8_t *counts;  // [chunks][E rounded up to 4]: tokens of the chunk that chose the expert (at most 32)
    int64_t rows;
};

// Segment starts from the experts' totals: seg[e] and seg[E], each segment padded to 128 rows.  Called by a
// whole workgroup of kGateThreads; `wsum` holds kGateWaves integers.
__device__ __forceinline__ void scan_segments(const int32_t *total, int E, int32_t *seg, int32_t *wsum) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int32_t v = tid < E ? (total[tid] + 127) / 128 * 128 : 0;
    const int32_t own = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t u = __shfl_up(v, d, 64);
        if (lane >= d) v += u;
    }
    if (lane == 63) wsum[wave] = v;
    __syncthreads();
    int32_t pre = 0;
    for (int w = 0; w < wave; w++) pre += wsum[w];
    if (tid < E) seg[tid] = pre + v - own;
    if (tid == E - 1) seg[E] = pre + v;
    __syncthreads();
}

// -1 into the rows that no token has: the ends of the segments and everything from seg[E] on.  Workgroup `part`
// of `parts` does its share.  (A workspace that another call overwrites gives other counts: no store leaves row_token.)
__device__ __forceinline__ void fill_empty(const LayoutArgs &o, const int32_t *seg, const int32_t *total, int E,
                                           int part, int parts) {
    const int tid = threadIdx.x;
    const int n = (E - part + parts - 1) / parts;  // experts part, part + parts, ...
    for (int q = tid; q < n * 128; q += kGateThreads) {
        const int e = part + parts * (q >> 7);
        const int64_t r = (int64_t)seg[e] + total[e] + (q & 127);
        if (r < seg[e + 1] && (uint64_t)r < (uint64_t)o.rows) o.row_token[r] = -1;
    }
    // seg[E] is a multiple of 128
    const int64_t r0 = seg[E] > 0 ? seg[E] : 0;
    if ((reinterpret_cast<uintptr_t>(o.row_token) & 15u) == 0) {
        const i32x4 none = {-1, -1, -1, -1};
        for (int64_t r = r0 + ((int64_t)part * kGateThreads + tid) * 4; r < o.rows; r += (int64_t)parts * kGateThreads * 4) {
            if (r + 4 <= o.rows)
                *reinterpret_cast<i32x4 *>(o.row_token + r) = none;
            else
                for (int64_t i = r; i < o.rows; i++) o.row_token[i] = -1;
        }
    } else {
        for (int64_t r = r0 + (int64_t)part * kGateThreads + tid; r < o.rows; r += (int64_t)parts * kGateThreads)
            o.row_token[r] = -1;
    }
}

// Gating of one chunk of tokens per workgroup.  Each token sets its bit in the 32-bit LDS mask of every expert
// it chose; its rank among the chunk's tokens of that expert is the number of bits below its own, whatever the
// order in which the bits arrived.
// ONE: all tokens fit in one chunk.  Every workgroup then gates all of them (which costs less than a second
// launch), workgroup 0 writes the outputs, and all of them share the filling of the empty rows.
template <int LT, int R, bool ONE, int THREADS, int CHUNK>
__global__ __launch_bounds__(THREADS) void moe_gate_kernel(GateArgs a, LayoutArgs o) {
    constexpr int kAtOnce = THREADS / LT;  // tokens
    constexpr int kPasses = CHUNK / kAtOnce;
    static_assert(kPasses * kAtOnce == CHUNK && (!ONE || THREADS == kGateThreads), "tokens");
    __shared__ uint32_t mask[kMoeMaxExperts];
    __shared__ int32_t total[ONE ? kMoeMaxExperts : 1];
    __shared__ int32_t seg[ONE ? kMoeMaxExperts + 1 : 1];
    __shared__ int32_t wsum[kGateWaves];
    const int tid = threadIdx.x, lane = tid & 63, in = tid % LT;
    const int64_t c = ONE ? 0 : blockIdx.x;
    const bool writer = !ONE || blockIdx.x == 0;
    const int cols = (a.E + 3) / 4;
    for (int e = tid; e < 4 * cols; e += THREADS) mask[e] = 0u;
    __syncthreads();
    int idx[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; i++) {
        const int tl = i * kAtOnce + tid / LT;
        const int64_t t = c * CHUNK + tl;
        const bool valid = t < a.T;
        idx[i] = -1;
        if (__ballot(valid) == 0) continue;
        float w;
        gate_token<LT, R>(a, t, valid, lane, idx[i], w);
        if (valid && in < a.k) {
            if (idx[i] >= 0) atomicOr(&mask[idx[i]], 1u << tl);
            if (writer) {
                o.topk_idx[t * a.k + in] = idx[i];
                o.topk_weight[t * a.k + in] = w;
            }
        }
    }
    __syncthreads();
    if constexpr (ONE) {
        if (tid < a.E) total[tid] = __popc(mask[tid]);
        __syncthreads();
        scan_segments(total, a.E, seg, wsum);
        fill_empty(o, seg, total, a.E, blockIdx.x, gridDim.x);
        if (!writer) return;
        if (tid < a.E) {
            o.offsets[tid] = seg[tid];
            if (o.load != nullptr) o.load[tid] = total[tid];
        }
        if (tid == 0) o.offsets[a.E] = seg[a.E];
    } else {
        if (tid < cols) {
            uint32_t packed = 0;
#pragma unroll
            for (int i = 0; i < 4; i++) packed |= (uint32_t)__popc(mask[4 * tid + i]) << (8 * i);
            reinterpret_cast<uint32_t *>(o.counts)[c * cols + tid] = packed;
        }
    }
#pragma unroll
    for (int i = 0; i < kPasses; i++) {
        const int tl = i * kAtOnce + tid / LT;
        const int64_t t = c * CHUNK + tl;
        if (t >= a.T || in >= a.k) continue;
        int32_t r = idx[i] >= 0 ? __popc(mask[idx[i]] & ((1u << tl) - 1u)) : -1;
        if constexpr (ONE) {
            if (r >= 0) {
                r += seg[idx[i]];
                if (r < o.rows) o.row_token[r] = (int32_t)t;
            }
        }
        o.row_of[t * a.k + in] = r;  // without ONE: the rank within the chunk, finished by the layout kernel
    }
}

// The layout from the chunks' counts.  Every workgroup adds up the counts of all chunks (bytes, in parts that
// its threads share), which gives the totals, the segment starts and the counts before its own chunks; it then
// places the tokens of its chunks [c0, c1) and does its share of the empty rows.
__global__ __launch_bounds__(kGateThreads) void moe_gate_layout_kernel(LayoutArgs o, int64_t T, int64_t C, int E,
                                                                       int k, int chunk, int64_t chunks_per_wg) {
    __shared__ int32_t part_all[4096], part_before[4096];
    __shared__ int32_t total[kMoeMaxExperts], base[kMoeMaxExperts];
    __shared__ int32_t seg[kMoeMaxExperts + 1];
    __shared__ int32_t wsum[kGateWaves];
    const int tid = threadIdx.x;
    const int cols = (E + 3) / 4;
    const int P = kGateThreads / cols < 16 ? kGateThreads / cols : 16;  // P * cols <= 1024
    const int64_t c0 = (int64_t)blockIdx.x * chunks_per_wg;
    const int64_t c1 = c0 + chunks_per_wg < C ? c0 + chunks_per_wg : C;
    const uint32_t *counts = reinterpret_cast<const uint32_t *>(o.counts);
    const int col = tid % cols, p = tid / cols;
    // The first chunk's slots (at most 512), loaded here so that their latency passes beside the counts'.
    const int64_t first = c0 * chunk * k + tid;
    const bool has = first < T * k && tid < chunk * k;
    const int first_e = has ? o.topk_idx[first] : -1, first_r = has ? o.row_of[first] : 0;
    if (p < P) {
        int32_t all[4] = {0, 0, 0, 0}, before[4] = {0, 0, 0, 0};
        for (int64_t c = p; c < C; c += (int64_t)8 * P) {  // 8 loads in flight
            uint32_t v[8];
#pragma unroll
            for (int u = 0; u < 8; u++) {
                const int64_t cc = c + (int64_t)u * P;
                v[u] = cc < C ? counts[cc * cols + col] : 0u;
            }
#pragma unroll
            for (int u = 0; u < 8; u++)
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int32_t n = (int32_t)((v[u] >> (8 * i)) & 255u);
                    all[i] += n;
                    before[i] += c + (int64_t)u * P < c0 ? n : 0;
                }
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
            part_all[(p * cols + col) * 4 + i] = all[i];
            part_before[(p * cols + col) * 4 + i] = before[i];
        }
    }
    __syncthreads();
    int32_t mine = 0;
    if (tid < E) {
        int32_t sum = 0;
        for (int q = 0; q < P; q++) {
            sum += part_all[q * cols * 4 + tid];
            mine += part_before[q * cols * 4 + tid];
        }
        total[tid] = sum;
    }
    __syncthreads();
    scan_segments(total, E, seg, wsum);
    if (tid < E) base[tid] = seg[tid] + mine;
    if (blockIdx.x == 0) {
        if (tid < E) {
            o.offsets[tid] = seg[tid];
            if (o.load != nullptr) o.load[tid] = total[tid];
        }
        if (tid == 0) o.offsets[E] = seg[E];
    }
    fill_empty(o, seg, total, E, blockIdx.x, gridDim.x);
    __syncthreads();
    for (int64_t c = c0; c < c1; c++) {
        const int64_t t0 = c * chunk;
        const int n = (int)((T - t0 < chunk ? T - t0 : chunk) * k);
        for (int i = tid; i < n; i += kGateThreads) {
            const int64_t at = t0 * k + i;
            const int e = c == c0 ? first_e : o.topk_idx[at];
            if (e < 0) continue;  // an empty slot: its row is already -1
            const int32_t r = base[e] + (c == c0 ? first_r : o.row_of[at]);
            o.row_of[at] = r;
            if ((uint64_t)(int64_t)r < (uint64_t)o.rows) o.row_token[r] = (int32_t)(t0 + i / k);
        }
        if (c + 1 < c1) {
            __syncthreads();
            if (tid < E) base[tid] += o.counts[c * cols * 4 + tid];
            __syncthreads();
        }
    }
}

// The gradient of the logits, LT lanes per token, R consecutive experts a lane.  With d_j = scale * grad_weight_j and v_j
// the chosen scores, renormalized weights give ds_j = (d_j - sum_i d_i v_i / S) / S, S = sum_i v_i + 1e-20, the others
// ds_j = d_j; then dx = ds s (1 - s) for sigmoid (1 - s as the sigmoid of -x: no cancellation), and for softmax dx = s
// (ds - c), c = sum_j ds_j v_j, which under renormalization is D / S * 1e-20 / S with D = sum_j d_j v_j (its two terms
// cancel).  The bias only takes part in the choice and has no gradient.  Masked experts get 0.  8192 x 64 bf16: 4.4 us, of
// which 2.6 MB take half a us: launch and latency (one wave a token: 6.4 us).
template <int LT, int R>
__global__ __launch_bounds__(256) void moe_gate_backward_kernel(GateArgs a, const int32_t *__restrict__ topk_idx,
                                                                const float *__restrict__ grad_weight,
                                                                void *__restrict__ grad_logits, bool vec_out) {
    const int lane = threadIdx.x & 63, in = lane % LT;
    const int64_t t = (int64_t)blockIdx.x * (256 / LT) + threadIdx.x / LT;
    const bool valid = t < a.T;
    const float ninf = -__builtin_inff();
    const int e0 = in * R;
    float x[R];
    load_logits<R>(a, t * a.ld + e0, valid ? a.E - e0 : 0, x);
    // The chosen slots, one per lane.
    int idx = -1;
    float d = 0.0f, y = ninf;
    if (valid && in < a.k) {
        idx = topk_idx[t * a.k + in];
        if (idx < 0 || idx >= a.E) {
            idx = -1;
        } else {
            d = a.scale * grad_weight[t * a.k + in];
            y = clean_logit(load_logit(a.logits, t * a.ld + idx, a.bf16));
        }
    }
    float m = 0.0f, inv = 1.0f;
    if (a.softmax) {
        m = x[0];
#pragma unroll
        for (int r = 1; r < R; r++) m = fmaxf(m, x[r]);
        m = fmaxf(unsort_key(lanes_max<LT>(sort_key(m))), -3.4028234663852886e38f);
        double sum = 0.0;
#pragma unroll
        for (int r = 0; r < R; r++) sum += multiple(exp_neg(x[r] - m));
        inv = reciprocal(fmaxf(lanes_sum_exact<LT>(sum), 1e-30f));
    }
    const float v = idx < 0 ? 0.0f : (a.softmax ? exp_neg(y - m) * inv : sigmoid(y));
    // (the slots are lanes 0 .. 15 of the token's: one DPP row; the others take the sums from there)
    float D = lanes_sum<16>(d * v), S = lanes_sum<16>(v) + kWeightEps;
    if constexpr (LT == 64) {
        D = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(D), 0));
        S = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(S), 0));
    }
    float c = D;
    if (a.renorm) {
        d = (d - D / S) / S;
        c = D / S * (kWeightEps / S);
    }
    float ds[R];
#pragma unroll
    for (int r = 0; r < R; r++) ds[r] = 0.0f;
    for (int j = 0; j < a.k; j++) {
        const int e = LT == 64 ? __builtin_amdgcn_readlane(idx, j) : __shfl(idx, (lane - in) + j, 64);
        const float dj = LT == 64 ? __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(d), j))
                                  : __shfl(d, (lane - in) + j, 64);
#pragma unroll
        for (int r = 0; r < R; r++) ds[r] = e0 + r == e ? dj : ds[r];
    }
    float out[R];
#pragma unroll
    for (int r = 0; r < R; r++) {
        if (a.softmax)
            out[r] = exp_neg(x[r] - m) * inv * (ds[r] - c);
        else
            out[r] = ds[r] * sigmoid(x[r]) * sigmoid(-x[r]);
        out[r] = x[r] > ninf ? out[r] : 0.0f;
    }
    if (!valid || e0 >= a.E) return;
    const int64_t at = t * a.E + e0;
    if (a.bf16) {
        uint16_t h[R];
#pragma unroll
        for (int r = 0; r < R; r++) h[r] = (uint16_t)pack_bf16x2(out[r], out[r]);
        uint16_t *to = static_cast<uint16_t *>(grad_logits) + at;
        if (vec_out) {
            constexpr int A = 2 * R < 16 ? 2 * R : 16;
#pragma unroll
            for (int i = 0; i < 2 * R; i += A)
                __builtin_memcpy(__builtin_assume_aligned(reinterpret_cast<char *>(to) + i, A),
                                 reinterpret_cast<const char *>(h) + i, A);
            return;
        }
#pragma unroll
        for (int r = 0; r < R; r++)
            if (e0 + r < a.E) to[r] = h[r];
    } else {
        float *to = static_cast<float *>(grad_logits) + at;
        if (vec_out) {
            constexpr int A = 4 * R < 16 ? 4 * R : 16;
#pragma unroll
            for (int i = 0; i < 4 * R; i += A)
                __builtin_memcpy(__builtin_assume_aligned(reinterpret_cast<char *>(to) + i, A),
                                 reinterpret_cast<const char *>(out) + i, A);
            return;
        }
#pragma unroll
        for (int r = 0; r < R; r++)
            if (e0 + r < a.E) to[r] = out[r];
    }
}

// Experts a lane holds, for n experts over `lanes` lanes: the next power of two.
int regs_for(int n, int lanes) {
    int r = 1;
    while (r * lanes < n) r *= 2;
    return r;
}

GateArgs gate_args(const GateShape &g, int lanes) {
    int pow2 = 1;
    while (pow2 < g.n_group) pow2 *= 2;
    GateArgs a;
    a.logits = g.logits;
    a.bias = g.bias;
    a.ld = g.ld;
    a.T = g.T;
    a.E = g.E;
    a.k = g.k;
    a.G = g.n_group;
    a.topk_group = g.topk_group;
    a.group_top = g.group_top;
    a.lanes_per_group = lanes / pow2;
    a.scale = g.scale;
    a.bf16 = g.bf16;
    a.softmax = g.softmax;
    a.renorm = g.renorm;
    a.vec = a.vec_bias = false;
    return a;
}

// Whether lanes that take R of every `n` elements of rows `ld` elements apart hold R or none, at addresses aligned to
// their size or 16 bytes.
bool lanes_aligned(const void *p, int64_t ld, int n, int R, bool bf16) {
    const int64_t size = bf16 ? 2 : 4, A = R * size < 16 ? R * size : 16;
    return n % R == 0 && (ld * size) % A == 0 && reinterpret_cast<uintptr_t>(p) % (uintptr_t)A == 0;
}

}  // namespace

namespace {
int64_t counts_bytes(int64_t T, int64_t E, int64_t chunk) { return (T + chunk - 1) / chunk * ((E + 3) / 4 * 4); }
// Tokens per workgroup: 16 while that gives every CU at most one workgroup, if the counts' rows need no padding (so that
// the workspace stays within the other routing's) and the workspace holds them, else 32.  (256 experts in 8 groups, both
// launches: 2048 tokens 14.1 us by 16, 16.1 by 32; 4096 tokens 15.8 and 16.7.)
int chunk_tokens(int64_t T, int64_t E, int64_t workspace_bytes) {
    return T <= 4096 && E % 4 == 0 && counts_bytes(T, E, 16) <= workspace_bytes ? 16 : kGateChunk;
}
}  // namespace

int64_t moe_gate_workspace_bytes(int64_t T, int64_t E) {
    return T <= kGateChunk ? 0 : counts_bytes(T, E, chunk_tokens(T, E, INT64_MAX));
}
int64_t moe_gate_least_workspace_bytes(int64_t T, int64_t E) {
    return T <= kGateChunk ? 0 : counts_bytes(T, E, kGateChunk);
}

hipError_t launch_moe_gate_topk(const GateShape &g, int32_t *topk_idx, float *topk_weight, int32_t *offsets,
                                int32_t *row_of, int32_t *row_token, int64_t rows, int32_t *load, void *workspace,
                                int64_t workspace_bytes, hipStream_t stream) {
    const LayoutArgs o = {topk_idx, topk_weight, offsets, row_of, row_token, load, static_cast<uint8_t *>(workspace),
                          rows};
    const bool one = g.T <= kGateChunk;
    const int chunk = one ? kGateChunk : chunk_tokens(g.T, g.E, workspace_bytes);
    const int64_t C = (g.T + chunk - 1) / chunk;
    // A few tokens: 64 lanes each, the shortest way to an answer.  Many: 16 lanes each, which takes half the instructions
    // (8192 tokens, 256 experts: 15.4 us by 64 lanes, 11.0 by 16), where a lane then holds at most 32 experts.
    GateArgs a = gate_args(g, 16);
    const bool narrow = chunk == kGateChunk && !one && a.lanes_per_group >= 1 &&
                        regs_for(g.E / g.n_group, a.lanes_per_group) <= 32;
    if (!narrow) a = gate_args(g, 64);
    const int R = regs_for(g.E / g.n_group, a.lanes_per_group);
    a.vec = lanes_aligned(g.logits, g.ld, g.E / g.n_group, R, g.bf16);
    a.vec_bias = lanes_aligned(g.bias, 0, g.E / g.n_group, R, false);
    // One chunk: a workgroup for every 2048 rows to fill, at most 32.
    const int64_t blocks = one ? (rows / 2048 < 1 ? 1 : (rows / 2048 > 32 ? 32 : rows / 2048)) : C;
    const dim3 grid((unsigned)blocks);
    switch (R) {
#define FP8Q_GATE_CASE(N)                                                                          \
    case N:                                                                                        \
        if (one)                                                                                   \
            moe_gate_kernel<64, N, true, kGateThreads, 32><<<grid, kGateThreads, 0, stream>>>(a, o); \
        else if (narrow)                                                                           \
            moe_gate_kernel<16, N, false, 512, 32><<<grid, 512, 0, stream>>>(a, o);                \
        else if (chunk == 16)                                                                      \
            moe_gate_kernel<64, N, false, 1024, 16><<<grid, 1024, 0, stream>>>(a, o);              \
        else                                                                                       \
            moe_gate_kernel<64, N, false, 1024, 32><<<grid, 1024, 0, stream>>>(a, o);              \
        break;
        FP8Q_GATE_CASE(1)
        FP8Q_GATE_CASE(2)
        FP8Q_GATE_CASE(4)
        FP8Q_GATE_CASE(8)
        FP8Q_GATE_CASE(16)
        FP8Q_GATE_CASE(32)
#undef FP8Q_GATE_CASE
        default: return hipErrorInvalidValue;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;  // the layout reads what this launch counts
    if (!one) {
        const int64_t per = (C + 255) / 256;  // at most 256 workgroups: each reads all counts
        moe_gate_layout_kernel<<<dim3((unsigned)((C + per - 1) / per)), kGateThreads, 0, stream>>>(o, g.T, C, g.E, g.k,
                                                                                                   chunk, per);
    }
    return hipGetLastError();
}

hipError_t launch_moe_gate_backward(const GateShape &g, const int32_t *topk_idx, const float *grad_weight,
                                    void *grad_logits, hipStream_t stream) {
    // 16 lanes a token where a lane then holds at most 16 experts, else 64.
    const bool narrow = g.E <= 256;
    const int R = regs_for(g.E, narrow ? 16 : 64), per = narrow ? 16 : 4;
    GateArgs a = gate_args(g, 64);
    a.vec = lanes_aligned(g.logits, g.ld, g.E, R, g.bf16);
    const bool vec_out = lanes_aligned(grad_logits, g.E, g.E, R, g.bf16);
    const dim3 grid((unsigned)((g.T + per - 1) / per));
    switch (R) {
#define FP8Q_GATE_BWD_CASE(N)                                                                                    \
    case N:                                                                                                      \
        if (narrow)                                                                                              \
            moe_gate_backward_kernel<16, N><<<grid, 256, 0, stream>>>(a, topk_idx, grad_weight, grad_logits, vec_out); \
        else                                                                                                     \
            moe_gate_backward_kernel<64, N><<<grid, 256, 0, stream>>>(a, topk_idx, grad_weight, grad_logits, vec_out); \
        break;
        FP8Q_GATE_BWD_CASE(1)
        FP8Q_GATE_BWD_CASE(2)
        FP8Q_GATE_BWD_CASE(4)
        FP8Q_GATE_BWD_CASE(8)
        FP8Q_GATE_BWD_CASE(16)
#undef FP8Q_GATE_BWD_CASE
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace fp8q
