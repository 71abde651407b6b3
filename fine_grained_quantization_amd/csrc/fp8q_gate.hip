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
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8q_device.h"
#include "fp8q_kernels.h"

namespace fp8q {
namespace {

constexpr int kGateChunk = 32;   // tokens per workgroup: 16 waves, 2 tokens each
constexpr int kGateThreads = 1024;
constexpr int kGateWaves = kGateThreads / 64;
constexpr int kTokensPerWave = kGateChunk / kGateWaves;
constexpr float kWeightEps = 1e-20f;

__device__ __forceinline__ float bf16_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

// One DPP step over 32-bit values; lanes whose row is not in `rmask` keep `old`.
template <int CTRL, int RMASK>
__device__ __forceinline__ uint32_t dpp(uint32_t old, uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)old, (int)v, CTRL, RMASK, 0xF, false);
}

// Largest value of the wave, the same in every lane (a scalar).
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
    v = row16_max(v);
    v = max(v, dpp<0x142, 0xA>(v, v));  // lane 15 of a row to the next row
    v = max(v, dpp<0x143, 0xC>(v, v));  // lane 31 to rows 2 and 3
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// Sum over the wave, in one fixed order, the same in every lane.
__device__ __forceinline__ float wave_fsum(float f) {
    uint32_t v = __float_as_uint(f);
    f += __uint_as_float(dpp<0x128, 0xF>(0, v));
    v = __float_as_uint(f);
    f += __uint_as_float(dpp<0x124, 0xF>(0, v));
    v = __float_as_uint(f);
    f += __uint_as_float(dpp<0x122, 0xF>(0, v));
    v = __float_as_uint(f);
    f += __uint_as_float(dpp<0x121, 0xF>(0, v));
    v = __float_as_uint(f);
    f += __uint_as_float(dpp<0x142, 0xA>(0, v));
    v = __float_as_uint(f);
    f += __uint_as_float(dpp<0x143, 0xC>(0, v));
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(f), 63));
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
    int lanes_per_group;  // 64 / (n_group rounded up to a power of two)
    float scale;
    bool bf16, softmax, renorm;
};

// One wave chooses the experts of one token.  Lane l holds up to R consecutive experts of group l /
// lanes_per_group, so (lane, register) order is expert order.  Lane j < k returns slot j's expert and weight.
template <int R>
__device__ __forceinline__ void gate_token(const GateArgs &a, int64_t t, int lane, int &idx, float &weight) {
    const int L = a.lanes_per_group;
    const int gs = a.E / a.G;
    const int g = lane / L;
    const int in0 = (lane % L) * R;  // first expert of the lane within its group
    const int e0 = g * gs + in0;
    const float ninf = -__builtin_inff();
    float s[R];
#pragma unroll
    for (int r = 0; r < R; r++)
        s[r] = g < a.G && in0 + r < gs ? clean_logit(load_logit(a.logits, t * a.ld + e0 + r, a.bf16)) : ninf;
    uint32_t key[R];
    uint32_t gone = 0;
#pragma unroll
    for (int r = 0; r < R; r++) gone |= s[r] == ninf ? 1u << r : 0u;
    if (a.softmax) {
        float m = ninf;
#pragma unroll
        for (int r = 0; r < R; r++) m = fmaxf(m, s[r]);
        m = unsort_key(wave_umax(sort_key(m)));
        float sum = 0.0f;
#pragma unroll
        for (int r = 0; r < R; r++) {
            s[r] = (gone >> r) & 1u ? 0.0f : expf(s[r] - m);
            sum += s[r];
        }
        sum = fmaxf(wave_fsum(sum), 1e-30f);
#pragma unroll
        for (int r = 0; r < R; r++) s[r] = s[r] / sum;
    } else {
#pragma unroll
        for (int r = 0; r < R; r++) s[r] = 1.0f / (1.0f + expf(-s[r]));
    }
#pragma unroll
    for (int r = 0; r < R; r++) {
        const float b = a.bias != nullptr && !((gone >> r) & 1u) ? a.bias[e0 + r] : 0.0f;
        key[r] = (gone >> r) & 1u ? 0u : sort_key(s[r] + b);
    }
    if (a.topk_group < a.G) {
        // The group's two largest keys, over the lane's registers and then over its lanes.
        uint32_t k1 = 0, k2 = 0;
#pragma unroll
        for (int r = 0; r < R; r++) {
            k2 = max(k2, min(k1, key[r]));
            k1 = max(k1, key[r]);
        }
        for (int d = 1; d < L; d <<= 1) {
            const uint32_t o1 = (uint32_t)__shfl_xor((int)k1, d, 64), o2 = (uint32_t)__shfl_xor((int)k2, d, 64);
            k2 = max(max(k2, o2), min(k1, o1));
            k1 = max(k1, o1);
        }
        float v = k1 ? unsort_key(k1) : ninf;
        if (a.group_top == 2 && k2) v += unsort_key(k2);
        int before = 0;  // groups ahead of this lane's
        for (int h = 0; h < a.G; h++) {
            const float o = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), h * L));
            before += o > v || (o == v && h < g) ? 1 : 0;
        }
        if (before >= a.topk_group) {
#pragma unroll
            for (int r = 0; r < R; r++) key[r] = 0;
        }
    }
    idx = -1;
    float score = 0.0f, sum = 0.0f;
    uint32_t best = 0;
    int at = 0;
#pragma unroll
    for (int r = 0; r < R; r++) {
        at = key[r] > best ? r : at;
        best = max(best, key[r]);
    }
    for (int j = 0; j < a.k; j++) {
        const uint32_t top = wave_umax(best);
        if (top == 0) break;  // no expert is left
        const int owner = __builtin_ctzll(__ballot(best == top));
        float sc = 0.0f;
#pragma unroll
        for (int r = 0; r < R; r++) sc = r == at ? s[r] : sc;
        const int e = __builtin_amdgcn_readlane(e0 + at, owner);
        sc = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(sc), owner));
        sum += sc;
        idx = lane == j ? e : idx;
        score = lane == j ? sc : score;
        if (lane == owner) {
            uint32_t nb = 0;
            int na = 0;
#pragma unroll
            for (int r = 0; r < R; r++) {
                if (r == at) key[r] = 0;
                na = key[r] > nb ? r : na;
                nb = max(nb, key[r]);
            }
            best = nb;
            at = na;
        }
    }
    weight = a.renorm ? a.scale * (score / (sum + kWeightEps)) : a.scale * score;
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
// of `parts` does its share.
__device__ __forceinline__ void fill_empty(const LayoutArgs &o, const int32_t *seg, const int32_t *total, int E,
                                           int part, int parts) {
    const int tid = threadIdx.x;
    const int n = (E - part + parts - 1) / parts;  // experts part, part + parts, ...
    for (int q = tid; q < n * 128; q += kGateThreads) {
        const int e = part + parts * (q >> 7);
        const int64_t r = (int64_t)seg[e] + total[e] + (q & 127);
        if (r < seg[e + 1]) o.row_token[r] = -1;
    }
    // seg[E] is a multiple of 128
    const int64_t r0 = seg[E];
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
template <int R, bool ONE>
__global__ __launch_bounds__(kGateThreads) void moe_gate_kernel(GateArgs a, LayoutArgs o) {
    __shared__ uint32_t mask[kMoeMaxExperts];
    __shared__ int32_t total[ONE ? kMoeMaxExperts : 1];
    __shared__ int32_t seg[ONE ? kMoeMaxExperts + 1 : 1];
    __shared__ int32_t wsum[kGateWaves];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t c = ONE ? 0 : blockIdx.x;
    const bool writer = !ONE || blockIdx.x == 0;
    for (int e = tid; e < kMoeMaxExperts; e += kGateThreads) mask[e] = 0u;
    __syncthreads();
    int idx[kTokensPerWave];
#pragma unroll
    for (int i = 0; i < kTokensPerWave; i++) {
        const int tl = wave * kTokensPerWave + i;
        const int64_t t = c * kGateChunk + tl;
        idx[i] = -1;
        if (t >= a.T) continue;  // the same in every lane
        float w;
        gate_token<R>(a, t, lane, idx[i], w);
        if (lane < a.k) {
            if (idx[i] >= 0) atomicOr(&mask[idx[i]], 1u << tl);
            if (writer) {
                o.topk_idx[t * a.k + lane] = idx[i];
                o.topk_weight[t * a.k + lane] = w;
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
        const int cols = (a.E + 3) / 4;
        if (tid < cols) {
            uint32_t packed = 0;
#pragma unroll
            for (int i = 0; i < 4; i++) packed |= (uint32_t)__popc(mask[4 * tid + i]) << (8 * i);
            reinterpret_cast<uint32_t *>(o.counts)[c * cols + tid] = packed;
        }
    }
#pragma unroll
    for (int i = 0; i < kTokensPerWave; i++) {
        const int tl = wave * kTokensPerWave + i;
        const int64_t t = c * kGateChunk + tl;
        if (t >= a.T || lane >= a.k) continue;
        int32_t r = idx[i] >= 0 ? __popc(mask[idx[i]] & ((1u << tl) - 1u)) : -1;
        if constexpr (ONE) {
            if (r >= 0) {
                r += seg[idx[i]];
                if (r < o.rows) o.row_token[r] = (int32_t)t;
            }
        }
        o.row_of[t * a.k + lane] = r;  // without ONE: the rank within the chunk, finished by the layout kernel
    }
}

// The layout from the chunks' counts.  Every workgroup adds up the counts of all chunks (bytes, in parts that
// its threads share), which gives the totals, the segment starts and the counts before its own chunks; it then
// places the tokens of its chunks [c0, c1) and does its share of the empty rows.
__global__ __launch_bounds__(kGateThreads) void moe_gate_layout_kernel(LayoutArgs o, int64_t T, int64_t C, int E,
                                                                       int k, int64_t chunks_per_wg) {
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
        const int64_t t0 = c * kGateChunk;
        const int n = (int)((T - t0 < kGateChunk ? T - t0 : kGateChunk) * k);
        for (int i = tid; i < n; i += kGateThreads) {
            const int64_t at = t0 * k + i;
            const int e = o.topk_idx[at];
            if (e < 0) continue;  // an empty slot: its row is already -1
            const int32_t r = base[e] + o.row_of[at];
            o.row_of[at] = r;
            if (r < o.rows) o.row_token[r] = (int32_t)(t0 + i / k);
        }
        if (c + 1 < c1) {
            __syncthreads();
            if (tid < E) base[tid] += o.counts[c * cols * 4 + tid];
            __syncthreads();
        }
    }
}

// The gradient of the logits, one wave per token.  With d_j = scale * grad_weight_j and v_j the chosen scores,
// renormalized weights give ds_j = (d_j - sum_i d_i v_i / S) / S, S = sum_i v_i + 1e-20, the others ds_j = d_j;
// then dx = ds s (1 - s) for sigmoid (1 - s as the sigmoid of -x: no cancellation), and for softmax dx = s (ds - c),
// c = sum_j ds_j v_j, which under renormalization is D / S * 1e-20 / S with D = sum_j d_j v_j (its two terms cancel).
// The bias only takes part in the choice and has no gradient.  Masked experts get 0.
template <int R>
__global__ __launch_bounds__(256) void moe_gate_backward_kernel(GateArgs a, const int32_t *__restrict__ topk_idx,
                                                                const float *__restrict__ grad_weight,
                                                                void *__restrict__ grad_logits) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    if (t >= a.T) return;
    const float ninf = -__builtin_inff();
    const int e0 = lane * R;
    float x[R];
#pragma unroll
    for (int r = 0; r < R; r++)
        x[r] = e0 + r < a.E ? clean_logit(load_logit(a.logits, t * a.ld + e0 + r, a.bf16)) : ninf;
    float m = 0.0f, sum = 1.0f;
    if (a.softmax) {
        m = x[0];
#pragma unroll
        for (int r = 1; r < R; r++) m = fmaxf(m, x[r]);
        m = fmaxf(unsort_key(wave_umax(sort_key(m))), -3.4028234663852886e38f);
        sum = 0.0f;
#pragma unroll
        for (int r = 0; r < R; r++) sum += expf(x[r] - m);
        sum = fmaxf(wave_fsum(sum), 1e-30f);
    }
    // The chosen slots, one per lane.
    int idx = -1;
    float d = 0.0f, v = 0.0f;
    if (lane < a.k) {
        idx = topk_idx[t * a.k + lane];
        if (idx < 0 || idx >= a.E) {
            idx = -1;
        } else {
            d = a.scale * grad_weight[t * a.k + lane];
            const float y = clean_logit(load_logit(a.logits, t * a.ld + idx, a.bf16));
            v = a.softmax ? expf(y - m) / sum : 1.0f / (1.0f + expf(-y));
        }
    }
    const float D = wave_fsum(d * v);
    float c = D;
    if (a.renorm) {
        const float S = wave_fsum(v) + kWeightEps;
        d = (d - D / S) / S;
        c = D / S * (kWeightEps / S);
    }
    float ds[R];
#pragma unroll
    for (int r = 0; r < R; r++) ds[r] = 0.0f;
    for (int j = 0; j < a.k; j++) {
        const int e = __builtin_amdgcn_readlane(idx, j);
        const float dj = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(d), j));
#pragma unroll
        for (int r = 0; r < R; r++) ds[r] = e0 + r == e ? dj : ds[r];
    }
#pragma unroll
    for (int r = 0; r < R; r++) {
        if (e0 + r >= a.E) continue;
        float out = 0.0f;
        if (x[r] > ninf) {
            if (a.softmax)
                out = expf(x[r] - m) / sum * (ds[r] - c);
            else
                out = ds[r] * (1.0f / (1.0f + expf(-x[r]))) * (1.0f / (1.0f + expf(x[r])));
        }
        if (a.bf16)
            static_cast<uint16_t *>(grad_logits)[t * a.E + e0 + r] = (uint16_t)pack_bf16x2(out, out);
        else
            static_cast<float *>(grad_logits)[t * a.E + e0 + r] = out;
    }
}

// Experts a lane holds, for n experts over `lanes` lanes: the next power of two.
int regs_for(int n, int lanes) {
    int r = 1;
    while (r * lanes < n) r *= 2;
    return r;
}

GateArgs gate_args(const GateShape &g) {
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
    a.lanes_per_group = 64 / pow2;
    a.scale = g.scale;
    a.bf16 = g.bf16;
    a.softmax = g.softmax;
    a.renorm = g.renorm;
    return a;
}

}  // namespace

int64_t moe_gate_workspace_bytes(int64_t T, int64_t E) {
    return T <= kGateChunk ? 0 : (T + kGateChunk - 1) / kGateChunk * ((E + 3) / 4 * 4);
}

hipError_t launch_moe_gate_topk(const GateShape &g, int32_t *topk_idx, float *topk_weight, int32_t *offsets,
                                int32_t *row_of, int32_t *row_token, int64_t rows, int32_t *load, void *workspace,
                                hipStream_t stream) {
    const GateArgs a = gate_args(g);
    const LayoutArgs o = {topk_idx, topk_weight, offsets, row_of, row_token, load, static_cast<uint8_t *>(workspace),
                          rows};
    const int R = regs_for(g.E / g.n_group, a.lanes_per_group);
    const int64_t C = (g.T + kGateChunk - 1) / kGateChunk;
    const bool one = C <= 1;
    // One chunk: a workgroup for every 4096 rows to fill, at most 16.
    const int64_t blocks = one ? (rows / 4096 < 1 ? 1 : (rows / 4096 > 16 ? 16 : rows / 4096)) : C;
    const dim3 grid((unsigned)blocks);
    switch (R) {
#define FP8Q_GATE_CASE(N)                                                          \
    case N:                                                                        \
        if (one)                                                                   \
            moe_gate_kernel<N, true><<<grid, kGateThreads, 0, stream>>>(a, o);     \
        else                                                                       \
            moe_gate_kernel<N, false><<<grid, kGateThreads, 0, stream>>>(a, o);    \
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
    if (!one) {
        const int64_t per = (C + 255) / 256;  // at most 256 workgroups: each reads all counts
        moe_gate_layout_kernel<<<dim3((unsigned)((C + per - 1) / per)), kGateThreads, 0, stream>>>(o, g.T, C, g.E, g.k,
                                                                                                   per);
    }
    return hipGetLastError();
}

hipError_t launch_moe_gate_backward(const GateShape &g, const int32_t *topk_idx, const float *grad_weight,
                                    void *grad_logits, hipStream_t stream) {
    const GateArgs a = gate_args(g);
    const dim3 grid((unsigned)((g.T + 3) / 4));
    switch (regs_for(g.E, 64)) {
#define FP8Q_GATE_BWD_CASE(N)                                                                                  \
    case N:                                                                                                    \
        moe_gate_backward_kernel<N><<<grid, 256, 0, stream>>>(a, topk_idx, grad_weight, grad_logits);          \
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
