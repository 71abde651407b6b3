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
// Matrix product.  A workgroup of 4 waves, WM along the rows x WN along the channels, computes a tile of
// BM = 32 TM WM rows x BN = 32 TN WN channels, a wave 32 TM x 32 TN of it with 32 x 32 x 32 MFMAs (weights as the
// row operand, so that a lane's 4 consecutive result registers are 4 consecutive channels of one row).  Both tiles
// travel in blocks of 128 codes from global memory straight into a ring of 5 LDS slots, each for one operand's block
// (A0 W0 A1 W1 A2 W2 ...): while block kb is multiplied, kb + 1 and A's kb + 2 are on the way or there.
// ---------------------------------------------------------------------------------------------------------

typedef int v16i __attribute__((ext_vector_type(16)));

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

// Waits for this wave's LDS reads and for all but its last N copies into LDS, then for the workgroup.
template <int N>
__device__ __forceinline__ void copies_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

template <int TM, int TN, int WM, int WN>
struct TileShape {
    static_assert(WM * WN == 4, "4 waves");
    static constexpr int BM = 32 * TM * WM, BN = 32 * TN * WN;
    static constexpr int kSlots = 5, kSlot = (BM > BN ? BM : BN) * 128, kLds = kSlots * kSlot;
    static constexpr int kRowsA = BM / 4, kRowsW = BN / 4;  // rows that a wave copies per block
    static constexpr int kCopyA = kRowsA / 8, kCopyW = kRowsW / 8;
};

// The order of one step's instructions.  Left alone, the compiler reads each fragment right before its MFMAs and waits
// for it.  These put the LDS reads (0x100) first, two before each MFMA (0x008), and the copies (0x010) after them,
// spread between the MFMAs that are left.
template <int READS, int MFMAS, int COPIES, int I = 0>
__device__ __forceinline__ void schedule_step() {
    constexpr int kRest = MFMAS - READS / 2;
    if constexpr (I < READS / 2) {
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    } else {
        constexpr int i = I - READS / 2, n = (i + 1) * COPIES / kRest - i * COPIES / kRest;
        if constexpr (n > 0) __builtin_amdgcn_sched_group_barrier(0x010, n, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    }
    if constexpr (I + 1 < MFMAS) schedule_step<READS, MFMAS, COPIES, I + 1>();
}

// One tile at (m0, n0): rows [m0, mend) of c, W / SW the weights and their scales.  With GATHER row r's codes are
// those of token rtok[r].
template <bool OUT_BF16, int TM, int TN, int WM, int WN, bool GATHER>
__device__ __forceinline__ void int8_tile(uint8_t *lds, const Int8Args &p, const uint8_t *W, const float *SW,
                                          int64_t m0, int64_t mend, int64_t n0) {
    using S = TileShape<TM, TN, WM, WN>;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6) & 3;
    const int wm = (wave % WM) * 32 * TM, wn = (wave / WM) * 32 * TN;
    const int64_t K = p.K;
    const int KB = (int)((K + 127) >> 7);
    const int64_t nrow = mend - m0 < S::BM ? mend - m0 : S::BM;
    const int64_t ncol = p.N - n0 < S::BN ? p.N - n0 : S::BN;

    // Copies: one instruction moves 8 rows (1 KB); lane l lands in row l / 8 of them, physical chunk l % 8, which
    // holds logical chunk (l % 8) ^ swzf(row).  Rows past the operand are given an offset past its resource.
    const i32x4 ra = GATHER ? make_rsrc(p.qa, (uint64_t)p.T * (uint64_t)K) : make_rsrc(p.qa + m0 * K, (uint64_t)(nrow * K));
    const i32x4 rw = make_rsrc(W + n0 * K, (uint64_t)(ncol * K));
    const int c0 = (lane & 7) ^ (lane >> 3);  // logical chunk in the copies of even j; c0 ^ 1 in the odd ones
    int avoff[S::kCopyA], wvoff[S::kCopyW];
#pragma unroll
    for (int j = 0; j < S::kCopyA; j++) {
        const int r = wave * S::kRowsA + 8 * j + (lane >> 3);
        const int ch = (lane & 7) ^ swzf(r);
        if constexpr (GATHER) {
            const int64_t tok = r < nrow ? p.rtok[m0 + r] : -1;
            avoff[j] = tok >= 0 && tok < p.T ? (int)(tok * K) + ch * 16 : kOutOfRange;
        } else {
            avoff[j] = r < nrow ? (int)(r * K) + ch * 16 : kOutOfRange;
        }
    }
#pragma unroll
    for (int j = 0; j < S::kCopyW; j++) {
        const int r = wave * S::kRowsW + 8 * j + (lane >> 3);
        wvoff[j] = r < ncol ? (int)(r * K) + (((lane & 7) ^ swzf(r)) << 4) : kOutOfRange;
    }
    // Half h of block kb's A or W rows into its slot; past the last block the resources are empty and nothing is
    // read.  In a block that K ends in, chunks past K read zeros.  (The scalar offset of the block is not
    // range-checked, the others are.)
    auto copy = [&](i32x4 rsrc, const int *voff, int per_wave, int h, int kb, int slot) {
        const bool in = kb < KB;
        const i32x4 rs = in ? rsrc : empty_rsrc(rsrc);
        const int so = in ? kb * 128 : 0;
        const int left = in ? (int)(K - (int64_t)kb * 128) : 128;
        const bool ok0 = c0 * 16 < left, ok1 = (c0 ^ 1) * 16 < left;
#pragma unroll
        for (int j = h * per_wave / 2; j < (h + 1) * per_wave / 2; j++)
            fp8q_raw_buffer_load_lds(rs, (lds_ptr)(lds + slot * S::kSlot + (wave * per_wave + j) * 1024), 16,
                                     (j & 1 ? ok1 : ok0) ? voff[j] : kOutOfRange, so, 0, 0);
    };
    auto copy_a = [&](int h, int kb, int slot) { copy(ra, avoff, S::kCopyA, h, kb, slot); };
    auto copy_w = [&](int h, int kb, int slot) { copy(rw, wvoff, S::kCopyW, h, kb, slot); };
    // Operand fragments of step ks (32 codes): lane l takes row l % 32 and chunk 2 ks + l / 32.
    auto frag = [&](const uint8_t *tile, int row0, int ks) {
        return *reinterpret_cast<const v4i *>(tile + swz(row0 + (lane & 31), 2 * ks + (lane >> 5)));
    };

    v16i acc[TN][TM];
#pragma unroll
    for (int ni = 0; ni < TN; ni++)
#pragma unroll
        for (int mi = 0; mi < TM; mi++)
#pragma unroll
            for (int r = 0; r < 16; r++) acc[ni][mi][r] = 0;

    copy_a(0, 0, 0);
    copy_a(1, 0, 0);
    copy_w(0, 0, 1);
    copy_w(1, 0, 1);
    copy_a(0, 1, 2);
    copy_a(1, 1, 2);
    copy_w(0, 1, 3);
    copies_barrier<S::kCopyA + S::kCopyW / 2>();  // block 0 is there
    v4i fa[2][TM], fw[2][TN];
#pragma unroll
    for (int i = 0; i < TM; i++) fa[0][i] = frag(lds, wm + 32 * i, 0);
#pragma unroll
    for (int i = 0; i < TN; i++) fw[0][i] = frag(lds + S::kSlot, wn + 32 * i, 0);
    // Slot of A's block kb (W's is the next one).  The fragments of a step are read while the MFMAs of the step
    // before it run, and a quarter of the copies of a block is issued in each step.  The last step's fragments are
    // in registers before the barrier that frees the block's slots.
    int slot = 0;
    for (int kb = 0; kb < KB; kb++) {
        const int s1 = slot + 1 < S::kSlots ? slot + 1 : slot + 1 - S::kSlots;
        const int s2 = slot + 2 < S::kSlots ? slot + 2 : slot + 2 - S::kSlots;
        const int s3 = slot + 3 < S::kSlots ? slot + 3 : slot + 3 - S::kSlots;
        const int s4 = slot + 4 < S::kSlots ? slot + 4 : slot + 4 - S::kSlots;
#pragma unroll
        for (int ks = 0; ks < 4; ks++) {
            if (ks == 3) {
                copies_barrier<S::kCopyA>();  // block kb + 1 is there; A's kb + 2 may still be on the way
                __builtin_amdgcn_sched_barrier(0);
            }
            const uint8_t *tA = lds + (ks < 3 ? slot : s2) * S::kSlot, *tW = lds + (ks < 3 ? s1 : s3) * S::kSlot;
#pragma unroll
            for (int i = 0; i < TM; i++) fa[(ks + 1) & 1][i] = frag(tA, wm + 32 * i, (ks + 1) & 3);
#pragma unroll
            for (int i = 0; i < TN; i++) fw[(ks + 1) & 1][i] = frag(tW, wn + 32 * i, (ks + 1) & 3);
            if (ks == 0) copy_w(1, kb + 1, s3);
            if (ks == 1) copy_a(0, kb + 2, s4);
            if (ks == 2) copy_a(1, kb + 2, s4);
            if (ks == 3) copy_w(0, kb + 2, slot);  // the slot that A's block kb leaves
#pragma unroll
            for (int ni = 0; ni < TN; ni++)
#pragma unroll
                for (int mi = 0; mi < TM; mi++)
                    acc[ni][mi] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[ks & 1][ni], fa[ks & 1][mi], acc[ni][mi],
                                                                        0, 0, 0);
            if (ks == 0 || ks == 3)
                schedule_step<TM + TN, TM * TN, S::kCopyW / 2>();
            else
                schedule_step<TM + TN, TM * TN, S::kCopyA / 2>();
            __builtin_amdgcn_sched_barrier(0);
        }
        slot = s2;
    }

    // Register 4 g + i of a lane is channel 8 g + 4 (lane / 32) + i of row lane % 32.  Results pass through LDS so
    // that whole row segments are stored: a wave's block of 32 TM rows x 256 bytes at a time, the 16-byte chunks
    // of row r at chunk ^ (r % 16).
    float sa[TM];
#pragma unroll
    for (int mi = 0; mi < TM; mi++) {
        const int64_t m = m0 + wm + 32 * mi + (lane & 31);
        int64_t src = m < mend ? m : -1;
        if constexpr (GATHER) {
            src = src >= 0 ? p.rtok[src] : -1;
            if (src >= p.T) src = -1;
        }
        sa[mi] = src >= 0 ? p.sa[src] : 0.0f;
    }
    constexpr int kEl = OUT_BF16 ? 2 : 4;
    constexpr int kSubs = TN * 32 * kEl > 256 ? 256 / (32 * kEl) : TN;  // channel subtiles per pass
    constexpr int kRowBytes = kSubs * 32 * kEl, kChunks = kRowBytes / 16;
    static_assert(4 * 32 * TM * kRowBytes <= S::kLds && (kChunks & (kChunks - 1)) == 0, "staging");
    copies_barrier<0>();
    uint8_t *blk = lds + wave * 32 * TM * kRowBytes;
#pragma unroll
    for (int n1 = 0; n1 < TN; n1 += kSubs) {
#pragma unroll
        for (int ni = n1; ni < n1 + kSubs; ni++)
#pragma unroll
            for (int g = 0; g < 4; g++) {
                const int nl = 32 * ni + 8 * g + 4 * (lane >> 5);
                const int64_t n = n0 + wn + nl;
                float4 sw = make_float4(0.f, 0.f, 0.f, 0.f);
                if (n < p.N) {
                    sw.x = SW[n];
                    sw.y = SW[n + 1];
                    sw.z = SW[n + 2];
                    sw.w = SW[n + 3];
                }
#pragma unroll
                for (int mi = 0; mi < TM; mi++) {
                    const int r = 32 * mi + (lane & 31);
                    v4f v;
                    v[0] = (float)acc[ni][mi][4 * g] * (sa[mi] * sw.x);
                    v[1] = (float)acc[ni][mi][4 * g + 1] * (sa[mi] * sw.y);
                    v[2] = (float)acc[ni][mi][4 * g + 2] * (sa[mi] * sw.z);
                    v[3] = (float)acc[ni][mi][4 * g + 3] * (sa[mi] * sw.w);
                    const int byte = (nl - 32 * n1) * kEl;
                    store4<OUT_BF16>(blk + r * kRowBytes + ((((byte >> 4) ^ r) & (kChunks - 1)) << 4) + (byte & 15), 0, v);
                }
            }
        // (the block is the wave's own: its LDS operations are in order)
#pragma unroll
        for (int j = 0; j < 32 * TM * kChunks / 64; j++) {
            const int idx = j * 64 + lane, r = idx / kChunks, ch = idx % kChunks;
            const int64_t m = m0 + wm + r, n = n0 + wn + 32 * n1 + ch * (16 / kEl);
            const u32x4 v = *reinterpret_cast<const u32x4 *>(blk + r * kRowBytes + (((ch ^ r) & (kChunks - 1)) << 4));
            if (m < mend && n < p.N)
                *reinterpret_cast<u32x4 *>(static_cast<uint8_t *>(p.c) + (m * p.N + n) * kEl) = v;
        }
    }
}

template <bool OUT_BF16, bool GROUPED, bool GATHER, int TM, int TN, int WM, int WN>
__global__ __launch_bounds__(256, 1) void gemm_int8_kernel(Int8Args p) {
    using S = TileShape<TM, TN, WM, WN>;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[S::kLds];
    int64_t m0, mend = p.M, n0, e = 0;
    if constexpr (GROUPED) {
        if (!grouped_tile<S::BM>(blockIdx.x, p.off, p.E, p.M, p.n_mtiles, p.n_ntiles, S::BN, threadIdx.x & 63, m0, mend,
                                 n0, e))
            return;
        // The same in every lane, but the compiler cannot see that: they come out of lane shuffles.
        e = __builtin_amdgcn_readfirstlane((int)e);
        m0 = __builtin_amdgcn_readfirstlane((int)m0);
        mend = __builtin_amdgcn_readfirstlane((int)mend);
    } else {
        int64_t mt, nt;
        if (!dense_tile_at(xcd_order(blockIdx.x), p.n_mtiles, p.n_ntiles, mt, nt)) return;
        m0 = mt * S::BM;
        n0 = nt * S::BN;
    }
    int8_tile<OUT_BF16, TM, TN, WM, WN, GATHER>(lds, p, p.qw + e * p.N * p.K, p.sw + e * p.N, m0, mend, n0);
}

constexpr int kTile = 128;  // the smallest tile's rows and channels

template <bool GROUPED, bool GATHER, int TM, int TN, int WM, int WN>
hipError_t launch_int8_tile(Int8Args p, bool out_bf16, hipStream_t stream) {
    using S = TileShape<TM, TN, WM, WN>;
    p.n_mtiles = GROUPED ? p.M / S::BM + p.E : (p.M + S::BM - 1) / S::BM;
    p.n_ntiles = (p.N + S::BN - 1) / S::BN;
    const dim3 grid((unsigned)((p.n_mtiles * p.n_ntiles + 255) / 256 * 256));
    if (out_bf16)
        gemm_int8_kernel<true, GROUPED, GATHER, TM, TN, WM, WN><<<grid, 256, 0, stream>>>(p);
    else
        gemm_int8_kernel<false, GROUPED, GATHER, TM, TN, WM, WN><<<grid, 256, 0, stream>>>(p);
    return hipGetLastError();
}

template <bool GROUPED, bool GATHER>
hipError_t launch_int8(Int8Args p, bool out_bf16, hipStream_t stream) {
    if (p.M >= 2048) return launch_int8_tile<GROUPED, GATHER, 4, 4, 2, 2>(p, out_bf16, stream);
    return launch_int8_tile<GROUPED, GATHER, 2, 2, 2, 2>(p, out_bf16, stream);
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
