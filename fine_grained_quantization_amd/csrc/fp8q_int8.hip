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
// which rounds to at most 127: no clamp.  Bound by memory: 4096 x 7168 in 19-21 us (4.2-4.6 TB/s), 8192 x 7168 in 31 us
// (5.7 TB/s); 64 rows in 4 us, a launch and one round trip.
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
// Matrix product.  A workgroup of WM waves along the rows x WN along the channels (8) computes a tile of
// BM = 16 TM WM rows x BN = 16 TN WN channels, a wave 16 TM x 16 TN of it with 16 x 16 x 64 MFMAs (weights as the
// row operand, so that a lane's 4 result registers are 4 consecutive channels of one row).  Both tiles
// travel in blocks of 128 codes from global memory straight into a ring of LDS slots, each for one operand's block (A0 W0
// A1 W1 A2 W2 ...): with 5 slots, while block kb is multiplied, kb + 1 and A's kb + 2 are on the way or there.
// The large tile, 256 x 256 by 8 waves of 64 x 128, is bound by power: 4096 x 16384 x 7168 took 385 us with normal codes
// and 272 us with zeros (an earlier 32 x 32 x 32 form).  So what counts is energy per product: 16 x 16 x 64 MFMAs reach
// 4.0 Pop/s of normal codes where 32 x 32 x 32 reach 3.4 (nothing but MFMAs on every CU; 5.0 is the peak), and in that
// order one operand changes from MFMA to MFMA.  Measured: 4096 x 18432 x 7168 in 400-425 us, 2.6 Pop/s (the library's
// INT8 product of the same sizes, without scales: 585 us); 8192 tokens to 8 of 64 experts of 2048 x 7168 in 820-880 us.
// 128 x 128 tiles, two workgroups to a CU, fill the chip at sizes where that tile does not (2048^3: 12.5 us).
// ---------------------------------------------------------------------------------------------------------

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
    int64_t n_tail, n_ntiles_tail;  // dense: columns from n_tail on are covered by tiles of half the width
};

// Waits for this wave's LDS reads and for all but its last N copies into LDS, then for the workgroup.
template <int N>
__device__ __forceinline__ void copies_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

constexpr int kBack = 4096;
// An offset past every resource here (they end below 2^31 + kBack), also with an instruction's offset on top.
constexpr int kFar = (int)0xFFFFF000u;

// AHEAD: blocks that A's copies run ahead; the ring has 2 AHEAD + 1 slots (A's block kb + AHEAD is copied into the slot that
// W's block kb - 1 has left, W's into that of A's block kb).
template <int TM, int TN, int WM, int WN, int AHEAD>
struct TileShape {
    static constexpr int kWaves = WM * WN;
    static_assert(kWaves == 8, "waves");
    static constexpr int BM = 16 * TM * WM, BN = 16 * TN * WN;
    static constexpr int kSlots = 2 * AHEAD + 1, kSlot = (BM > BN ? BM : BN) * 128, kLds = kSlots * kSlot;
    static constexpr int kRowsA = BM / kWaves, kRowsW = BN / kWaves;  // rows that a wave copies per block
    static constexpr int kCopyA = kRowsA / 8, kCopyW = kRowsW / 8;
    static_assert(kCopyA % 2 == 0 && kCopyW % 2 == 0, "copies go out in halves");
};

// f(0), f(1), ... f(N - 1) with the index as a compile-time constant.
template <int I>
struct Index {
    static constexpr int value = I;
};
template <int N, int I = 0, typename F>
__device__ __forceinline__ void static_for(const F &f) {
    if constexpr (I < N) {
        f(Index<I>{});
        static_for<N, I + 1>(f);
    }
}

// One tile at (m0, n0): rows [m0, mend) of c, W / SW the weights and their scales.  With GATHER row r's codes are
// those of token rtok[r].
template <bool OUT_BF16, int TM, int TN, int WM, int WN, int AHEAD, bool GATHER>
__device__ __forceinline__ void int8_tile(uint8_t *lds, const Int8Args &p, const uint8_t *W, const float *SW,
                                          int64_t m0, int64_t mend, int64_t n0) {
    using S = TileShape<TM, TN, WM, WN, AHEAD>;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6) & (S::kWaves - 1);
    // Waves w and w + 4 share a SIMD; they take different rows, so that absent rows idle half of every SIMD and not both
    // waves of some.
    static_assert(WM <= 4, "waves along the rows");
    const int wn = (wave / WM) * 16 * TN, wm = (wave >= 4 ? (wave % WM) ^ (WM - 1) : wave % WM) * 16 * TM;
    const int64_t K = p.K;
    const int KB = __builtin_amdgcn_readfirstlane((int)((K + 127) >> 7));
    const int64_t nrow = mend - m0 < S::BM ? mend - m0 : S::BM;
    const int64_t ncol = p.N - n0 < S::BN ? p.N - n0 : S::BN;

    // Copies: one instruction moves 8 rows (1 KB); lane l lands in row l / 8 of them, physical chunk l % 8, which
    // holds logical chunk (l % 8) ^ swzf(row).  Rows past the operand are given an offset past its resource.
    // The LDS address of a copy is a base register plus the instruction's offset, which counts for the memory address
    // too: four copies share one base, and the memory offsets of copy j are kBack - 1024 (j % 4) with resources that
    // start kBack bytes early.  (Writing the base register for every copy makes each wait for the one before it.)
    const i32x4 ra = GATHER ? make_rsrc(p.qa - kBack, (uint64_t)p.T * (uint64_t)K + kBack)
                            : make_rsrc(p.qa + m0 * K - kBack, (uint64_t)(nrow * K) + kBack);
    const i32x4 rw = make_rsrc(W + n0 * K - kBack, (uint64_t)(ncol * K) + kBack);
    const int c0 = (lane & 7) ^ (lane >> 3);  // logical chunk in the copies of even j; c0 ^ 1 in the odd ones
    int avoff[S::kCopyA], wvoff[S::kCopyW];
#pragma unroll
    for (int j = 0; j < S::kCopyA; j++) {
        const int r = wave * S::kRowsA + 8 * j + (lane >> 3);
        const int ch = (lane & 7) ^ swzf(r);
        if constexpr (GATHER) {
            const int64_t tok = r < nrow ? p.rtok[m0 + r] : -1;
            avoff[j] = tok >= 0 && tok < p.T ? (int)(tok * K + ch * 16 + kBack - 1024 * (j & 3)) : kFar;
        } else {
            avoff[j] = r < nrow ? (int)(r * K + ch * 16 + kBack - 1024 * (j & 3)) : kFar;
        }
    }
#pragma unroll
    for (int j = 0; j < S::kCopyW; j++) {
        const int r = wave * S::kRowsW + 8 * j + (lane >> 3);
        wvoff[j] = r < ncol ? (int)(r * K) + (((lane & 7) ^ swzf(r)) << 4) + kBack - 1024 * (j & 3) : kFar;
    }
    // Copies [j0, j1) of block kb's A or W rows into its slot; past the last block the resources are empty and nothing
    // is read.  K may end inside a block: that one goes first (the integer sums do not depend on the order), with the
    // chunks past K masked, so that the loop below copies whole blocks only.  Block kb > 0 starts at code
    // (kb - 1) * 128.  (The scalar offset of the block is not range-checked, the others are.)
    auto copy_one = [&](auto index, i32x4 rs, int voff, int so, int per_wave, int slot) __attribute__((always_inline)) {
        constexpr int j = decltype(index)::value;
        fp8q_raw_buffer_load_lds(rs, (lds_ptr)(lds + slot * S::kSlot + (wave * per_wave + (j & ~3)) * 1024), 16, voff, so,
                                 (j & 3) * 1024, 0);
    };
    auto copy_a = [&](auto index, int kb, int slot) __attribute__((always_inline)) {
        i32x4 rs = ra;
        rs[2] = __builtin_amdgcn_readfirstlane(kb < KB ? rs[2] : 0);
        copy_one(index, rs, avoff[decltype(index)::value], __builtin_amdgcn_readfirstlane(kb - 1) * 128, S::kCopyA, slot);
    };
    auto copy_w = [&](auto index, int kb, int slot) __attribute__((always_inline)) {
        i32x4 rs = rw;
        rs[2] = __builtin_amdgcn_readfirstlane(kb < KB ? rs[2] : 0);
        copy_one(index, rs, wvoff[decltype(index)::value], __builtin_amdgcn_readfirstlane(kb - 1) * 128, S::kCopyW, slot);
    };
    // Operand fragments of step ks (64 codes): lane l takes row l % 16 and chunk 2 (l / 16) + ks of the block's 8.  (Which
    // codes a step multiplies does not matter as long as both operands agree; chunk 4 ks + l / 16 would put lanes that the
    // LDS serves together into the same banks, half of all its cycles.)
    auto frag = [&](const uint8_t *tile, int row0, int ks) {
        return *reinterpret_cast<const v4i *>(tile + swz(row0 + (lane & 15), 2 * (lane >> 4) + ks));
    };

    v4i acc[TN][TM];
#pragma unroll
    for (int ni = 0; ni < TN; ni++)
#pragma unroll
        for (int mi = 0; mi < TM; mi++) acc[ni][mi] = (v4i){0, 0, 0, 0};

    const int left = (int)(K - (int64_t)(KB - 1) * 128);
    const bool ok0 = c0 * 16 < left, ok1 = (c0 ^ 1) * 16 < left;
    static_for<S::kCopyA>([&](auto j) __attribute__((always_inline)) {
        copy_one(j, ra, (j.value & 1 ? ok1 : ok0) ? avoff[j.value] : kFar, (KB - 1) * 128, S::kCopyA, 0);
    });
    static_for<S::kCopyW>([&](auto j) __attribute__((always_inline)) {
        copy_one(j, rw, (j.value & 1 ? ok1 : ok0) ? wvoff[j.value] : kFar, (KB - 1) * 128, S::kCopyW, 1);
    });
    static_for<AHEAD - 1>([&](auto block) __attribute__((always_inline)) {
        constexpr int kb = decltype(block)::value + 1;
        static_for<S::kCopyA>([&](auto j) __attribute__((always_inline)) { copy_a(j, kb, 2 * kb); });
        static_for<S::kCopyW>([&](auto j) __attribute__((always_inline)) { copy_w(j, kb, 2 * kb + 1); });
    });
    copies_barrier<(AHEAD - 1) * (S::kCopyA + S::kCopyW)>();  // block 0 is there

    // A block is 2 TN phases: phase g multiplies channel subtile g % TN by all row subtiles, for the 64 codes of step
    // g / TN.  Channel fragments are read kAhead phases before their use, row fragments a step before.  The last of
    // the block's fragments is read kAhead phases before the end; the barrier after that phase frees the block's slots,
    // and the next block's first fragments and the copies into A's slot follow it.
    constexpr int kAhead = 3, kPhases = 2 * TN, kBarrier = kPhases - kAhead;
    constexpr int kLater = (AHEAD - 1) * S::kCopyA + (AHEAD - 2) * S::kCopyW;  // copies of the blocks past kb + 1
    static_assert(kPhases % (kAhead + 1) == 0 && kBarrier > TN && TM % 2 == 0, "phases");
    v4i fa[2][TM], fw[kAhead + 1];
#pragma unroll
    for (int i = 0; i < TM; i++) fa[0][i] = frag(lds, wm + 16 * i, 0);
#pragma unroll
    for (int i = 0; i < kAhead; i++) fw[i] = frag(lds + S::kSlot, wn + 16 * i, 0);
    // Block kb with A in slot `slot` and W in the next.
    auto block = [&](auto index, int kb) __attribute__((always_inline)) {
        constexpr int slot = decltype(index)::value;
        constexpr int s1 = (slot + 1) % S::kSlots, s2 = (slot + 2) % S::kSlots, s3 = (slot + 3) % S::kSlots,
                      last = (slot + S::kSlots - 1) % S::kSlots;  // W's block kb - 1 has left it
        const uint8_t *tA = lds + slot * S::kSlot, *tW = lds + s1 * S::kSlot;
        const uint8_t *nA = lds + s2 * S::kSlot, *nW = lds + s3 * S::kSlot;
        static_for<kPhases>([&](auto phase) __attribute__((always_inline)) {
            constexpr int g = decltype(phase)::value, ks = g / TN, ni = g % TN, gw = (g + kAhead) % kPhases;
            constexpr int after = g - kBarrier;  // phases since the barrier
            // Row fragments [r0, r1) and copies [a0, a1) of A, [w0, w1) of W that this phase issues.
            constexpr int r0 = ks == 0 ? ni * TM / TN : (after == 1 ? TM / 2 : 0);
            constexpr int r1 = ks == 0 ? (ni + 1) * TM / TN : (after == 0 ? TM / 2 : (after == 1 ? TM : 0));
            constexpr int a0 = ks == 0 ? ni * S::kCopyA / TN : 0, a1 = ks == 0 ? (ni + 1) * S::kCopyA / TN : 0;
            constexpr int w0 = after < 0 ? 0 : after * S::kCopyW / kAhead;
            constexpr int w1 = after < 0 ? 0 : (after + 1) * S::kCopyW / kAhead;
            if constexpr (after == 0) {
                copies_barrier<kLater>();  // block kb + 1 is there; the later ones may still be on the way
                __builtin_amdgcn_sched_barrier(0);
            }
            fw[gw % (kAhead + 1)] = frag(after < 0 ? tW : nW, wn + 16 * (gw % TN), gw / TN);
#pragma unroll
            for (int i = r0; i < r1; i++) fa[ks ^ 1][i] = frag(ks == 0 ? tA : nA, wm + 16 * i, ks ^ 1);
            static_for<a1 - a0>([&](auto j) __attribute__((always_inline)) {
                copy_a(Index<a0 + decltype(j)::value>{}, kb + AHEAD, last);
            });
            static_for<w1 - w0>([&](auto j) __attribute__((always_inline)) {
                copy_w(Index<w0 + decltype(j)::value>{}, kb + AHEAD, slot);  // A's block kb has left it
            });
            // (every other phase takes the rows backwards, so that one operand changes from MFMA to MFMA, not two)
#pragma unroll
            for (int i = 0; i < TM; i++) {
                const int mi = g & 1 ? TM - 1 - i : i;
                acc[ni][mi] =
                    __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[g % (kAhead + 1)], fa[ks][mi], acc[ni][mi], 0, 0, 0);
            }
            // Left alone, the compiler reads each fragment right before its MFMAs and waits for it.
            if constexpr (1 + r1 - r0 > 0) __builtin_amdgcn_sched_group_barrier(0x100, 1 + r1 - r0, 0);  // LDS reads
            if constexpr (a1 - a0 + w1 - w0 > 0) __builtin_amdgcn_sched_group_barrier(0x010, a1 - a0 + w1 - w0, 0);  // copies
            __builtin_amdgcn_sched_group_barrier(0x008, TM, 0);  // MFMAs
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    // A wave whose rows are all absent (past the tile's last, or rows of no token), or whose channels are, copies for the
    // others and stores zeros where rows and channels are its own.
    constexpr int kEl = OUT_BF16 ? 2 : 4;
    uint64_t rows_here = 0;
#pragma unroll
    for (int i = 0; i < 16 * TM; i += 64) {
        const int r = wm + i + lane;
        bool here = i + lane < 16 * TM && r < nrow && wn < ncol;
        if constexpr (GATHER) {
            const int64_t tok = here ? p.rtok[m0 + r] : -1;
            here = tok >= 0 && tok < p.T;
        }
        rows_here |= __ballot(here);
    }
    if (__builtin_amdgcn_readfirstlane((int)(rows_here != 0)) == 0) {
        for (int kb = 0, slot = 0; kb < KB; kb++) {
            const int last = slot > 0 ? slot - 1 : S::kSlots - 1;
            static_for<S::kCopyA>([&](auto j) __attribute__((always_inline)) { copy_a(j, kb + AHEAD, last); });
            copies_barrier<kLater>();
            static_for<S::kCopyW>([&](auto j) __attribute__((always_inline)) { copy_w(j, kb + AHEAD, slot); });
            slot = slot + 2 < S::kSlots ? slot + 2 : slot + 2 - S::kSlots;
        }
        copies_barrier<0>();
        const u32x4 zero = {0u, 0u, 0u, 0u};
        constexpr int kChunks = TN * kEl;  // 16-byte chunks of a row's 16 TN channels
        for (int idx = lane; idx < 16 * TM * kChunks; idx += 64) {
            const int64_t m = m0 + wm + idx / kChunks, n = n0 + wn + idx % kChunks * (16 / kEl);
            if (m < mend && n < p.N) *reinterpret_cast<u32x4 *>(static_cast<uint8_t *>(p.c) + (m * p.N + n) * kEl) = zero;
        }
        return;
    }
    // As many blocks at a time as there are slots, so that the slots are constants: block kb's A is in slot 2 kb % kSlots.
    static_assert(S::kSlots <= 9, "steps below");
    for (int kb = 0;; kb += S::kSlots) {
#define FP8Q_INT8_STEP(I)                                  \
    if constexpr (I < S::kSlots) {                         \
        block(Index<2 * (I) % S::kSlots>{}, kb + (I));     \
        if (kb + (I) + 1 >= KB) break;                     \
    }
        FP8Q_INT8_STEP(0)
        FP8Q_INT8_STEP(1)
        FP8Q_INT8_STEP(2)
        FP8Q_INT8_STEP(3)
        FP8Q_INT8_STEP(4)
        FP8Q_INT8_STEP(5)
        FP8Q_INT8_STEP(6)
        FP8Q_INT8_STEP(7)
        FP8Q_INT8_STEP(8)
#undef FP8Q_INT8_STEP
    }

    // A lane holds channels 4 (lane / 16) .. + 3 of row lane % 16 of each subtile.  Results pass through LDS so that
    // whole row segments are stored: a wave's block of 16 TM rows x at most 256 bytes at a time, the 16-byte chunks of row r
    // at chunk ^ (r % 16).
    float sa[TM];
    bool there[TM];  // (a row of no token is +0 whatever the channels' scales are: negative, infinite, NaN)
#pragma unroll
    for (int mi = 0; mi < TM; mi++) {
        const int64_t m = m0 + wm + 16 * mi + (lane & 15);
        int64_t src = m < mend ? m : -1;
        if constexpr (GATHER) {
            src = src >= 0 ? p.rtok[src] : -1;
            if (src >= p.T) src = -1;
        }
        there[mi] = !GATHER || src >= 0;
        sa[mi] = src >= 0 ? p.sa[src] : 0.0f;
    }
    constexpr int kMaxRow = S::kWaves * 16 * TM * 256 <= S::kLds ? 256 : 128;
    constexpr int kSubs = TN * 16 * kEl > kMaxRow ? kMaxRow / (16 * kEl) : TN;  // channel subtiles per pass
    constexpr int kRowBytes = kSubs * 16 * kEl, kChunks = kRowBytes / 16;
    static_assert(S::kWaves * 16 * TM * kRowBytes <= S::kLds && (kChunks & (kChunks - 1)) == 0, "staging");
    copies_barrier<0>();
    uint8_t *blk = lds + wave * 16 * TM * kRowBytes;
#pragma unroll
    for (int n1 = 0; n1 < TN; n1 += kSubs) {
#pragma unroll
        for (int ni = n1; ni < n1 + kSubs; ni++) {
            const int nl = 16 * ni + 4 * (lane >> 4);
            const int64_t n = n0 + wn + nl;
            float sw[4] = {0.f, 0.f, 0.f, 0.f};
            if (n < p.N) {
#pragma unroll
                for (int r = 0; r < 4; r++) sw[r] = SW[n + r];
            }
#pragma unroll
            for (int mi = 0; mi < TM; mi++) {
                const int r = 16 * mi + (lane & 15);
                v4f v;
#pragma unroll
                for (int i = 0; i < 4; i++) v[i] = there[mi] ? (float)acc[ni][mi][i] * (sa[mi] * sw[i]) : 0.0f;
                const int byte = (nl - 16 * n1) * kEl;
                store4<OUT_BF16>(blk + r * kRowBytes + ((((byte >> 4) ^ r) & (kChunks - 1)) << 4) + (byte & 15), 0, v);
            }
        }
        // (the block is the wave's own: its LDS operations are in order)
#pragma unroll
        for (int j = 0; j < 16 * TM * kChunks / 64; j++) {
            const int idx = j * 64 + lane, r = idx / kChunks, ch = idx % kChunks;
            const int64_t m = m0 + wm + r, n = n0 + wn + 16 * n1 + ch * (16 / kEl);
            const u32x4 v = *reinterpret_cast<const u32x4 *>(blk + r * kRowBytes + (((ch ^ r) & (kChunks - 1)) << 4));
            if (m < mend && n < p.N)
                *reinterpret_cast<u32x4 *>(static_cast<uint8_t *>(p.c) + (m * p.N + n) * kEl) = v;
        }
    }
}

// One tile per workgroup.  GROUPED: tiles of an expert-sorted layout.  TAIL (dense): the tiles of columns [0, n_tail), then
// tiles of half the width over the other columns, which fill what would be a last round of few whole tiles.
template <bool OUT_BF16, bool GROUPED, bool GATHER, bool TAIL, int TM, int TN, int WM, int WN, int AHEAD>
__global__ __launch_bounds__(64 * WM * WN, TM * TN <= 8 && AHEAD == 2 ? 4 : 2) void gemm_int8_kernel(Int8Args p) {
    using S = TileShape<TM, TN, WM, WN, AHEAD>;
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
        const int64_t i = xcd_order(blockIdx.x);
        int64_t mt, nt;
        if (!dense_tile_at(i, p.n_mtiles, p.n_ntiles, mt, nt)) {
            if constexpr (TAIL) {
                if (dense_tile_at(i - p.n_mtiles * p.n_ntiles, p.n_mtiles, p.n_ntiles_tail, mt, nt))
                    int8_tile<OUT_BF16, TM, TN / 2, WM, WN, AHEAD, false>(lds, p, p.qw, p.sw, mt * S::BM, p.M,
                                                                   p.n_tail + nt * (S::BN / 2));
            }
            return;
        }
        m0 = mt * S::BM;
        n0 = nt * S::BN;
    }
    int8_tile<OUT_BF16, TM, TN, WM, WN, AHEAD, GATHER>(lds, p, p.qw + e * p.N * p.K, p.sw + e * p.N, m0, mend, n0);
}

// ---------------------------------------------------------------------------------------------------------
// Few rows: a workgroup of 8 waves computes 16 TM rows x up to 16 NS channels, and the waves split K: wave w takes
// blocks w, w + 8, ... of 128 codes, copies the block's rows of both operands into an LDS slot of its own, reads its
// fragments, starts the copies of its next block and multiplies, with no barrier between the waves.  The 8 partial
// sums meet in LDS by integer adds, whose order does not matter.  Bound by memory: 1 x 18432 x 7168 in 22 us (5.9 TB/s,
// partly from the Infinity Cache), 64 x 18432 x 7168 in 29 us (4.6 TB/s; every CU also reads all 64 rows).  One slice of
// channels per CU is best there (72 of 18432; 40: 29 us where 72 took 26, 24: 31).
// ---------------------------------------------------------------------------------------------------------

constexpr int kSplitWaves = 8;

// GATHER: expert segments, row r's codes those of token rtok[r]; a workgroup takes one slice of one expert's channels and
// walks the segment's rows 16 TM at a time; where none of them has a token it only stores zeros.  Else dense.
template <bool OUT_BF16, bool GATHER, int TM, int NS>
__global__ __launch_bounds__(64 * kSplitWaves, 2) void gemm_int8_split_kernel(Int8Args p, int64_t cols_per_wg) {
    constexpr int kA = TM * 2048, kSlot = (TM + NS) * 2048, kSum = TM * NS * 1024;
    constexpr int kLds = kSplitWaves * kSlot > kSum ? kSplitWaves * kSlot : kSum;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6) & (kSplitWaves - 1);
    const int64_t K = p.K;
    const int KB = (int)((K + 127) >> 7);
    int64_t m0, mend, n0, e = 0;
    if constexpr (!GATHER) {
        // Row tiles of one slice of channels are neighbours, so that the slice's weights are read by them together.
        const int64_t nt = blockIdx.x / p.n_mtiles;
        m0 = (blockIdx.x - nt * p.n_mtiles) * 16 * TM;
        mend = p.M - m0 < 16 * TM ? p.M : m0 + 16 * TM;
        n0 = nt * cols_per_wg;
    } else {
        e = blockIdx.x / p.n_ntiles;
        n0 = (blockIdx.x - e * p.n_ntiles) * cols_per_wg;
        // the segment, cut to [0, M)
        const int64_t lo = p.off[e], hi = p.off[e + 1];
        m0 = lo < 0 ? 0 : (lo > p.M ? p.M : lo);
        mend = hi < m0 ? m0 : (hi > p.M ? p.M : hi);
    }
    const int64_t ncol = p.N - n0 < cols_per_wg ? p.N - n0 : cols_per_wg;
    const i32x4 rw = make_rsrc(p.qw + (e * p.N + n0) * K, (uint64_t)(ncol * K));
    const float *SW = p.sw + e * p.N + n0;
    uint8_t *slot = lds + wave * kSlot;
    const int c0 = (lane & 7) ^ (lane >> 3);
    // Rows 8 j + lane / 8 of either operand, as in the tile kernel.
    int wvoff[2 * NS], avoff[2 * TM];
#pragma unroll
    for (int j = 0; j < 2 * NS; j++) {
        const int r = 8 * j + (lane >> 3);
        wvoff[j] = r < ncol ? r * (int)K + (j & 1 ? c0 ^ 1 : c0) * 16 : kFar;
    }
    int *sum = reinterpret_cast<int *>(lds);
    for (; m0 < mend; m0 += 16 * TM) {
        const int64_t nrow = mend - m0 < 16 * TM ? mend - m0 : 16 * TM;
        if constexpr (GATHER) {
            int64_t tok = lane < nrow ? p.rtok[m0 + lane] : -1;
            static_assert(16 * TM <= 64, "a lane per row");
            if (__ballot(tok >= 0 && tok < p.T) == 0) {  // the same in every wave
                constexpr int kEl = OUT_BF16 ? 2 : 4;
                const u32x4 zero = {0u, 0u, 0u, 0u};
                const int chunks = (int)(ncol * kEl / 16);  // channels come in multiples of 8
                for (int i = tid; i < nrow * chunks; i += 64 * kSplitWaves)
                    *reinterpret_cast<u32x4 *>(static_cast<uint8_t *>(p.c) + ((m0 + i / chunks) * p.N + n0) * kEl +
                                               i % chunks * 16) = zero;
                continue;
            }
        }
        const i32x4 ra = GATHER ? make_rsrc(p.qa, (uint64_t)(p.T * K)) : make_rsrc(p.qa + m0 * K, (uint64_t)(nrow * K));
#pragma unroll
        for (int j = 0; j < 2 * TM; j++) {
            const int r = 8 * j + (lane >> 3);
            int64_t row = r < nrow ? r : -1;
            if constexpr (GATHER) row = row >= 0 ? p.rtok[m0 + row] : -1;
            avoff[j] = row >= 0 && (!GATHER || row < p.T) ? (int)(row * K + (j & 1 ? c0 ^ 1 : c0) * 16) : kFar;
        }
        auto issue = [&](int kb) {
            const bool in = kb < KB;
            i32x4 ta = ra, tw = rw;
            ta[2] = in ? ta[2] : 0;
            tw[2] = in ? tw[2] : 0;
            const int so = in ? kb * 128 : 0;
            const int left = in ? (int)(K - (int64_t)kb * 128) : 128;
            const bool ok0 = c0 * 16 < left, ok1 = (c0 ^ 1) * 16 < left;
#pragma unroll
            for (int j = 0; j < 2 * NS; j++)
                fp8q_raw_buffer_load_lds(tw, (lds_ptr)(slot + kA + j * 1024), 16, (j & 1 ? ok1 : ok0) ? wvoff[j] : kFar, so,
                                         0, 0);
#pragma unroll
            for (int j = 0; j < 2 * TM; j++)
                fp8q_raw_buffer_load_lds(ta, (lds_ptr)(slot + j * 1024), 16, (j & 1 ? ok1 : ok0) ? avoff[j] : kFar, so, 0,
                                         0);
        };
        v4i acc[NS][TM];
#pragma unroll
        for (int ni = 0; ni < NS; ni++)
#pragma unroll
            for (int mi = 0; mi < TM; mi++) acc[ni][mi] = (v4i){0, 0, 0, 0};
        issue(wave);
        for (int kb = wave; kb < KB; kb += kSplitWaves) {
            __builtin_amdgcn_s_waitcnt(0);  // the block is there
            asm volatile("" ::: "memory");
            v4i fa[2][TM], fw[2][NS];
#pragma unroll
            for (int ks = 0; ks < 2; ks++) {
                const int ch = 2 * (lane >> 4) + ks;  // as in the tile kernel
#pragma unroll
                for (int i = 0; i < TM; i++)
                    fa[ks][i] = *reinterpret_cast<const v4i *>(slot + swz(16 * i + (lane & 15), ch));
#pragma unroll
                for (int i = 0; i < NS; i++)
                    fw[ks][i] = *reinterpret_cast<const v4i *>(slot + kA + swz(16 * i + (lane & 15), ch));
            }
            __builtin_amdgcn_s_waitcnt(0xC07F);  // the fragments are in registers: the slot may be overwritten
            asm volatile("" ::: "memory");
            issue(kb + kSplitWaves);
#pragma unroll
            for (int ks = 0; ks < 2; ks++)
#pragma unroll
                for (int ni = 0; ni < NS; ni++)
#pragma unroll
                    for (int mi = 0; mi < TM; mi++)
                        acc[ni][mi] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[ks][ni], fa[ks][mi], acc[ni][mi], 0, 0, 0);
        }
        // The last copies (of no bytes) have retired and every wave is done with its slot before the sums take its place.
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
        for (int i = tid; i < kSum / 4; i += 64 * kSplitWaves) sum[i] = 0;
        __syncthreads();
#pragma unroll
        for (int ni = 0; ni < NS; ni++)
#pragma unroll
            for (int mi = 0; mi < TM; mi++)
#pragma unroll
                for (int r = 0; r < 4; r++) atomicAdd(&sum[((ni * TM + mi) * 4 + r) * 64 + lane], acc[ni][mi][r]);
        __syncthreads();
        for (int q = wave; q < NS * TM; q += kSplitWaves) {
            const int ni = q / TM, mi = q % TM;
            const int64_t m = m0 + 16 * mi + (lane & 15);
            const int nl = 16 * ni + 4 * (lane >> 4);  // channels nl .. nl + 3 of the slice: all in or all out
            if (m >= mend || nl >= ncol) continue;
            int64_t src = m;
            if constexpr (GATHER) {
                src = p.rtok[m];
                if (src >= p.T) src = -1;
            }
            const float sa = src >= 0 ? p.sa[src] : 0.0f;
            v4f v;
#pragma unroll
            for (int r = 0; r < 4; r++)
                v[r] = src >= 0 ? (float)sum[(q * 4 + r) * 64 + lane] * (sa * SW[nl + r]) : 0.0f;
            store4<OUT_BF16>(p.c, m * p.N + n0 + nl, v);
        }
        __syncthreads();  // the sums have been read before the next rows' copies overwrite them
    }
}

template <bool GATHER, int TM, int NS>
hipError_t launch_int8_split(Int8Args p, int64_t cols, bool out_bf16, hipStream_t stream) {
    p.n_mtiles = GATHER ? p.E : (p.M + 16 * TM - 1) / (16 * TM);
    p.n_ntiles = (p.N + cols - 1) / cols;
    const dim3 grid((unsigned)(p.n_mtiles * p.n_ntiles));
    if (out_bf16)
        gemm_int8_split_kernel<true, GATHER, TM, NS><<<grid, 64 * kSplitWaves, 0, stream>>>(p, cols);
    else
        gemm_int8_split_kernel<false, GATHER, TM, NS><<<grid, 64 * kSplitWaves, 0, stream>>>(p, cols);
    return hipGetLastError();
}

template <int TM, bool GATHER>
hipError_t launch_int8_split_cols(const Int8Args &p, int64_t cols, bool out_bf16, hipStream_t stream) {
    switch ((cols + 15) / 16) {
        case 1: return launch_int8_split<GATHER, TM, 1>(p, cols, out_bf16, stream);
        case 2: return launch_int8_split<GATHER, TM, 2>(p, cols, out_bf16, stream);
        case 3: return launch_int8_split<GATHER, TM, 3>(p, cols, out_bf16, stream);
        case 4: return launch_int8_split<GATHER, TM, 4>(p, cols, out_bf16, stream);
        default: return launch_int8_split<GATHER, TM, 5>(p, cols, out_bf16, stream);
    }
}

constexpr int kTile = 128;  // the smallest tile's rows and channels

template <bool GROUPED, bool GATHER, bool TAIL, int TM, int TN, int WM, int WN, int AHEAD = 2>
hipError_t launch_int8_tile(Int8Args p, int64_t n_tail, bool out_bf16, hipStream_t stream) {
    using S = TileShape<TM, TN, WM, WN, AHEAD>;
    p.n_mtiles = GROUPED ? p.M / S::BM + p.E : (p.M + S::BM - 1) / S::BM;
    p.n_ntiles = (n_tail + S::BN - 1) / S::BN;
    p.n_tail = n_tail;
    p.n_ntiles_tail = (p.N - n_tail + S::BN / 2 - 1) / (S::BN / 2);
    const dim3 grid((unsigned)((p.n_mtiles * (p.n_ntiles + p.n_ntiles_tail) + 255) / 256 * 256));
    if (out_bf16)
        gemm_int8_kernel<true, GROUPED, GATHER, TAIL, TM, TN, WM, WN, AHEAD><<<grid, S::kWaves * 64, 0, stream>>>(p);
    else
        gemm_int8_kernel<false, GROUPED, GATHER, TAIL, TM, TN, WM, WN, AHEAD><<<grid, S::kWaves * 64, 0, stream>>>(p);
    return hipGetLastError();
}

// The dense product's kernel and its shape, by estimated time in us.  The estimates were fitted to measurements on
// shapes from 64 x 1024 x 16384 to 4096 x 16384 x 7168; they matter by their ratios, at the crossings.
struct Int8Plan {
    enum Kind { kSplitK, kSmall, kDeep, kTall, kWide, kLarge } kind;
    int tm;          // kSplitK: 16-row subtiles of a workgroup
    int64_t cols;    // kSplitK: channels of a workgroup
    int64_t n_tail;  // kLarge: columns covered by whole tiles
};

Int8Plan plan_int8(int64_t M, int64_t N, int64_t K) {
    const double ncu = cu_count();
    const double KB = (double)((K + 127) / 128);
    auto tiles = [](int64_t n, int64_t t) { return (double)((n + t - 1) / t); };
    auto rounds = [](double n, double d) { return (double)(int64_t)((n + d - 1) / d); };
    // 128 x 128 tiles by 8 waves of 32 x 64, two to a CU: 0.60 us a block with one on every CU, 0.92 with two, 1.05 over
    // many rounds.  (4 waves of 64 x 64 read a third less from the LDS and were 0 to 13% slower, with one wave a SIMD.)
    // Where every tile has a CU to itself and K is long, the copies run 4 blocks ahead instead of 2 (the LDS then holds
    // one tile): 512 x 4096 x 7168 33 -> 30 us, 1024 x 4096 x 7168 35 -> 31; no gain at K = 2048 and less.
    const double ts = tiles(M, 128) * tiles(N, 128);
    const bool deep = ts <= ncu && KB >= 32;
    Int8Plan best{deep ? Int8Plan::kDeep : Int8Plan::kSmall, 0, 0, N};
    double cost = 5.0 + (deep            ? KB * (0.42 + 0.07 * ts / ncu)
                         : ts <= ncu     ? KB * (0.42 + 0.18 * ts / ncu)
                         : ts <= 2 * ncu ? KB * (0.28 + 0.32 * ts / ncu) + 3.0
                                         : rounds(ts, 2 * ncu) * (KB * 1.05 + 3.0));
    // 256 x 128 or 128 x 256 tiles, one to a CU: 0.88 us a block.
    const double half = KB * 0.88 + 3.0, tt = tiles(M, 256) * tiles(N, 128), tw = tiles(M, 128) * tiles(N, 256);
    if (5.0 + rounds(tt, ncu) * half < cost) {
        cost = 5.0 + rounds(tt, ncu) * half;
        best = {Int8Plan::kTall, 0, 0, N};
    }
    if (5.0 + rounds(tw, ncu) * half < cost) {
        cost = 5.0 + rounds(tw, ncu) * half;
        best = {Int8Plan::kWide, 0, 0, N};
    }
    // 256 x 256 tiles, one to a CU: 1.48 us a block; all of them, or whole rounds and then 256 x 128 tiles.
    const double mt = tiles(M, 256), nt = tiles(N, 256), large = KB * 1.48 + 5.0;
    if (5.0 + rounds(mt * nt, ncu) * large < cost) {
        cost = 5.0 + rounds(mt * nt, ncu) * large;
        best = {Int8Plan::kLarge, 0, 0, N};
    }
    const int64_t full = (int64_t)(mt * nt / ncu), cols = (int64_t)((double)full * ncu / mt);
    if (full >= 1 && cols >= 1 && cols * 256 < N) {
        const double tail = mt * tiles(N - cols * 256, 128);
        const double c = 5.0 + (double)full * large + rounds(tail, ncu) * half;
        if (c < cost) {
            cost = c;
            best = {Int8Plan::kLarge, 0, 0, cols * 256};
        }
    }
    // Waves that split K: a workgroup takes 8 blocks a round, whose copies come at up to 116 bytes a ns per CU and
    // 14000 a ns over the chip; then the partial sums.
    for (int tm = 1; tm <= 4; tm *= 2) {
        if (tm > 1 && M <= 8 * tm) break;  // half of the rows would be absent
        for (int64_t c = 8; c <= 80; c += 8) {
            const double w = tiles(M, 16 * tm) * tiles(N, c), ns = (double)((c + 15) / 16);
            if (w > 16 * ncu) continue;
            const double act = w < ncu ? w : ncu, rate = 14000.0 / act < 116.0 ? 14000.0 / act : 116.0;
            const double round = (16.0 * tm + (double)c) * 1.024 / rate;
            const double t = 2.0 + rounds(w, ncu) * (rounds(KB, 8.0) * round + 0.165 * tm * ns);
            if (t < cost) {
                cost = t;
                best = {Int8Plan::kSplitK, tm, c, N};
            }
            if (c >= N) break;
        }
    }
    return best;
}

// The host sees how many rows there are and not the segments: a capacity (T k + 127 E rows, rounded up to 128), or the rows
// in use, all of which may carry tokens.  Where the former would leave next to none, T tokens still have a row each (64 full
// segments of 128 rows, 2048 x 7168: 1080 us where the waves split K, 205 by 128 x 128 tiles; 8 such: 136 and 38).
//  - Gathered rows, up to 2 an expert on average, or up to 16 and so few 128 x 128 tiles that they leave CUs idle: the waves
//    split K.  Measured, top-8 (split K / 128 x 128 tiles): 64 experts of 2048 x 7168, one token 25 / 38 us, 4 tokens 83 / 79,
//    32 tokens 198 / 177; 64 of 7168 x 2048, one token 40 / 37; 256 of them, one token 80 / 153; 8 experts of 2048 x 7168,
//    top-2, one token 11 / 34, 32 tokens 23 / 38.  Not for rows in place: every 16 rows of a segment, padding too, would
//    read the weights again, where a tile reads them once for 128 (the first layer: one token 141 / 39, 16 tokens 1018 /
//    196; the second, 4 tokens 466 / 122).
//  - Up to 32 rows, or where the estimated time is less: 128 x 128 tiles, two to a CU.  Measured with 64 experts of 2048 x
//    7168 (256 x 256 tiles / 128 x 128): 4 rows on average 204 / 180 us, 16 rows 207 / 186, 64 rows 212 / 231, 256 rows 300
//    / 359, 1024 rows 876 / 1098.
//  - Else 256 x 256 tiles.
template <bool GATHER>
hipError_t launch_int8_grouped(const Int8Args &p, bool out_bf16, hipStream_t stream) {
    int64_t rows = p.M > 127 * p.E + 64 ? p.M - 127 * p.E - 64 : 0;
    if (GATHER && rows < p.T) rows = p.T < p.M ? p.T : p.M;
    const int64_t ncu = cu_count(), KB = (p.K + 127) / 128;
    auto tiles = [](int64_t n, int64_t t) { return (n + t - 1) / t; };
    if constexpr (GATHER) {
        if (rows <= 2 * p.E || (rows <= 16 * p.E && p.E * tiles(p.N, 128) <= ncu)) {
            // A slice of channels per workgroup and expert: as few slices as put a workgroup on every CU, at most 80
            // channels.
            const int64_t want = (ncu + p.E - 1) / p.E;
            int64_t cols = 8 * ((p.N / 8 + want - 1) / want);
            cols = cols < 80 ? cols : 80;
            if (p.E * tiles(p.N, cols) <= 0xFFFFFFFFll / (64 * kSplitWaves))
                return launch_int8_split_cols<1, true>(p, cols, out_bf16, stream);
        }
    }
    const int64_t small = (rows + 64 * p.E) / 128 * tiles(p.N, 128);
    const int64_t large = ((rows + 64 * p.E) / 256 + p.E / 4) * tiles(p.N, 256);
    const double t_small = small <= ncu ? KB * 0.60 + 5.0 : (double)tiles(small, 2 * ncu) * (KB * 1.05 + 3.0);
    const double t_large = (double)tiles(large, ncu) * (KB * 1.48 + 6.0);
    const double t_read = (double)p.E * p.N * p.K / 5.0e6;  // the weights from memory, at 5 TB/s
    if (rows <= 32 * p.E || (t_small < t_large && t_large > t_read))
        return launch_int8_tile<true, GATHER, false, 2, 4, 4, 2>(p, p.N, out_bf16, stream);
    return launch_int8_tile<true, GATHER, false, 4, 8, 4, 2>(p, p.N, out_bf16, stream);
}

}  // namespace

int64_t gemm_int8_blocks(int64_t M, int64_t N, int64_t E) {
    // An upper bound over the kernels: 128 x 128 tiles (the others launch fewer workgroups, or at most 16 for each CU);
    // -1 past 2^40.
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
    const Int8Args p = {qa, sa, qw, sw, c, M, N, K, nullptr, nullptr, 0, M, 0, 0, 0, 0};
    const Int8Plan plan = plan_int8(M, N, K);
    switch (plan.kind) {
        case Int8Plan::kSplitK:
            if (plan.tm == 1) return launch_int8_split_cols<1, false>(p, plan.cols, out_bf16, stream);
            if (plan.tm == 2) return launch_int8_split_cols<2, false>(p, plan.cols, out_bf16, stream);
            return launch_int8_split_cols<4, false>(p, plan.cols, out_bf16, stream);
        case Int8Plan::kSmall: return launch_int8_tile<false, false, false, 2, 4, 4, 2>(p, N, out_bf16, stream);
        case Int8Plan::kDeep: return launch_int8_tile<false, false, false, 2, 4, 4, 2, 4>(p, N, out_bf16, stream);
        case Int8Plan::kTall: return launch_int8_tile<false, false, false, 4, 4, 4, 2>(p, N, out_bf16, stream);
        case Int8Plan::kWide: return launch_int8_tile<false, false, false, 4, 4, 2, 4>(p, N, out_bf16, stream);
        default: break;
    }
    if (plan.n_tail < N) return launch_int8_tile<false, false, true, 4, 8, 4, 2>(p, plan.n_tail, out_bf16, stream);
    return launch_int8_tile<false, false, false, 4, 8, 4, 2>(p, N, out_bf16, stream);
}

hipError_t launch_grouped_gemm_int8(const uint8_t *qa, const float *sa, int64_t T, const int32_t *row_token,
                                    const uint8_t *qw, const float *sw, void *c, bool out_bf16, const int32_t *off,
                                    int64_t E, int64_t M_total, int64_t N, int64_t K, hipStream_t stream) {
    const Int8Args p = {qa, sa, qw, sw, c, M_total, N, K, off, row_token, E, T, 0, 0, 0, 0};
    return row_token != nullptr ? launch_int8_grouped<true>(p, out_bf16, stream)
                                : launch_int8_grouped<false>(p, out_bf16, stream);
}

}  // namespace fp8q
