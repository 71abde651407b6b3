// Weight gradients from transposed copies, dense and per expert:
//   dW[n][k] = sum_mb 2^(eg[mb][n] + ex[mb][k] - 254) * sum_{m in mb} gt[n][m] xt[k][m]   (+ dW)
// with E4M3 codes in groups of 128 tokens of one channel and one power of two each, so that a group's scale is a scale of
// the matrix instruction and nothing is left to do between two blocks of tokens.
//
// Two forms, by the result's type:
//  - bf16: v_mfma_scale_f32_16x16x128_f8f6f4, a block of 128 tokens per instruction, scales applied by it.  The E4M3 MFMAs
//    line their 128 products up before adding them and cut what falls below: each result is 1.4e-5 (relative, rms, for codes
//    of normal values) off the exact sum, at K = 128 as at K = 32768, without a bias.  That is 1/100 of bf16's own rounding.
//  - fp32: the codes, times their scales, become bf16 (exactly: 4 significant bits and a power of two; bytes 0 to 2 lose what is
//    below bf16's least step, 2^-133) in registers, and v_mfma_f32_16x16x32_bf16, which takes subnormal numbers as they are,
//    adds them to 1e-7.  Half of the peak rate.
#include "fp8q_device.h"
#include "fp8q_kernels.h"
#include "fp8q_tiles.h"

namespace fp8q {
namespace {

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

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

struct WgradArgs {
    const uint8_t *gt, *eg, *xt, *ex;
    void *dw;
    const int32_t *off;  // null: one product over all M columns
    int64_t M, N, K, E;
    int64_t n_tiles, k_tiles;
    float *sums;  // [parts][N][K]
    int64_t parts;
};

// Rows in groups of 64: row 4 i + j of a group is row i of the group's 16-row subtile j.  So a lane's scale bytes of the 4
// subtiles are one dword (the instruction picks the byte), and in the result the 4 subtiles of a column group are 4
// consecutive columns.  In LDS the subtiles lie one behind the other, place 16 j + i, 128 codes (8 chunks of 16) each, chunk c
// at c ^ swzf(place): a fragment read touches 16 neighbouring places at one chunk, all banks alike.  (With row 4 i + j at that
// place, every row of a fragment starts in the same half of the 64 banks, and half of the reads' cycles were conflicts.)
__device__ __forceinline__ int row_at(int place) { return (place & ~63) + 4 * (place & 15) + ((place >> 4) & 3); }

__device__ __forceinline__ v8i wfrag(const uint8_t *tile, int place, int g) {
    const u32x4 lo = *reinterpret_cast<const u32x4 *>(tile + swz(place, 2 * g));
    const u32x4 hi = *reinterpret_cast<const u32x4 *>(tile + swz(place, 2 * g + 1));
    v8i f;
    f[0] = (int)lo[0]; f[1] = (int)lo[1]; f[2] = (int)lo[2]; f[3] = (int)lo[3];
    f[4] = (int)hi[0]; f[5] = (int)hi[1]; f[6] = (int)hi[2]; f[7] = (int)hi[3];
    return f;
}

// 8 codes (two dwords) times a power of two, in bf16.
__device__ __forceinline__ v8bf to_bf16(int d0, int d1, float s) {
    const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)d0, s, false);
    const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)d0, s, true);
    const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)d1, s, false);
    const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)d1, s, true);
    v8bf r;
    r[0] = a[0]; r[1] = a[1]; r[2] = b[0]; r[3] = b[1]; r[4] = c[0]; r[5] = c[1]; r[6] = d[0]; r[7] = d[1];
    return r;
}

// 16 codes times a power of two, in bf16.
__device__ __forceinline__ void widen16(const v4i &d, float s, v8bf (&o)[2]) {
    o[0] = to_bf16(d[0], d[1], s);
    o[1] = to_bf16(d[2], d[3], s);
}

// The power of two of byte j of a scale dword, for the conversions above.  (They read the exponent's bits only: the pattern 0 is
// byte 0's 2^-127, which groups of zeros have and groups of values up to 448 2^-127.)
__device__ __forceinline__ float power_of(uint32_t s, int j) { return __uint_as_float(((s >> (8 * j)) & 255u) << 23); }

// 4 results as they are in memory, and in fp32.
template <bool BF16>
struct Four {
    uint2 lo, hi;
    __device__ __forceinline__ void load(const void *c, int64_t idx) {
        const uint2 *at = reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(c) + idx * (BF16 ? 2 : 4));
        lo = at[0];
        if constexpr (!BF16) hi = at[1];
    }
    __device__ __forceinline__ v4f value() const {
        if constexpr (BF16) return (v4f){bf16_lo(lo.x), bf16_hi(lo.x), bf16_lo(lo.y), bf16_hi(lo.y)};
        return (v4f){__uint_as_float(lo.x), __uint_as_float(lo.y), __uint_as_float(hi.x), __uint_as_float(hi.y)};
    }
};

template <bool BF16>
__device__ __forceinline__ v4f load4(const void *c, int64_t idx) {
    Four<BF16> f;
    f.load(c, idx);
    return f.value();
}

// ---------------------------------------------------------------------------------------------------------
// Small results: 128 x 128 tiles by 4 waves of 64 x 64, two workgroups to a CU, blocks of 128 tokens through two LDS stages.
// kParts: the blocks are dealt to several workgroups a tile, whose sums go to the workspace [parts][N][K] in fp32 and are added
// in order by a second launch.  Bound by the latency of a block's copies (0.6 us, nothing else is on the way): 300 x 576 x 2064
// (3 blocks) 6.8 us; 16384 x 512 x 512 79 us by 16 workgroups, 15.7 by 256.
// ---------------------------------------------------------------------------------------------------------

constexpr int kTile = 128;
constexpr int kScaleAt = 2 * kTile * 128, kStage = kScaleAt + 1024;  // a stage: rows, columns, and the scale bytes of both

enum Store { kStoreBf16, kStoreF32, kAddBf16, kAddF32, kParts };

template <bool EXACT, int STORE>
__global__ __launch_bounds__(256, 2) void wgrad_small_kernel(WgradArgs p) {
    __shared__ __attribute__((aligned(1024))) uint8_t stage0[kStage];
    __shared__ __attribute__((aligned(1024))) uint8_t stage1[kStage];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave & 1, wn = wave >> 1;
    const int i = lane & 15, g = lane >> 4;
    const int64_t per = p.n_tiles * p.k_tiles;
    int64_t e = 0, part = 0, nt, kt;
    if constexpr (STORE == kParts) {  // a tile's parts are far apart, neighbours share an operand
        part = blockIdx.x / per;
        const int64_t r = blockIdx.x - part * per;
        nt = r / p.k_tiles;
        kt = r % p.k_tiles;
    } else if (p.off == nullptr) {
        // (the XCD order spreads the tiles over all workgroups of a round, so blockIdx may be past the number of tiles)
        if (!dense_tile_at(xcd_order(blockIdx.x), p.n_tiles, p.k_tiles, nt, kt)) return;
    } else {
        e = blockIdx.x / per;
        if (e >= p.E) return;
        const int64_t r = blockIdx.x - e * per;
        nt = r / p.k_tiles;
        kt = r % p.k_tiles;
    }
    const int64_t n0 = nt * kTile, k0 = kt * kTile;
    // the segment, cut to [0, M) and to whole blocks
    int64_t lo = 0, hi = p.M;
    if (p.off != nullptr) {
        lo = p.off[e];
        hi = p.off[e + 1];
        lo = lo < 0 ? 0 : (lo > p.M ? p.M : lo & ~127);
        hi = hi < lo ? lo : (hi > p.M ? p.M : hi & ~127);
    }
    if constexpr (STORE == kParts) {
        const int64_t each = (p.M / 128 + p.parts - 1) / p.parts * 128;
        lo = part * each < p.M ? part * each : p.M;
        hi = lo + each < p.M ? lo + each : p.M;
    }
    const int b0 = __builtin_amdgcn_readfirstlane((int)(lo >> 7));
    const int KB = __builtin_amdgcn_readfirstlane((int)((hi - lo) >> 7));
    const int64_t ld = p.M;
    const int64_t nrow = p.N - n0 < kTile ? p.N - n0 : kTile, ncol = p.K - k0 < kTile ? p.K - k0 : kTile;
    const i32x4 ra = make_rsrc(p.gt + n0 * ld + (int64_t)b0 * 128, (uint64_t)((nrow - 1) * ld + (int64_t)KB * 128));
    const i32x4 rb = make_rsrc(p.xt + k0 * ld + (int64_t)b0 * 128, (uint64_t)((ncol - 1) * ld + (int64_t)KB * 128));
    int av[4], bv[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const int place = (wave * 4 + j) * 8 + (lane >> 3), r = row_at(place);
        const int at = (int)(r * ld) + (((lane & 7) ^ swzf(place)) << 4);
        av[j] = r < nrow ? at : kOutOfRange;
        bv[j] = r < ncol ? at : kOutOfRange;
    }
    // Block kb's codes and scale bytes into a stage.
    auto issue = [&](uint8_t *st, int kb) __attribute__((always_inline)) {
        if (kb >= KB) return;  // (no copy is on its way into LDS when the workgroup ends)
        if (wave < 2) {  // 4 scale bytes a lane: wave 0 the rows', wave 1 the columns'
            const bool rows = wave == 0;
            const int64_t n = rows ? nrow : ncol;
            const i32x4 rs = make_rsrc((rows ? p.eg + (int64_t)(b0 + kb) * p.N + n0 : p.ex + (int64_t)(b0 + kb) * p.K + k0),
                                       (uint64_t)n);
            fp8q_raw_buffer_load_lds(rs, (lds_ptr)(st + kScaleAt + wave * 512), 4, lane * 4, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < 4; j++) fp8q_raw_buffer_load_lds(ra, (lds_ptr)(st + (wave * 4 + j) * 1024), 16, av[j], kb * 128, 0, 0);
#pragma unroll
        for (int j = 0; j < 4; j++)
            fp8q_raw_buffer_load_lds(rb, (lds_ptr)(st + kTile * 128 + (wave * 4 + j) * 1024), 16, bv[j], kb * 128, 0, 0);
    };
    v4f acc[4][4];
#pragma unroll
    for (int a = 0; a < 4; a++)
#pragma unroll
        for (int b = 0; b < 4; b++) acc[a][b] = (v4f){0.f, 0.f, 0.f, 0.f};
    issue(stage0, 0);
    // A lane holds, of row 4 (4 g + r) + a of the wave's 64, columns 4 i .. 4 i + 3: 16 lanes store 64 consecutive columns.
    constexpr bool kBf16 = STORE == kStoreBf16 || STORE == kAddBf16, kAdd = STORE == kAddBf16 || STORE == kAddF32;
    const int64_t k = k0 + wn * 64 + 4 * i;
    void *out = STORE == kParts ? static_cast<void *>(p.sums) : p.dw;
    auto there = [&](int a, int r) { return k < p.K && n0 + wm * 64 + 4 * (4 * g + r) + a < p.N; };
    auto place = [&](int a, int r) {  // (one of e and part is 0)
        return ((e + part) * p.N + n0 + wm * 64 + 4 * (4 * g + r) + a) * p.K + k;
    };
    Four<kBf16> old[4][4];  // on the way while the blocks are multiplied
    if constexpr (kAdd) {
#pragma unroll
        for (int a = 0; a < 4; a++)
#pragma unroll
            for (int r = 0; r < 4; r++) {
                old[a][r].lo = old[a][r].hi = (uint2){0u, 0u};
                if (there(a, r)) old[a][r].load(out, place(a, r));
            }
    }
    for (int kb = 0; kb < KB; kb++) {
        uint8_t *cur = (kb & 1) ? stage1 : stage0, *nxt = (kb & 1) ? stage0 : stage1;
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
        issue(nxt, kb + 1);
        const uint32_t sa = *reinterpret_cast<const uint32_t *>(cur + kScaleAt + wm * 64 + 4 * i);
        const uint32_t sb = *reinterpret_cast<const uint32_t *>(cur + kScaleAt + 512 + wn * 64 + 4 * i);
        v8i af[4];
        v8bf ab[EXACT ? 4 : 1][4];
#pragma unroll
        for (int a = 0; a < 4; a++) af[a] = wfrag(cur, wm * 64 + 16 * a + i, g);
        if constexpr (EXACT) {
#pragma unroll
            for (int a = 0; a < 4; a++)
#pragma unroll
                for (int q = 0; q < 4; q++) ab[a][q] = to_bf16(af[a][2 * q], af[a][2 * q + 1], power_of(sa, a));
        }
        static_for<4>([&](auto b_) __attribute__((always_inline)) {
            constexpr int b = decltype(b_)::value;
            const v8i bf = wfrag(cur + kTile * 128, wn * 64 + 16 * b + i, g);
            if constexpr (EXACT) {
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    const v8bf bb = to_bf16(bf[2 * q], bf[2 * q + 1], power_of(sb, b));
#pragma unroll
                    for (int a = 0; a < 4; a++)
                        acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ab[a][q], bb, acc[a][b], 0, 0, 0);
                }
            } else {
                static_for<4>([&](auto a_) __attribute__((always_inline)) {
                    constexpr int a = decltype(a_)::value;
                    acc[a][b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(af[a], bf, acc[a][b], 0, 0, a, (int)sa, b,
                                                                                (int)sb);
                });
            }
        });
    }
#pragma unroll
    for (int a = 0; a < 4; a++)
#pragma unroll
        for (int r = 0; r < 4; r++) {
            v4f v = {acc[a][0][r], acc[a][1][r], acc[a][2][r], acc[a][3][r]};
            if constexpr (kAdd) v += old[a][r].value();
            if (there(a, r)) store4<kBf16>(out, place(a, r), v);
        }
}

// The parts' sums, in order, 4 results a thread.
template <int STORE>
__global__ __launch_bounds__(256) void wgrad_parts_kernel(WgradArgs p) {
    constexpr bool kBf16 = STORE == kStoreBf16 || STORE == kAddBf16;
    const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4, size = p.N * p.K;
    if (at >= size) return;
    v4f v = load4<false>(p.sums, at);
#pragma unroll 4
    for (int64_t s = 1; s < p.parts; s++) v += load4<false>(p.sums, s * size + at);
    if constexpr (STORE == kAddBf16 || STORE == kAddF32) v += load4<kBf16>(p.dw, at);
    store4<kBf16>(p.dw, at, v);
}

// ---------------------------------------------------------------------------------------------------------
// Large results: 256 x 256 tiles by 8 waves of 64 x 128, one workgroup to a CU, each walking up to 64 tiles b, b + G, ... as one
// stream of blocks of 128 tokens: the copies of the next tile's first blocks are under way while a tile's results are stored.
// A ring of 5 LDS slots of one operand's block each (A0 B0 A1 B1 A2 ...): while block s is multiplied, s + 1 and A's s + 2
// are on the way or there.  Block s has A in slot 2 s mod 5; A's s + 2 goes where B's s - 1 was, B's s + 2 where A's s was.
// The scale bytes come straight into registers, a block ahead.
// 4096 x 18432 x 7168: bf16 376-400 us, 2.7-2.9 PFLOP/s, at the power limit (304 us with zeros for codes), 423 where it adds to
// older results; fp32 732-750 us, 1.45 PFLOP/s, 817-842 where it adds to 528 MB of older results: the matrix cores are busy for
// 0.69 of the cycles, 0.60 with the older results, at 2.1 GHz; the conversions and addresses (two vector instructions to one of
// theirs) fill most of the rest.  64 experts of 1152 rows, 2048 x 7168 in bf16: 1030 us, of which 1.9 GB of results cost 300
// (722 without the stores), 1233 added to older ones; in fp32 1770 and 2200.
// ---------------------------------------------------------------------------------------------------------

constexpr int kSlot = 256 * 128, kSlots = 5, kMostTiles = 64;

// Waits for this wave's LDS reads and for all but its last N loads and stores, then for the workgroup.
template <int N>
__device__ __forceinline__ void copies_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// The same in every lane, but the compiler may not see that.
__device__ __forceinline__ void uniform(i32x4 &r) {
#pragma unroll
    for (int k = 0; k < 4; k++) r[k] = __builtin_amdgcn_readfirstlane(r[k]);
}

struct WgradTile {
    int e, n0, k0, nrow, ncol, b0, KB;  // expert, corner, rows and columns that exist, first block, blocks
};

// A workgroup's tiles, one to a lane, in 32-bit arithmetic: tile T = expert by expert, each in the dense order (columns of 16
// tiles along k, in them squares of 16 x 16 in blocks of 4 x 8).
struct WgradTiles {
    int e, at;  // at: n tile << 16 | k tile

    // Returns the tile's blocks; -1: there is no such tile.
    __device__ __forceinline__ int init(const WgradArgs &p, uint32_t t) {
        const uint32_t nt = (uint32_t)p.n_tiles, kt = (uint32_t)p.k_tiles, per = nt * kt;
        uint32_t T = (t / 256) * 256 + (t % 8) * 32 + (t % 256) / 8;  // xcd_order
        e = at = 0;
        if (T >= (uint32_t)p.E * per) return -1;
        e = (int)(T / per);
        T -= (uint32_t)e * per;
        const uint32_t sg = T / (16 * nt), hn = min(kt - 16 * sg, 16u);
        uint32_t j = T - sg * 16 * nt;
        const uint32_t sm = j / (16 * hn), hm = min(nt - 16 * sm, 16u);
        j -= sm * 16 * hn;
        const uint32_t qn = j / (8 * hm), wq = min(hn - 8 * qn, 8u);
        j -= qn * 8 * hm;
        const uint32_t qm = j / (4 * wq), hq = min(hm - 4 * qm, 4u);
        j -= qm * 4 * wq;
        at = (int)((16 * sm + 4 * qm + j % hq) << 16 | (16 * sg + 8 * qn + j / hq));
        int b0, KB;
        blocks(p, e, b0, KB);
        return KB;
    }
    // An expert's blocks: its segment, cut to [0, M) and to whole blocks.
    static __device__ __forceinline__ void blocks(const WgradArgs &p, int e, int &b0, int &KB) {
        int lo = 0, hi = (int)p.M;
        if (p.off != nullptr) {
            lo = p.off[e];
            hi = p.off[e + 1];
            lo = lo < 0 ? 0 : (lo > (int)p.M ? (int)p.M : lo & ~127);
            hi = hi < lo ? lo : (hi > (int)p.M ? (int)p.M : hi & ~127);
        }
        b0 = lo >> 7;
        KB = (hi - lo) >> 7;
    }
    __device__ __forceinline__ WgradTile get(const WgradArgs &p, int i) const {
        WgradTile w;
        const int x = __builtin_amdgcn_readlane(at, i);
        w.e = __builtin_amdgcn_readlane(e, i);
        w.n0 = ((uint32_t)x >> 16) * 256;
        w.k0 = (x & 0xFFFF) * 256;
        w.nrow = min((int)p.N - w.n0, 256);
        w.ncol = min((int)p.K - w.k0, 256);
        blocks(p, w.e, w.b0, w.KB);
        w.b0 = __builtin_amdgcn_readfirstlane(w.b0);
        w.KB = __builtin_amdgcn_readfirstlane(w.KB);
        return w;
    }
};

// Zeros into the tiles of no tokens.
template <int EL>
__device__ __forceinline__ void wgrad_zero(const WgradArgs &p, const WgradTiles &list, uint64_t none, int tid, int threads) {
    for (; none != 0; none &= none - 1) {
        const WgradTile w = list.get(p, __builtin_ctzll(none));
        uint8_t *c = static_cast<uint8_t *>(p.dw) + (((int64_t)w.e * p.N + w.n0) * p.K + w.k0) * EL;
        const int chunks = w.ncol * EL / 16;
        for (int at = tid; at < w.nrow * chunks; at += threads) {
            const int r = at / chunks;
            *reinterpret_cast<u32x4 *>(c + r * p.K * EL + (at - r * chunks) * 16) = (u32x4){0u, 0u, 0u, 0u};
        }
    }
}

// Columns of a wave's 128 in its 8 column subtiles, so that a lane's results of a row come 16 bytes at a time: column i of
// subtile b is column 8 i + b of them (bf16), or 64 (b / 4) + 4 i + b % 4 (fp32).  Its place in LDS is 16 b + i.
template <bool EXACT>
__device__ __forceinline__ int col_at(int place) {
    return EXACT ? row_at(place) : (place & ~127) + 8 * (place & 15) + ((place >> 4) & 7);
}

// Streaming stores: 64 gradients of 2048 x 7168 that nothing else delays (one block each) take 313 us with them (6.0 TB/s),
// 432 without.
constexpr int kNonTemporal = 2;
// An offset past every tile's resource (256 rows of at most 2^22 bytes), also with a few rows added to it.
constexpr int kFar = 0x60000000;

// A lane holds, of row 4 (4 g + r) + a of a wave's 64, columns 8 i .. 8 i + 7, or 4 i .. 4 i + 3 of either half: 16 lanes store
// 256 consecutive bytes.  kStores of them whatever the tile's size (those past it are out of range): the waits for copies that
// are older than the stores count on it.
template <bool EXACT>
constexpr int kStores = EXACT ? 32 : 16;
// Loads of a block's scale bytes; the waits count on these too.  (They are written as the instructions that they become: two
// loads of neighbouring dwords would be merged, and a wait too short.  tests/test_wgrad_waits.py counts all of them in the
// compiler's listing.)
template <bool EXACT>
constexpr int kScaleLoads = EXACT ? 3 : 2;

// Rows past the tile are past the resource, from nrow * pitch on; columns past it are sent there.  The whole offset goes into
// the lane's: behind a store with a scalar offset the compiler lets the next instruction overwrite the store's data registers,
// and the store was seen to take the new value there.
template <bool EXACT, bool ACCUMULATE>
__device__ __forceinline__ void wgrad_store(const WgradArgs &p, const v4f (&acc)[4][8], const WgradTile &w, int row, int col) {
    constexpr int kEl = EXACT ? 4 : 2;
    const i32x4 rs = make_rsrc(static_cast<uint8_t *>(p.dw) + (((int64_t)w.e * p.N + w.n0) * p.K + w.k0) * kEl,
                               (uint64_t)(((w.nrow - 1) * p.K + w.ncol) * kEl));
    const int pitch = (int)p.K * kEl, at = row * pitch + col * kEl;
    const int at0 = col < w.ncol ? at : kFar, at1 = col + 64 < w.ncol ? at + 64 * kEl : kFar;
#pragma unroll
    for (int r = 0; r < 4; r++) {
        i32x4 old[4][2];
        if constexpr (ACCUMULATE) {
#pragma unroll
            for (int a = 0; a < 4; a++) {
                old[a][0] = fp8q_raw_buffer_load_b128(rs, at0 + (4 * r + a) * pitch, 0, 0);
                if constexpr (EXACT) old[a][1] = fp8q_raw_buffer_load_b128(rs, at1 + (4 * r + a) * pitch, 0, 0);
            }
        }
#pragma unroll
        for (int a = 0; a < 4; a++) {
            if constexpr (EXACT) {
#pragma unroll
                for (int c = 0; c < 2; c++) {
                    v4f v = {acc[a][4 * c][r], acc[a][4 * c + 1][r], acc[a][4 * c + 2][r], acc[a][4 * c + 3][r]};
                    if constexpr (ACCUMULATE) v += __builtin_bit_cast(v4f, old[a][c]);
                    fp8q_raw_buffer_store_b128(__builtin_bit_cast(i32x4, v), rs, (c ? at1 : at0) + (4 * r + a) * pitch, 0,
                                               kNonTemporal);
                }
            } else {
                i32x4 o;
#pragma unroll
                for (int c = 0; c < 4; c++) {
                    float x = acc[a][2 * c][r], y = acc[a][2 * c + 1][r];
                    if constexpr (ACCUMULATE) {
                        x += bf16_lo((uint32_t)old[a][0][c]);
                        y += bf16_hi((uint32_t)old[a][0][c]);
                    }
                    o[c] = (int)pack_bf16x2(x, y);
                }
                fp8q_raw_buffer_store_b128(o, rs, at0 + (4 * r + a) * pitch, 0, kNonTemporal);
            }
        }
    }
}

template <bool EXACT, bool ACCUMULATE>
__global__ __launch_bounds__(512, 2) void wgrad_stream_kernel(WgradArgs p) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kSlots * kSlot];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6) & 7;
    const int wm = wave & 3, wn = wave >> 2;
    const int i = lane & 15, g = lane >> 4;
    const int col = wn * 128 + (EXACT ? 4 : 8) * i;  // of the lane's results
    const int64_t ld = p.M;
    WgradTiles list;
    const int blocks = list.init(p, blockIdx.x + gridDim.x * lane);
    const uint64_t work = __ballot(blocks > 0);
    if constexpr (!ACCUMULATE) wgrad_zero<EXACT ? 4 : 2>(p, list, __ballot(blocks == 0), tid, 512);
    if (work == 0) return;

    // Copies: an instruction moves 8 places (1 KB); lane l lands in place l / 8 of them, chunk l % 8, which holds logical chunk
    // (l % 8) ^ swzf(place).  Rows past the operand are past its resource: their offset is at least nrow * ld.
    // (Places j + 2 hold the rows after those of places j: the scalar offset takes that.)
    int avoff[2], bvoff[2];
#pragma unroll
    for (int j = 0; j < 2; j++) {
        const int place = wave * 32 + j * 8 + (lane >> 3), chunk = ((lane & 7) ^ swzf(place)) << 4;
        avoff[j] = (int)(row_at(place) * ld) + chunk;
        bvoff[j] = (int)(col_at<EXACT>(place) * ld) + chunk;
    }
    // The stream's issue end: the block that is copied next.
    uint64_t ahead = work;  // tiles from its tile on
    i32x4 ra, rb, sra, srb;
    int ikb = 0, iKB = 0, vsa = 0, vsb = 0;
    auto open_tile = [&]() __attribute__((always_inline)) {  // the first of `ahead`; none: nothing is read
        const WgradTile w = list.get(p, ahead ? __builtin_ctzll(ahead) : 0);
        ikb = 0;
        iKB = ahead ? w.KB : 0x7FFFFFFF;
        // (the range check takes the lane's and the scalar offset together)
        ra = make_rsrc(p.gt + w.n0 * ld + (int64_t)w.b0 * 128, ahead ? (uint64_t)((w.nrow - 1) * ld + w.KB * 128) : 0);
        rb = make_rsrc(p.xt + w.k0 * ld + (int64_t)w.b0 * 128, ahead ? (uint64_t)((w.ncol - 1) * ld + w.KB * 128) : 0);
        sra = make_rsrc(p.eg + (int64_t)w.b0 * p.N + w.n0, ahead ? (uint64_t)((w.KB - 1) * p.N + w.nrow) : 0);
        srb = make_rsrc(p.ex + (int64_t)w.b0 * p.K + w.k0, ahead ? (uint64_t)((w.KB - 1) * p.K + w.ncol) : 0);
        const int a = wm * 64 + 4 * i;
        vsa = a < w.nrow ? a : kOutOfRange;
        vsb = col < w.ncol ? col : kOutOfRange;
        uniform(ra);
        uniform(rb);
        uniform(sra);
        uniform(srb);
        ahead &= ahead - 1;
    };
    auto copy_a = [&](int j, int slot) __attribute__((always_inline)) {
        fp8q_raw_buffer_load_lds(ra, (lds_ptr)(lds + slot * kSlot + (wave * 4 + j) * 1024), 16, avoff[j & 1],
                                 ikb * 128 + (j >> 1) * (int)ld, 0, 0);
    };
    auto copy_b = [&](int j, int slot) __attribute__((always_inline)) {
        fp8q_raw_buffer_load_lds(rb, (lds_ptr)(lds + slot * kSlot + (wave * 4 + j) * 1024), 16, bvoff[j & 1],
                                 ikb * 128 + (j >> 1) * (int)ld, 0, 0);
    };
    auto scales = [&](uint32_t (&s)[3]) __attribute__((always_inline)) {
        s[0] = __float_as_uint(fp8q_raw_buffer_load_f32(sra, vsa, ikb * (int)p.N, 0));
        if constexpr (EXACT) {
            s[1] = __float_as_uint(fp8q_raw_buffer_load_f32(srb, vsb, ikb * (int)p.K, 0));
            // (Past the tile's columns these are other columns' bytes, or zeros: they meet codes of zero, and no result is
            // stored.)
            s[2] = __float_as_uint(fp8q_raw_buffer_load_f32(srb, (int)((uint32_t)vsb + 64u), ikb * (int)p.K, 0));
        } else {
            const fp8q_i32x2 both = fp8q_raw_buffer_load_b64(srb, vsb, ikb * (int)p.K, 0);
            s[1] = (uint32_t)both[0];
            s[2] = (uint32_t)both[1];
        }
    };
    // Chunk 2 g of the lane's row of a wave's first subtile; chunk 2 g + 1: ^ 16.
    const int chunk = ((2 * g) ^ (i & 7) ^ (i >> 3)) << 4;
    const int fa_at = wm * 8192 + i * 128 + chunk, fb_at = wn * 16384 + i * 128 + chunk;
    auto read8 = [&](int at0, int at1, int off) __attribute__((always_inline)) {  // 32 codes of a row: both chunks
        const u32x4 lo = *reinterpret_cast<const u32x4 *>(lds + at0 + off);
        const u32x4 hi = *reinterpret_cast<const u32x4 *>(lds + at1 + off);
        v8i f;
        f[0] = (int)lo[0]; f[1] = (int)lo[1]; f[2] = (int)lo[2]; f[3] = (int)lo[3];
        f[4] = (int)hi[0]; f[5] = (int)hi[1]; f[6] = (int)hi[2]; f[7] = (int)hi[3];
        return f;
    };

    auto read4 = [&](int at, int off) __attribute__((always_inline)) {  // 16 codes of a row: a chunk
        return *reinterpret_cast<const v4i *>(lds + at + off);
    };

    // The lane, so that the compiler does not form the stores' addresses before the loop: 5 to 11 registers of the fp32 form
    // spilled then, and a reload waits for all copies before it.
    auto lane_again = []() __attribute__((always_inline)) {
        int l = (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
        asm volatile("" : "+v"(l));
        return l;
    };
    uint32_t sc[2][3];  // block s's are in sc[s % 2]
    open_tile();
    scales(sc[0]);
#pragma unroll
    for (int j = 0; j < 4; j++) copy_a(j, 0);
#pragma unroll
    for (int j = 0; j < 4; j++) copy_b(j, 1);
    if (++ikb >= iKB) open_tile();
#pragma unroll
    for (int j = 0; j < 4; j++) copy_a(j, 2);
#pragma unroll
    for (int j = 0; j < 4; j++) copy_b(j, 3);
    copies_barrier<8>();  // block 0 is there
    int slot = 0;
    auto wrap = [](int s) { return s >= kSlots ? s - kSlots : s; };
    v4f acc[4][8];
    bool stored = false;  // a tile's results were stored between this block and the one before
    // Block s + 1 is there: younger are this block's 4 copies and its scales' loads, and a finished tile's stores, which need not have
    // reached memory.  (The compiler would move matrix instructions before the branch behind it.)
    auto next_block_is_there = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int a = 0; a < 4; a++)
#pragma unroll
            for (int b = 0; b < (EXACT ? 6 : 5); b++) asm volatile("" : "+v"(acc[a][b]));
        if (stored)
            copies_barrier<4 + kScaleLoads<EXACT> + kStores<EXACT>>();
        else
            copies_barrier<4 + kScaleLoads<EXACT>>();
        __builtin_amdgcn_sched_barrier(0);
    };
    // Fragments that are alive between blocks: for bf16 the codes of 4 rows (32 of each) and of up to 4 columns; for fp32
    // the 4 rows widened (16 codes of each) and the codes of up to 3 columns.
    v8i fa[EXACT ? 1 : 4], fb[EXACT ? 1 : 4];
    v8bf wide[EXACT ? 4 : 1][2];
    v4i raw[EXACT ? 3 : 1];
    if constexpr (!EXACT) {
#pragma unroll
        for (int a = 0; a < 4; a++) fa[a] = read8(fa_at, fa_at ^ 16, a * 2048);
#pragma unroll
        for (int b = 0; b < 3; b++) fb[b] = read8(kSlot + fb_at, kSlot + (fb_at ^ 16), b * 2048);
    } else {
#pragma unroll
        for (int b = 0; b < 2; b++) raw[b] = read4(kSlot + fb_at, b * 2048);
#pragma unroll
        for (int a = 0; a < 4; a++) widen16(read4(fa_at, a * 2048), power_of(sc[0][0], a), wide[a]);
    }
    auto mfma = [&](const uint32_t (&s)[3], auto a_, auto b_) __attribute__((always_inline)) {
        constexpr int a = decltype(a_)::value, b = decltype(b_)::value;
        acc[a][b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fa[a], fb[b & 3], acc[a][b], 0, 0, a, (int)s[0], b & 3,
                                                                     (int)s[1 + b / 4]);
    };
    // One block.  Phases 0 to 4: column subtile b by the 4 row subtiles, while subtile b + 3 is read.  Then everything of
    // the block is in registers: the barrier frees its slots, and subtiles 5 to 7 are taken row by row, each row's fragment
    // being replaced by the next block's when it is done.  (Every other phase runs backwards, so that one operand changes
    // from MFMA to MFMA.)
    auto block = [&](auto turn_) __attribute__((always_inline)) {
        constexpr int turn = decltype(turn_)::value;
        uint32_t(&s)[3] = sc[turn];
        const int nA = wrap(slot + 2), last = wrap(slot + 4);
        const int b0 = wrap(slot + 1) * kSlot + fb_at, b1 = b0 ^ 16;             // this block's columns
        const int nb0 = wrap(slot + 3) * kSlot + fb_at, nb1 = nb0 ^ 16;          // the next block's
        const int na0 = nA * kSlot + fa_at, na1 = na0 ^ 16;
        scales(sc[turn ^ 1]);
        if (++ikb >= iKB) open_tile();  // (here, where no matrix instruction could be moved behind its branch)
        if constexpr (!EXACT) {
            static_for<5>([&](auto b_) __attribute__((always_inline)) {
                constexpr int b = decltype(b_)::value;
                fb[(b + 3) & 3] = read8(b0, b1, (b + 3) * 2048);
                if constexpr (b < 4) copy_a(b, last);
                static_for<4>([&](auto a_) __attribute__((always_inline)) {
                    mfma(s, Index<(b & 1) ? 3 - decltype(a_)::value : decltype(a_)::value>{}, b_);
                });
                __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
                if constexpr (b < 4) __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x008, 4, 0);
                __builtin_amdgcn_sched_barrier(0);
            });
            next_block_is_there();
            fb[0] = read8(nb0, nb1, 0);
            static_for<4>([&](auto a_) __attribute__((always_inline)) {
                constexpr int a = decltype(a_)::value;
                copy_b(a, slot);
                static_for<3>([&](auto c_) __attribute__((always_inline)) {
                    constexpr int c = decltype(c_)::value;
                    mfma(s, a_, Index<5 + ((a & 1) ? 2 - c : c)>{});
                });
                fa[a] = read8(na0, na1, a * 2048);
                __builtin_amdgcn_sched_barrier(0);
            });
            fb[1] = read8(nb0, nb1, 2048);
            fb[2] = read8(nb0, nb1, 2 * 2048);
        } else {
            const int a1 = (slot * kSlot + fa_at) ^ 16;
            static_for<2>([&](auto half_) __attribute__((always_inline)) {
                constexpr int half = decltype(half_)::value;
                // (the compiler is not to keep the powers of one half for the other: their registers would be missing)
                asm volatile("" : "+v"(s[0]), "+v"(s[1]), "+v"(s[2]));
                v4i rows[4];
                v8bf cols[2][2];
                widen16(raw[0], power_of(s[1], 0), cols[0]);
                static_for<6>([&](auto b_) __attribute__((always_inline)) {
                    constexpr int b = decltype(b_)::value;
                    raw[(b + 2) % 3] = read4(half ? b1 : b0, (b + 2) * 2048);
                    if constexpr (half == 0 && b < 4) copy_a(b, last);
                    if constexpr (half == 0 && b > 3) rows[b - 4] = read4(a1, (b - 4) * 2048);
                    // (the next column's codes are widened beside this one's products)
                    widen16(raw[(b + 1) % 3], power_of(s[1 + (b + 1) / 4], (b + 1) & 3), cols[(b + 1) & 1]);
#pragma unroll
                    for (int h = 0; h < 2; h++)
#pragma unroll
                        for (int a = 0; a < 4; a++)
                            acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wide[a][h], cols[b & 1][h], acc[a][b], 0, 0, 0);
                    __builtin_amdgcn_sched_barrier(0);
                });
                if constexpr (half == 1) {
                    next_block_is_there();
#pragma unroll
                    for (int a = 0; a < 2; a++) rows[a] = read4(na0, a * 2048);
                }
                widen16(raw[7 % 3], power_of(s[2], 3), cols[1]);  // columns 6 and 7
#pragma unroll
                for (int b = 0; b < 2; b++) raw[b] = read4(half ? nb0 : b1, b * 2048);
                __builtin_amdgcn_sched_barrier(0);
                static_for<4>([&](auto a_) __attribute__((always_inline)) {
                    constexpr int a = decltype(a_)::value;
                    if constexpr (half == 1) copy_b(a, slot);
                    if constexpr (a < 2) rows[a + 2] = read4(half ? na0 : a1, (a + 2) * 2048);
#pragma unroll
                    for (int h = 0; h < 2; h++)
#pragma unroll
                        for (int c = 0; c < 2; c++)
                            acc[a][6 + c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wide[a][h], cols[c][h], acc[a][6 + c], 0, 0, 0);
                    widen16(rows[a], power_of(half ? sc[turn ^ 1][0] : s[0], a), wide[a]);
                    if constexpr (half == 1) asm volatile("" : "+v"(wide[a][0]), "+v"(wide[a][1]));  // (not behind the branch)
                    __builtin_amdgcn_sched_barrier(0);
                });
            });
        }
        slot = nA;
        stored = false;
    };
#define FP8Q_WGRAD_ZERO()                         \
    _Pragma("unroll") for (int a = 0; a < 4; a++) \
        _Pragma("unroll") for (int b = 0; b < 8; b++) acc[a][b] = (v4f){0.f, 0.f, 0.f, 0.f};
    FP8Q_WGRAD_ZERO()
    uint64_t todo = work;  // tiles from the one being multiplied on
    int left = list.get(p, __builtin_ctzll(todo)).KB;
    for (;;) {
        // (two blocks at a time, so that a block's scales stay in the registers that they were loaded into)
#define FP8Q_WGRAD_STEP(TURN)                                                                                  \
    block(Index<TURN>{});                                                                                      \
    if (--left == 0) {                                                                                         \
        wgrad_store<EXACT, ACCUMULATE>(p, acc, list.get(p, __builtin_ctzll(todo)),                             \
                                       wm * 64 + 16 * (lane_again() >> 4),                                     \
                                       wn * 128 + (EXACT ? 4 : 8) * (lane_again() & 15));                      \
        todo &= todo - 1;                                                                                      \
        if (todo == 0) break;                                                                                  \
        left = list.get(p, __builtin_ctzll(todo)).KB;                                                          \
        stored = true;                                                                                         \
        FP8Q_WGRAD_ZERO()                                                                                      \
    }
        FP8Q_WGRAD_STEP(0)
        FP8Q_WGRAD_STEP(1)
#undef FP8Q_WGRAD_STEP
#undef FP8Q_WGRAD_ZERO
    }
    __builtin_amdgcn_s_waitcnt(0);  // the last (zero-byte) copies have retired before the workgroup ends
}

int64_t tiles_of(int64_t n, int64_t t) { return (n + t - 1) / t; }

// 128 x 128 tiles where all of them are under way at once, two to a CU; 256 x 256 tiles else.  us by large and by small tiles,
// 4096 tokens: 576 x 7168 (280 small tiles) bf16 47, 29, fp32 87, 52; 4096 x 2048 (512) 50, 34 and 96, 65; 2816 x 3584 (616)
// 50, 50 and 97, 84; 4096 x 4096 (1024) 51, 61 and 98, 112.  The rule is one for both types: fp32 results just past it lose by
// it (2816 x 3584; 16 experts of 1024 x 1024, 1024 rows each: 49, 42), bf16 ones do not (27, 31).
bool large_tiles(int64_t E, int64_t N, int64_t K) { return E * tiles_of(N, kTile) * tiles_of(K, kTile) > 2 * cu_count(); }

// Parts of a tile's blocks (small tiles, one product), by estimated time in us: a block of a tile takes 0.6 with one
// workgroup to a CU and 1.0 with two (fp32: 0.95 and 1.6), a second launch 4, and every part a write and a read of N K sums
// at 5 TB/s.
int64_t wgrad_parts(int64_t M, int64_t N, int64_t K, bool out_bf16) {
    if (large_tiles(1, N, K)) return 1;
    const int64_t blocks = M / 128, tiles = tiles_of(N, kTile) * tiles_of(K, kTile), cu = cu_count();
    int64_t best = 1;
    double least = 0;
    for (int64_t parts = 1; parts <= 64 && parts <= blocks; parts++) {
        const int64_t each = tiles_of(blocks, parts), wgs = tiles * parts;
        if (parts > 1 && wgs > 2 * cu) break;
        if (each * (parts - 1) >= blocks) continue;  // the last would have none
        const double block = (out_bf16 ? 1.0 : 1.6) * (wgs <= cu ? 0.6 : (double)tiles_of(wgs, 2 * cu));
        const double t = (double)each * block + (parts > 1 ? 4.0 + (double)parts * (double)(N * K) * 8.0 / 5e6 : 0.0);
        if (parts == 1 || t < least) {
            least = t;
            best = parts;
        }
    }
    return best;
}

template <bool EXACT, bool ACCUMULATE>
hipError_t launch_wgrad(WgradArgs p, hipStream_t stream) {
    constexpr int kHow = EXACT ? (ACCUMULATE ? kAddF32 : kStoreF32) : (ACCUMULATE ? kAddBf16 : kStoreBf16);
    if (large_tiles(p.E, p.N, p.K)) {
        p.n_tiles = tiles_of(p.N, 256);
        p.k_tiles = tiles_of(p.K, 256);
        const int64_t wgs = tiles_of(p.E * p.n_tiles * p.k_tiles, 256 * kMostTiles) * 256;
        wgrad_stream_kernel<EXACT, ACCUMULATE><<<dim3((unsigned)wgs), 512, 0, stream>>>(p);
        return hipGetLastError();
    }
    p.n_tiles = tiles_of(p.N, kTile);
    p.k_tiles = tiles_of(p.K, kTile);
    if (p.parts > 1) {
        wgrad_small_kernel<EXACT, kParts><<<dim3((unsigned)(p.parts * p.n_tiles * p.k_tiles)), 256, 0, stream>>>(p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        wgrad_parts_kernel<kHow><<<dim3((unsigned)tiles_of(p.N * p.K, 1024)), 256, 0, stream>>>(p);
        return hipGetLastError();
    }
    const int64_t wgs = tiles_of(p.E * p.n_tiles * p.k_tiles, 256) * 256;
    wgrad_small_kernel<EXACT, kHow><<<dim3((unsigned)wgs), 256, 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace

int64_t gemm_wgrad_workspace_bytes(int64_t M, int64_t N, int64_t K, bool out_bf16) {
    const int64_t parts = N > 0 && K > 0 ? wgrad_parts(M, N, K, out_bf16) : 1;
    return parts > 1 ? parts * N * K * 4 : 0;
}

int64_t gemm_wgrad_blocks(int64_t N, int64_t K, int64_t E) {
    const int64_t per = tiles_of(N, kTile) * tiles_of(K, kTile);
    if (per > 0 && E > (int64_t(1) << 40) / per) return -1;
    return per * E + 256;
}

hipError_t launch_gemm_wgrad(const uint8_t *gt, const uint8_t *eg, const uint8_t *xt, const uint8_t *ex, void *dw,
                             bool out_bf16, bool accumulate, const int32_t *off, int64_t E, int64_t M, int64_t N,
                             int64_t K, float *workspace, hipStream_t stream) {
    const WgradArgs p = {gt, eg, xt, ex, dw, off, M, N, K, E, 0, 0, workspace, off == nullptr ? wgrad_parts(M, N, K, out_bf16) : 1};
    if (out_bf16) return accumulate ? launch_wgrad<false, true>(p, stream) : launch_wgrad<false, false>(p, stream);
    return accumulate ? launch_wgrad<true, true>(p, stream) : launch_wgrad<true, false>(p, stream);
}

}  // namespace fp8q
