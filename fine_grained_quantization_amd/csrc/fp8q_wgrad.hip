// Weight gradients from transposed copies, dense and per expert:
//   dW[n][k] = sum_mb 2^(eg[mb][n] + ex[mb][k] - 254) * sum_{m in mb} gt[n][m] xt[k][m]   (+ dW)
// with E4M3 codes in groups of 128 tokens of one channel and one power of two each, so that a group's scale is a scale of
// the matrix instruction and nothing is left to do between two blocks of tokens.
//
// Two forms, by the result's type:
//  - bf16: v_mfma_scale_f32_16x16x128_f8f6f4, a block of 128 tokens per instruction, scales applied by it.  The E4M3 MFMAs
//    line their 128 products up before adding them and cut what falls below: each result is 1.4e-5 (relative, rms, for codes
//    of normal values) off the exact sum, at K = 128 as at K = 32768, without a bias.  That is 1/100 of bf16's own rounding.
//  - fp32: the codes, times their scales, become bf16 (exactly: 4 significant bits and a power of two) in registers, and
//    v_mfma_f32_16x16x32_bf16 adds them to 1e-7.  Half of the peak rate.
#include "fp8q_device.h"
#include "fp8q_kernels.h"
#include "fp8q_tiles.h"

namespace fp8q {
namespace {

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
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
};

// Rows in groups of 64: row 4 i + j of a group is row i of the group's 16-row subtile j.  So a lane's scale bytes of the 4
// subtiles are one dword (the instruction picks the byte), and in the result the 4 subtiles of a column group are 4
// consecutive columns.  A tile row (128 codes, 8 chunks of 16) holds logical chunk c at c ^ wswz(row): a fragment read
// touches rows 4 i + j of 16 i at one chunk, and the chunks of 8 neighbouring i are all different.
__device__ __forceinline__ int wswz(int r) { return ((r >> 2) & 7) ^ ((r >> 5) & 1); }

__device__ __forceinline__ v8i wfrag(const uint8_t *tile, int r, int g) {
    const u32x4 lo = *reinterpret_cast<const u32x4 *>(tile + r * 128 + (((2 * g) ^ wswz(r)) << 4));
    const u32x4 hi = *reinterpret_cast<const u32x4 *>(tile + r * 128 + (((2 * g + 1) ^ wswz(r)) << 4));
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

template <int WM, int WN, int CG>
struct WgradShape {
    static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
    static constexpr int BM = 64 * WM, BN = 64 * CG * WN;
    static constexpr int kScale = (BM + BN) * 128;           // scale bytes behind the codes: rows, then columns
    static constexpr int kStage = kScale + 1024;
    static constexpr int kCopyA = BM / 8 / kWaves, kCopyB = BN / 8 / kWaves;
};

// One tile of BM rows (n) x BN columns (k) by WM x WN waves of 64 x 64 CG.
template <bool EXACT, bool ACCUMULATE, int WM, int WN, int CG>
__global__ __launch_bounds__(64 * WM * WN, 2) void wgrad_kernel(WgradArgs p) {
    using S = WgradShape<WM, WN, CG>;
    __shared__ __attribute__((aligned(1024))) uint8_t stage0[S::kStage];
    __shared__ __attribute__((aligned(1024))) uint8_t stage1[S::kStage];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const int i = lane & 15, g = lane >> 4;
    const int64_t per = p.n_tiles * p.k_tiles;
    // (dense: the XCD order spreads the tiles over all workgroups of a round, so blockIdx may be past the number of tiles)
    const int64_t e = p.off == nullptr ? 0 : blockIdx.x / per;
    int64_t nt, kt;
    if (p.off == nullptr) {
        if (!dense_tile_at(xcd_order(blockIdx.x), p.n_tiles, p.k_tiles, nt, kt)) return;
    } else {
        if (e >= p.E) return;
        const int64_t r = blockIdx.x - e * per;
        nt = r / p.k_tiles;
        kt = r % p.k_tiles;
    }
    const int64_t n0 = nt * S::BM, k0 = kt * S::BN;
    // the segment, cut to [0, M) and to whole blocks
    int64_t lo = 0, hi = p.M;
    if (p.off != nullptr) {
        lo = p.off[e];
        hi = p.off[e + 1];
        lo = lo < 0 ? 0 : (lo > p.M ? p.M : lo & ~127);
        hi = hi < lo ? lo : (hi > p.M ? p.M : hi & ~127);
    }
    const int b0 = __builtin_amdgcn_readfirstlane((int)(lo >> 7));
    const int KB = __builtin_amdgcn_readfirstlane((int)((hi - lo) >> 7));
    const int64_t ld = p.M;
    const int64_t nrow = p.N - n0 < S::BM ? p.N - n0 : S::BM, ncol = p.K - k0 < S::BN ? p.K - k0 : S::BN;
    const i32x4 ra = make_rsrc(p.gt + n0 * ld + (int64_t)b0 * 128, (uint64_t)((nrow - 1) * ld + (int64_t)KB * 128));
    const i32x4 rb = make_rsrc(p.xt + k0 * ld + (int64_t)b0 * 128, (uint64_t)((ncol - 1) * ld + (int64_t)KB * 128));
    int av[S::kCopyA], bv[S::kCopyB];
#pragma unroll
    for (int j = 0; j < S::kCopyA; j++) {
        const int r = (wave * S::kCopyA + j) * 8 + (lane >> 3);
        av[j] = r < nrow ? (int)(r * ld) + (((lane & 7) ^ wswz(r)) << 4) : kOutOfRange;
    }
#pragma unroll
    for (int j = 0; j < S::kCopyB; j++) {
        const int r = (wave * S::kCopyB + j) * 8 + (lane >> 3);
        bv[j] = r < ncol ? (int)(r * ld) + (((lane & 7) ^ wswz(r)) << 4) : kOutOfRange;
    }
    // Block kb's codes and scale bytes into a stage; past the last block nothing is read (zeros land).
    auto issue = [&](uint8_t *st, int kb) __attribute__((always_inline)) {
        const bool in = kb < KB;
        const i32x4 ta = in ? ra : empty_rsrc(ra), tb = in ? rb : empty_rsrc(rb);
        const int so = in ? kb * 128 : 0;
        if (wave < 2) {  // 4 scale bytes a lane: wave 0 the rows', wave 1 the columns'
            const bool rows = wave == 0;
            const int64_t n = rows ? nrow : ncol;
            const i32x4 rs = make_rsrc((rows ? p.eg + (int64_t)(b0 + kb) * p.N + n0 : p.ex + (int64_t)(b0 + kb) * p.K + k0),
                                       in ? (uint64_t)n : 0);
            fp8q_raw_buffer_load_lds(rs, (lds_ptr)(st + S::kScale + wave * 512), 4, lane * 4, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < S::kCopyA; j++)
            fp8q_raw_buffer_load_lds(ta, (lds_ptr)(st + (wave * S::kCopyA + j) * 1024), 16, av[j], so, 0, 0);
#pragma unroll
        for (int j = 0; j < S::kCopyB; j++)
            fp8q_raw_buffer_load_lds(tb, (lds_ptr)(st + S::BM * 128 + (wave * S::kCopyB + j) * 1024), 16, bv[j], so, 0, 0);
    };
    v4f acc[4][CG * 4];
#pragma unroll
    for (int a = 0; a < 4; a++)
#pragma unroll
        for (int b = 0; b < CG * 4; b++) acc[a][b] = (v4f){0.f, 0.f, 0.f, 0.f};
    issue(stage0, 0);
    for (int kb = 0; kb < KB; kb++) {
        uint8_t *cur = (kb & 1) ? stage1 : stage0, *nxt = (kb & 1) ? stage0 : stage1;
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
        issue(nxt, kb + 1);
        const uint8_t *tB = cur + S::BM * 128;
        const uint32_t sa = *reinterpret_cast<const uint32_t *>(cur + S::kScale + wm * 64 + 4 * i);
        v8i af[4];
        v8bf ab[EXACT ? 4 : 1][4];
#pragma unroll
        for (int a = 0; a < 4; a++) af[a] = wfrag(cur, wm * 64 + 4 * i + a, g);
        if constexpr (EXACT) {
#pragma unroll
            for (int a = 0; a < 4; a++) {
                const float s = __uint_as_float(((sa >> (8 * a)) & 255u) << 23);
#pragma unroll
                for (int q = 0; q < 4; q++) ab[a][q] = to_bf16(af[a][2 * q], af[a][2 * q + 1], s);
            }
        }
        static_for<CG>([&](auto cg_) __attribute__((always_inline)) {
            constexpr int cg = decltype(cg_)::value;
            const int c0 = (wn * CG + cg) * 64 + 4 * i;
            const uint32_t sb = *reinterpret_cast<const uint32_t *>(cur + S::kScale + 512 + c0);
            static_for<4>([&](auto b_) __attribute__((always_inline)) {
                constexpr int b = decltype(b_)::value;
                const v8i bf = wfrag(tB, c0 + b, g);
                if constexpr (EXACT) {
                    const float s = __uint_as_float(((sb >> (8 * b)) & 255u) << 23);
#pragma unroll
                    for (int q = 0; q < 4; q++) {
                        const v8bf bb = to_bf16(bf[2 * q], bf[2 * q + 1], s);
#pragma unroll
                        for (int a = 0; a < 4; a++)
                            acc[a][cg * 4 + b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ab[a][q], bb, acc[a][cg * 4 + b], 0, 0, 0);
                    }
                } else {
                    static_for<4>([&](auto a_) __attribute__((always_inline)) {
                        constexpr int a = decltype(a_)::value;
                        acc[a][cg * 4 + b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            af[a], bf, acc[a][cg * 4 + b], 0, 0, a, (int)sa, b, (int)sb);
                    });
                }
            });
        });
    }
    // A lane holds, of row 4 (4 g + r) + a of the wave's 64, columns 4 i .. 4 i + 3 of each column group: 16 lanes store 64
    // consecutive columns.
    constexpr bool kBf16 = !EXACT;
    const int64_t base = e * p.N * p.K;
#pragma unroll
    for (int a = 0; a < 4; a++)
#pragma unroll
        for (int r = 0; r < 4; r++) {
            const int64_t n = n0 + wm * 64 + 4 * (4 * g + r) + a;
            if (n >= p.N) continue;
#pragma unroll
            for (int cg = 0; cg < CG; cg++) {
                const int64_t k = k0 + (wn * CG + cg) * 64 + 4 * i;
                if (k >= p.K) continue;
                const int64_t at = base + n * p.K + k;
                v4f v = {acc[a][cg * 4][r], acc[a][cg * 4 + 1][r], acc[a][cg * 4 + 2][r], acc[a][cg * 4 + 3][r]};
                if constexpr (ACCUMULATE) {
                    if constexpr (kBf16) {
                        const uint2 o = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p.dw) + at);
                        v[0] += bf16_lo(o.x); v[1] += bf16_hi(o.x); v[2] += bf16_lo(o.y); v[3] += bf16_hi(o.y);
                    } else {
                        const float4 o = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.dw) + at);
                        v[0] += o.x; v[1] += o.y; v[2] += o.z; v[3] += o.w;
                    }
                }
                store4<kBf16>(p.dw, at, v);
            }
        }
}

template <bool EXACT, bool ACCUMULATE>
hipError_t launch_wgrad(WgradArgs p, hipStream_t stream) {
    auto tiles = [](int64_t n, int64_t t) { return (n + t - 1) / t; };
    if (p.E * tiles(p.N, 256) * tiles(p.K, 256) >= cu_count()) {
        using S = WgradShape<4, 2, 2>;
        p.n_tiles = tiles(p.N, S::BM);
        p.k_tiles = tiles(p.K, S::BN);
        const dim3 grid((unsigned)((p.E * p.n_tiles * p.k_tiles + 255) / 256 * 256));
        wgrad_kernel<EXACT, ACCUMULATE, 4, 2, 2><<<grid, S::kThreads, 0, stream>>>(p);
    } else {
        using S = WgradShape<2, 2, 1>;
        p.n_tiles = tiles(p.N, S::BM);
        p.k_tiles = tiles(p.K, S::BN);
        const dim3 grid((unsigned)((p.E * p.n_tiles * p.k_tiles + 255) / 256 * 256));
        wgrad_kernel<EXACT, ACCUMULATE, 2, 2, 1><<<grid, S::kThreads, 0, stream>>>(p);
    }
    return hipGetLastError();
}

}  // namespace

int64_t gemm_wgrad_workspace_bytes(int64_t, int64_t, int64_t, bool) { return 0; }

int64_t gemm_wgrad_blocks(int64_t N, int64_t K, int64_t E) {
    const int64_t per = ((N + 127) / 128) * ((K + 127) / 128);
    if (per > 0 && E > (int64_t(1) << 40) / per) return -1;
    return per * E + 256;
}

hipError_t launch_gemm_wgrad(const uint8_t *gt, const uint8_t *eg, const uint8_t *xt, const uint8_t *ex, void *dw,
                             bool out_bf16, bool accumulate, const int32_t *off, int64_t E, int64_t M, int64_t N,
                             int64_t K, float *, hipStream_t stream) {
    const WgradArgs p = {gt, eg, xt, ex, dw, off, M, N, K, E, 0, 0};
    if (out_bf16) return accumulate ? launch_wgrad<false, true>(p, stream) : launch_wgrad<false, false>(p, stream);
    return accumulate ? launch_wgrad<true, true>(p, stream) : launch_wgrad<true, false>(p, stream);
}

}  // namespace fp8q
