// Pieces that the gfx950 matrix product kernels share: the LDS placement of a tile row, buffer resources, the
// order in which tiles are dealt to the XCDs, the tiles of an expert-sorted layout, and 4-wide output stores.
#pragma once

#include "fp8q_device.h"

namespace fp8q {

// Multiprocessor count of the current device (cached).
int cu_count();

namespace {

// LDS placement of a tile row: row r (128 bytes = 8 chunks of 16 bytes) stores logical chunk c at
// physical chunk c ^ swzf(r).  Fragment reads touch 16 consecutive rows at one logical chunk; swzf is a
// permutation of 0..7 within each aligned group of 8 rows and also within the 8 even and the 8 odd
// rows of each aligned group of 16, so those reads are bank-conflict free whether the LDS serves 8
// lanes (128 bytes) or 16 lanes (256 bytes) of a 16-byte read per cycle.
__device__ __forceinline__ int swzf(int r) { return (r & 7) ^ ((r >> 3) & 1); }
__device__ __forceinline__ int swz(int r, int c) { return r * 128 + ((c ^ swzf(r)) << 4); }

template <bool OUT_BF16>
__device__ __forceinline__ void store4(void *c, int64_t idx, const v4f &v) {
    if (OUT_BF16) {
        uint2 o;
        o.x = pack_bf16x2(v[0], v[1]);
        o.y = pack_bf16x2(v[2], v[3]);
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(c) + idx) = o;
    } else {
        *reinterpret_cast<float4 *>(static_cast<float *>(c) + idx) = make_float4(v[0], v[1], v[2], v[3]);
    }
}

typedef __attribute__((address_space(3))) void *lds_ptr;

// Buffer resource for `bytes` bytes at `base` (raw buffer: stride 0, range-checked by byte offset).
__device__ __forceinline__ i32x4 make_rsrc(const void *base, uint64_t bytes) {
    const uint64_t a = reinterpret_cast<uint64_t>(base);
    i32x4 r;
    r[0] = (int)(uint32_t)a;
    r[1] = (int)(uint32_t)(a >> 32);  // stride 0
    r[2] = (int)(uint32_t)(bytes < 0xFFFFFFFFull ? bytes : 0xFFFFFFFFull);
    r[3] = 0x00020000;
    return r;
}

// The same resource with a byte count of 0: every load through it is out of range and returns zeros without
// touching memory, whatever its per-lane and scalar offsets.
__device__ __forceinline__ i32x4 empty_rsrc(i32x4 r) {
    r[2] = 0;
    return r;
}

// Workgroups are dispatched to the 8 XCDs round-robin (t % 8), 256 of them (one per CU) at a time.  This
// permutation gives XCD x the 32 consecutive indices [256 r + 32 x, +32) of each round r of 256; it is a
// bijection on every whole round.
__device__ __forceinline__ int64_t xcd_order(int64_t t) { return (t / 256) * 256 + (t % 8) * 32 + (t % 256) / 8; }

// Tile (mt, nt) of the i-th tile of a dense n_mt x n_nt grid, in an order made for the XCD permutation above:
// columns of 16 N tiles ("supergroup columns", the last may be narrower), each cut into supergroups of 16 M
// tiles (the last may be shorter), each enumerated as 8-wide sub-block columns of 4-high sub-blocks, M
// fastest.  Only tiles inside the grid are enumerated, so every round of 256 indices is 256 tiles whatever the
// grid's shape.  In a full 16 x 16 supergroup each XCD's 32 tiles form a 4 (M) x 8 (N) block sharing 4
// activation and 8 weight tile rows in that XCD's L2, and a round's 16 x 16 square shares its operands in the
// Infinity Cache.  Returns false past the last tile.
__device__ __forceinline__ bool dense_tile_at(int64_t i, int64_t n_mt, int64_t n_nt, int64_t &mt, int64_t &nt) {
    if (i >= n_mt * n_nt) return false;
    const int64_t colw = 16 * n_mt;
    const int64_t sgn = i / colw;
    const int64_t hn = n_nt - 16 * sgn < 16 ? n_nt - 16 * sgn : 16;
    int64_t j = i - sgn * colw;
    const int64_t sgm = j / (16 * hn);
    const int64_t hm = n_mt - 16 * sgm < 16 ? n_mt - 16 * sgm : 16;
    j -= sgm * 16 * hn;
    const int64_t qn = j / (8 * hm);
    const int64_t wq = hn - 8 * qn < 8 ? hn - 8 * qn : 8;
    j -= qn * 8 * hm;
    const int64_t qm = j / (4 * wq);
    const int64_t hq = hm - 4 * qm < 4 ? hm - 4 * qm : 4;
    j -= qm * 4 * wq;
    mt = 16 * sgm + 4 * qm + j % hq;
    nt = 16 * sgn + 8 * qn + j / hq;
    return true;
}

// Coordinates of grouped tile t: tiles are enumerated expert by expert (expert e owns ceil(len_e / BM) M
// tiles of its segment), tile T = mt * n_ntiles + nt with N fastest.  Workgroups are dealt to the 8 XCDs
// round-robin; the permutation below gives XCD x the 32 consecutive tiles [256 r + 32 x, +32) of each round r
// of 256, so the tiles sharing activation rows (and, mostly, an expert's weights) meet in one L2.  Returns
// false past the last expert's tiles.
template <int BM>
__device__ __forceinline__ bool grouped_tile(int64_t t, const int32_t *__restrict__ off, int64_t E, int64_t M,
                                             int64_t n_mtiles, int64_t n_ntiles, int64_t bn, int lane, int64_t &m0,
                                             int64_t &mend, int64_t &n0, int64_t &e) {
    const int64_t T = xcd_order(t);
    const int64_t mt = T / n_ntiles;  // n_mtiles is an upper bound on the number of M tiles
    if (mt >= n_mtiles) return false;
    n0 = (T % n_ntiles) * bn;
    // The expert owning M tile mt: a prefix sum of the experts' tile counts, 64 experts per pass (lane i
    // holds expert base + i), and the first lane whose running total exceeds mt.
    // A segment is cut to [0, M) before its tiles are counted (in 64-bit arithmetic), so offsets that break
    // the layout rules can neither overflow the count nor yield rows outside the buffer.
    int64_t before = 0;
    for (int64_t base = 0; base < E; base += 64) {
        const int64_t i = base + lane;
        int lo = 0, hi = 0, cnt = 0;
        if (i < E) {
            const int64_t l = (int64_t)off[i] < 0 ? 0 : ((int64_t)off[i] > M ? M : (int64_t)off[i]);
            const int64_t h = (int64_t)off[i + 1] < l ? l : ((int64_t)off[i + 1] > M ? M : (int64_t)off[i + 1]);
            lo = (int)l;
            hi = (int)h;
            cnt = (int)((h - l + BM - 1) / BM);
        }
        int incl = cnt;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int u = __shfl_up(incl, d, 64);
            if (lane >= d) incl += u;
        }
        const uint64_t hit = __ballot(i < E && before + incl > mt);
        if (hit) {
            const int L = __builtin_ctzll(hit);
            e = base + L;
            const int lo_e = __shfl(lo, L, 64), hi_e = __shfl(hi, L, 64);
            const int64_t first = before + __shfl(incl, L, 64) - __shfl(cnt, L, 64);
            m0 = lo_e + (mt - first) * BM;
            mend = hi_e;
            return m0 < mend;
        }
        before += __shfl(incl, 63, 64);
    }
    return false;
}

}  // namespace
}  // namespace fp8q
