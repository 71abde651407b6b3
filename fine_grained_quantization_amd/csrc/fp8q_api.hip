// C-ABI entry points of the fp8q library (declared in include/fp8q.h): argument and device
// validation, then one launch on the caller's stream.  No allocation, no synchronization.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cstring>

#include "../../include/fp8q.h"
#include "fp8q_kernels.h"

namespace {

constexpr int kMaxDevices = 64;
// Per device: 0 = not yet checked, 1 = gfx950, 2 = other architecture.
std::atomic<int> g_device_kind[kMaxDevices];

int check_device() {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) {
        (void)hipGetLastError();
        return FP8Q_ERR_NO_DEVICE;
    }
    if (dev >= kMaxDevices) return FP8Q_ERR_UNSUPPORTED_DEVICE;
    int kind = g_device_kind[dev].load(std::memory_order_relaxed);
    if (kind == 0) {
        hipDeviceProp_t prop;
        if (hipGetDeviceProperties(&prop, dev) != hipSuccess) {
            (void)hipGetLastError();
            return FP8Q_ERR_NO_DEVICE;
        }
        kind = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
        g_device_kind[dev].store(kind, std::memory_order_relaxed);
    }
    return kind == 1 ? FP8Q_OK : FP8Q_ERR_UNSUPPORTED_DEVICE;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Element alignment of an FP8Q_OUT_* typed pointer.
bool aligned_elem(const void *p, int dtype) {
    return (reinterpret_cast<uintptr_t>(p) & (dtype == FP8Q_OUT_BF16 ? 1u : 3u)) == 0;
}

constexpr int64_t kMaxGrid = 0x7FFFFFFF;  // 1-D grids: workgroup count must fit in 31 bits
constexpr int64_t kMaxK = int64_t(1) << 23;  // GEMM tiles address 256 rows of K bytes with 32-bit offsets
// A launch has fewer than 2^32 threads: workgroups of 256 and of 512.
constexpr int64_t kMaxGrid256 = 0xFFFFFFFFll / 256, kMaxGrid512 = 0xFFFFFFFFll / 512;
constexpr int64_t kMaxGateTokens = 0xFFFFFFFFll / 64;  // 64 lanes a token at most

constexpr int64_t kMaxNormRows = int64_t(1) << 22;  // a workgroup of up to 1024 threads a row
constexpr int64_t kMaxWgrad = int64_t(1) << 20;     // 256 rows of fp32 results are addressed with 32-bit offsets
constexpr int64_t kMaxInt8K = 131056;        // INT8 sums of products of codes down to -128 stay below 2^31

int finish(hipError_t e) { return e == hipSuccess ? FP8Q_OK : FP8Q_ERR_HIP; }

static_assert(fp8q::kRouteScratchBytes == FP8Q_MOE_ROUTE_NOALLOC_BYTES, "the header states the array's size");

}  // namespace

extern "C" {

int fp8q_version(void) { return 100; }

const char *fp8q_status_string(int status) {
    switch (status) {
        case FP8Q_OK: return "FP8Q_OK: success";
        case FP8Q_ERR_NULL: return "FP8Q_ERR_NULL: a required pointer is NULL";
        case FP8Q_ERR_SHAPE: return "FP8Q_ERR_SHAPE: invalid shape (negative size, K or N not a multiple of 128, or bad grouping)";
        case FP8Q_ERR_ALIGN: return "FP8Q_ERR_ALIGN: a tensor base address is not 16-byte aligned";
        case FP8Q_ERR_DTYPE: return "FP8Q_ERR_DTYPE: unknown output dtype";
        case FP8Q_ERR_NO_DEVICE: return "FP8Q_ERR_NO_DEVICE: no HIP device available";
        case FP8Q_ERR_UNSUPPORTED_DEVICE: return "FP8Q_ERR_UNSUPPORTED_DEVICE: the current device is not gfx950 (MI355X)";
        case FP8Q_ERR_HIP: return "FP8Q_ERR_HIP: the HIP runtime reported a launch error";
        case FP8Q_ERR_WORKSPACE: return "FP8Q_ERR_WORKSPACE: the workspace is smaller than the call needs";
        case FP8Q_ERR_OPTION: return "FP8Q_ERR_OPTION: an option argument has an unknown value";
        default: return "fp8q: unknown status";
    }
}

int fp8q_quant_act_1x128(const uint16_t *x, int64_t M, int64_t K, uint8_t *q, float *s, void *stream) {
    if (M < 0 || K < 0 || K % 128) return FP8Q_ERR_SHAPE;
    if (M == 0 || K == 0) return FP8Q_OK;
    if (!x || !q || !s) return FP8Q_ERR_NULL;
    if (!aligned16(x) || !aligned16(q) || !aligned16(s)) return FP8Q_ERR_ALIGN;
    if (((M + 15) / 16) * ((K / 128 + 3) / 4) > kMaxGrid) return FP8Q_ERR_SHAPE;
    int rc = check_device();
    if (rc) return rc;
    return finish(fp8q::launch_quant_act_1x128(x, M, K, q, s, static_cast<hipStream_t>(stream)));
}

int fp8q_swiglu_quant_act_1x128(const uint16_t *x, const uint16_t *y, int64_t ld, int64_t M, int64_t K, uint8_t *q,
                                float *s, void *stream) {
    if (M < 0 || K < 0 || K % 128 || ld < K || ld % 8) return FP8Q_ERR_SHAPE;
    if (M == 0 || K == 0) return FP8Q_OK;
    if (!x || !y || !q || !s) return FP8Q_ERR_NULL;
    if (!aligned16(x) || !aligned16(y) || !aligned16(q) || !aligned16(s)) return FP8Q_ERR_ALIGN;
    if (((M + 15) / 16) * ((K / 128 + 3) / 4) > kMaxGrid) return FP8Q_ERR_SHAPE;
    int rc = check_device();
    if (rc) return rc;
    return finish(fp8q::launch_swiglu_quant_act_1x128(x, y, ld, M, K, q, s, static_cast<hipStream_t>(stream)));
}

int fp8q_quant_act_fp4_1x128(const uint16_t *x, int64_t M, int64_t K, uint8_t *q, float *s, void *stream) {
    if (M < 0 || K < 0 || K % 128) return FP8Q_ERR_SHAPE;
    if (M == 0 || K == 0) return FP8Q_OK;
    if (!x || !q || !s) return FP8Q_ERR_NULL;
    if (!aligned16(x) || !aligned16(q) || !aligned16(s)) return FP8Q_ERR_ALIGN;
    if (((M + 15) / 16) * ((K / 128 + 3) / 4) > kMaxGrid) return FP8Q_ERR_SHAPE;
    int rc = check_device();
    if (rc) return rc;
    return finish(fp8q::launch_quant_act_fp4_1x128(x, M, K, q, s, static_cast<hipStream_t>(stream)));
}

int fp8q_quant_w_fp4_128x128(const uint16_t *w, int64_t N, int64_t K, uint8_t *q, float *s, void *stream) {
    if (N < 0 || K < 0 || N % 128 || K % 128) return FP8Q_ERR_SHAPE;
    if (N == 0 || K == 0) return FP8Q_OK;
    if (!w || !q || !s) return FP8Q_ERR_NULL;
    if (!aligned16(w) || !aligned16(q) || !aligned16(s)) return FP8Q_ERR_ALIGN;
    if ((N / 128) * (K / 128) > kMaxGrid) return FP8Q_ERR_SHAPE;
    int rc = check_device();
    if (rc) return rc;
    return finish(fp8q::launch_quant_w_fp4_128x128(w, N, K, q, s, static_cast<hipStream_t>(stream)));
}

int fp8q_quant_act_e5m6_1x128(const uint16_t *x, int64_t M, int64_t K, uint8_t *q, float *s, void *stream) {
    if (M < 0 || K < 0 || K % 128) return FP8Q_ERR_SHAPE;
    if (M == 0 || K == 0) return FP8Q_OK;
    if (!x || !q || !s) return FP8Q_ERR_NULL;
    if (!aligned16(x) || !aligned16(q) || !aligned16(s)) return FP8Q_ERR_ALIGN;
    if (((M + 15) / 16) * ((K / 128 + 3) / 4) > kMaxGrid) return FP8Q_ERR_SHAPE;
    int rc = check_device();
    if (rc) return rc;
    return finish(fp8q::launch_quant_act_e5m6_1x128(x, M, K, q, s, static_cast<hipStream_t>(stream)));
}

int fp8q_quant_w_per_channel(const uint16_t *w, int64_t N, int64_t K, uint8_t *q, float *s, void *stream) {
    if (N < 0 || K < 0 || K % 8) return FP8Q_ERR_SHAPE;
    if (N == 0) return FP8Q_OK;
    if (!s || (K > 0 && (!w || !q))) return FP8Q_ERR_NULL;  // K == 0: only the (zero) scales are written
    if (!aligned4(s) || (K > 0 && (!aligned16(w) || !aligned16(q)))) return FP8Q_ERR_ALIGN;
    if (N > kMaxGrid) return FP8Q_ERR_SHAPE;  // one workgroup per row
    int rc = check_device();
    if (rc) return rc;
    return finish(fp8q::launch_quant_w_per_channel(w, N, K, q, s, static_cast<hipStream_t>(stream)));
}

int fp8q_quant_act_dual(const uint16_t *x, int64_t M, int64_t K, uint8_t *q, float *s, uint8_t *qt, float *st,
                        void *stream) {
    if (M < 0 || K < 0 || M % 128 || K % 128) return FP8Q_ERR_SHAPE;
    if (M == 0 || K == 0) return FP8Q_OK;
    if (!x || !q || !s || !qt || !st) return FP8Q_ERR_NULL;
    if (!aligned16(x) || !aligned16(q) || !aligned16(s) || !aligned16(qt) || !aligned16(st)) return FP8Q_ERR_ALIGN;
    if ((M / 128) * (K / 128) > kMaxGrid) return FP8Q_ERR_SHAPE;
    int rc = check_device();
    if (rc) return rc;
    return finish(fp8q::launch_quant_act_dual(x, M, K, q, s, qt, st, static_cast<hipStream_t>(stream)));
}

int fp8q_swiglu_bf16(const uint16_t *x, const uint16_t *y, int64_t ld, int64_t M, int64_t K, uint16_t *h,
                     void *stream) {
    if (M < 0 || K < 0 || K % 8 || ld < K || ld % 8) return FP8Q_ERR_SHAPE;
    if (M == 0 || K == 0) return FP8Q_OK;
    if (!x || !y || !h) return FP8Q_ERR_NULL;
    if (!aligned16(x) || !aligned16(y) || !aligned16(h)) return FP8Q_ERR_ALIGN;
    if (K / 8 > kMaxGrid / M * 256) return FP8Q_ERR_SHAPE;  // M * K / 2048 workgroups
    int rc = check_device();
    if (rc) return rc;
    return finish(fp8q::launch_swiglu_bf16(x, y, ld, M, K, h, static_cast<hipStream_t>(stream)));
}

int fp8q_quant_w_128x128(const uint16_t *w, int64_t N, int64_t K, uint8_t *q, float *s, void *stream) {
    if (N < 0 || K < 0 || N % 128 || K % 128) return FP8Q_ERR_SHAPE;
    if (N == 0 || K == 0) return FP8Q_OK;
    if (!w || !q || !s) return FP8Q_ERR_NULL;
    if (!aligned16(w) || !aligned16(q) || !aligned16(s)) return FP8Q_ERR_ALIGN;
    if ((N / 128) * (K / 128) > kMaxGrid) return FP8Q_ERR_SHAPE;
    int rc = check_device();
    if (rc) return rc;
    return finish(fp8q::launch_quant_w_128x128(w, N, K, q, s, static_cast<hipStream_t>(stream)));
}

int fp8q_dequant_w_128x128(const uint8_t *q, const float *s, int64_t N, int64_t K, uint16_t *w, void *stream) {
    if (N < 0 || K < 0 || N % 128 || K % 128) return FP8Q_ERR_SHAPE;
    if (N == 0 || K == 0) return FP8Q_OK;
    if (!q || !s || !w) return FP8Q_ERR_NULL;
    if (!aligned16(q) || !aligned16(s) || !aligned16(w)) return FP8Q_ERR_ALIGN;
    if (K / 128 > kMaxGrid / N * 8) return FP8Q_ERR_SHAPE;  // N * K / 8192 workgroups
    int rc = check_device();
    if (rc) return rc;
    return finish(fp8q::launch_dequant_w_128x128(q, s, N, K, w, static_cast<hipStream_t>(stream)));
}

int fp8q_gemm_blockscaled(const uint8_t *qa, const float *sa, const uint8_t *qw, const float *sw, void *c,
                          int out_dtype, int64_t M, int64_t N, int64_t K, void *stream) {
    if (M < 0 || N < 0 || K < 128 || K > kMaxK || N % 128 || K % 128) return FP8Q_ERR_SHAPE;
    if (out_dtype != FP8Q_OUT_BF16 && out_dtype != FP8Q_OUT_F32) return FP8Q_ERR_DTYPE;
    if (M == 0 || N == 0) return FP8Q_OK;
    if (!qa || !sa || !qw || !sw || !c) return FP8Q_ERR_NULL;
    if (!aligned16(qa) || !aligned16(sa) || !aligned16(qw) || !aligned16(sw) || !aligned16(c)) return FP8Q_ERR_ALIGN;
    if (fp8q::gemm_blocks(M, N) > kMaxGrid) return FP8Q_ERR_SHAPE;
    int rc = check_device();
    if (rc) return rc;
    return finish(fp8q::launch_gemm_blockscaled(qa, sa, qw, sw, c, out_dtype == FP8Q_OUT_BF16, M, N, K,
                                                static_cast<hipStream_t>(stream)));
}

int fp8q_grouped_gemm_blockscaled(const uint8_t *qa, const float *sa, const uint8_t *qw, const float *sw, void *c,
                                  int out_dtype, const int32_t *off, int64_t E, int64_t M_total, int64_t N,
                                  int64_t K, void *stream) {
    if (E < 1 || M_total < 0 || M_total % 128 || N < 0 || K < 128 || K > kMaxK || N % 128 || K % 128)
        return FP8Q_ERR_SHAPE;
    if (M_total > 0x7FFFFFFF) return FP8Q_ERR_SHAPE;  // offsets are int32
    if (out_dtype != FP8Q_OUT_BF16 && out_dtype != FP8Q_OUT_F32) return FP8Q_ERR_DTYPE;
    if (M_total == 0 || N == 0) return FP8Q_OK;
    if (!qa || !sa || !qw || !sw || !c || !off) return FP8Q_ERR_NULL;
    if (!aligned16(qa) || !aligned16(sa) || !aligned16(qw) || !aligned16(sw) || !aligned16(c)) return FP8Q_ERR_ALIGN;
    if ((reinterpret_cast<uintptr_t>(off) & 3u) != 0) return FP8Q_ERR_ALIGN;
    const int64_t blocks = fp8q::grouped_gemm_blocks(M_total, N, E);
    if (blocks < 0 || blocks > kMaxGrid) return FP8Q_ERR_SHAPE;
    int rc = check_device();
    if (rc) return rc;
    return finish(fp8q::launch_grouped_gemm_blockscaled(qa, sa, qw, sw, c, out_dtype == FP8Q_OUT_BF16, off, E,
                                                        M_total, N, K, static_cast<hipStream_t>(stream)));
}

int fp8q_grouped_gemm_blockscaled_gather(const uint8_t *q, const float *s, int64_t T, const int32_t *row_token,
                                         const uint8_t *qw, const float *sw, void *c, int out_dtype,
                                         const int32_t *off, int64_t E, int64_t M_total, int64_t N, int64_t K,
                                         void *stream) {
    if (E < 1 || M_total < 0 || M_total % 128 || N < 0 || K < 128 || K > kMaxK || N % 128 || K % 128 || T < 0)
        return FP8Q_ERR_SHAPE;
    if (M_total > 0x7FFFFFFF) return FP8Q_ERR_SHAPE;           // offsets are int32
    if (T > 0 && T > (int64_t)0x7FFFFFFF / K) return FP8Q_ERR_SHAPE;  // token offsets are 32-bit
    if (out_dtype != FP8Q_OUT_BF16 && out_dtype != FP8Q_OUT_F32) return FP8Q_ERR_DTYPE;
    if (M_total == 0 || N == 0) return FP8Q_OK;
    if (!row_token || !qw || !sw || !c || !off || (T > 0 && (!q || !s))) return FP8Q_ERR_NULL;
    if (!aligned16(qw) || !aligned16(sw) || !aligned16(c) || !aligned4(off) || !aligned4(row_token) ||
        (T > 0 && (!aligned16(q) || !aligned4(s))))
        return FP8Q_ERR_ALIGN;
    const int64_t blocks = fp8q::grouped_gemm_blocks(M_total, N, E);
    if (blocks < 0 || blocks > kMaxGrid) return FP8Q_ERR_SHAPE;
    int rc = check_device();
    if (rc) return rc;
    return finish(fp8q::launch_grouped_gemm_gather(q, s, T, row_token, qw, sw, c, out_dtype == FP8Q_OUT_BF16, off, E,
                                                   M_total, N, K, static_cast<hipStream_t>(stream)));
}

int64_t fp8q_moe_route_capacity(int64_t T, int64_t E, int64_t k) {
    if (T < 0 || E < 1 || E > fp8q::kMoeMaxExperts || k < 1 || k > E || k > fp8q::kMoeMaxK) return -1;
    if (T > (int64_t(1) << 40)) return -1;
    return (T * k + 127 * E + 127) / 128 * 128;
}

int64_t fp8q_moe_route_workspace_bytes(int64_t T, int64_t E) {
    if (T < 0 || E < 1 || E > fp8q::kMoeMaxExperts || T > (int64_t(1) << 40)) return -1;
    return fp8q::moe_route_workspace_bytes(T, E);
}

int fp8q_moe_route_topk(const float *logits, int64_t T, int64_t E, int64_t k, int32_t *topk_idx, int32_t *offsets,
                        int32_t *row_of, int32_t *row_token, int64_t rows, void *workspace, int64_t workspace_bytes,
                        void *stream) {
    const int64_t cap = fp8q_moe_route_capacity(T, E, k);
    if (cap < 0 || rows < cap || rows > 0x7FFFFFFF) return FP8Q_ERR_SHAPE;
    if (!offsets || !row_token) return FP8Q_ERR_NULL;
    if (T > 0 && (!logits || !topk_idx || !row_of || !workspace)) return FP8Q_ERR_NULL;
    if (!aligned4(offsets) || !aligned4(row_token) || (T > 0 && (!aligned4(logits) || !aligned4(topk_idx) ||
                                                                 !aligned4(row_of) || !aligned4(workspace))))
        return FP8Q_ERR_ALIGN;
    if (workspace_bytes < fp8q::moe_route_workspace_bytes(T, E)) return FP8Q_ERR_WORKSPACE;
    int rc = check_device();
    if (rc) return rc;
    return finish(fp8q::launch_moe_route_topk(logits, T, (int)E, (int)k, topk_idx, offsets, row_of, row_token, rows,
                                              static_cast<int32_t *>(workspace), static_cast<hipStream_t>(stream)));
}

int fp8q_moe_route_topk_noalloc(const float *logits, int64_t T, int64_t E, int64_t k, int32_t *topk_idx,
                                int32_t *offsets, int32_t *row_of, int32_t *row_token, int64_t rows, void *stream) {
    const int64_t cap = fp8q_moe_route_capacity(T, E, k);
    if (cap < 0 || rows < cap || rows > 0x7FFFFFFF) return FP8Q_ERR_SHAPE;
    if (!offsets || !row_token) return FP8Q_ERR_NULL;
    if (T > 0 && (!logits || !topk_idx || !row_of)) return FP8Q_ERR_NULL;
    if (!aligned4(offsets) || !aligned4(row_token) ||
        (T > 0 && (!aligned4(logits) || !aligned4(topk_idx) || !aligned4(row_of))))
        return FP8Q_ERR_ALIGN;
    if (fp8q::moe_route_workspace_bytes(T, E) > fp8q::kRouteScratchBytes) return FP8Q_ERR_WORKSPACE;
    int rc = check_device();
    if (rc) return rc;
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess) {
        (void)hipGetLastError();
        return FP8Q_ERR_NO_DEVICE;
    }
    int32_t *ws = nullptr;
    if (fp8q::route_scratch(dev, &ws) != hipSuccess) return FP8Q_ERR_HIP;
    return finish(fp8q::launch_moe_route_topk(logits, T, (int)E, (int)k, topk_idx, offsets, row_of, row_token, rows,
                                              ws, static_cast<hipStream_t>(stream)));
}

int fp8q_moe_gather_fp8(const uint8_t *q, const float *s, int64_t T, int64_t K, int64_t k, const int32_t *row_of,
                        const int32_t *row_token, const int32_t *offsets, int64_t E, int64_t rows, uint8_t *qa,
                        float *sa, void *stream) {
    if (T < 0 || T > 0x7FFFFFFF || K < 0 || K % 128 || k < 1 || k > 0x7FFFFFFF / (T > 0 ? T : 1) || E < 1 ||
        E > 0x7FFFFFFF || rows < 0 || rows > 0x7FFFFFFF)
        return FP8Q_ERR_SHAPE;
    if (rows == 0 || K == 0) return FP8Q_OK;
    if (!row_token || !offsets || !qa || !sa || (T > 0 && (!q || !s || !row_of))) return FP8Q_ERR_NULL;
    if (!aligned16(qa) || !aligned4(sa) || !aligned4(row_token) || !aligned4(offsets) ||
        (T > 0 && (!aligned16(q) || !aligned4(s) || !aligned4(row_of))))
        return FP8Q_ERR_ALIGN;
    int rc = check_device();
    if (rc) return rc;
    return finish(fp8q::launch_moe_gather_fp8(q, s, T, K, (int)k, row_of, row_token, offsets, (int)E, rows, qa, sa,
                                              static_cast<hipStream_t>(stream)));
}

int64_t fp8q_moe_gate_workspace_bytes(int64_t T, int64_t E) {
    if (T < 0 || E < 1 || E > fp8q::kMoeMaxExperts || T > (int64_t(1) << 40)) return -1;
    return fp8q::moe_gate_workspace_bytes(T, E);
}

int fp8q_moe_gate_topk(const void *logits, int dtype, int64_t ld, int64_t T, int64_t E, int64_t k, int score,
                       const float *bias, int64_t n_group, int64_t topk_group, int64_t group_top, int renormalize,
                       float scale, int32_t *topk_idx, float *topk_weight, int32_t *offsets, int32_t *row_of,
                       int32_t *row_token, int64_t rows, int32_t *load, void *workspace, int64_t workspace_bytes,
                       void *stream) {
    const int64_t cap = fp8q_moe_route_capacity(T, E, k);
    if (cap < 0 || rows < cap || rows > 0x7FFFFFFF || T > kMaxGateTokens || ld < E) return FP8Q_ERR_SHAPE;
    if (n_group < 1 || n_group > fp8q::kMoeMaxGroups || E % n_group || topk_group < 1 || topk_group > n_group ||
        k > topk_group * (E / n_group))
        return FP8Q_ERR_SHAPE;
    if (dtype != FP8Q_OUT_BF16 && dtype != FP8Q_OUT_F32) return FP8Q_ERR_DTYPE;
    if ((score != FP8Q_SCORE_SIGMOID && score != FP8Q_SCORE_SOFTMAX) || (group_top != 1 && group_top != 2) ||
        (renormalize != 0 && renormalize != 1))
        return FP8Q_ERR_OPTION;
    const int64_t need = fp8q::moe_gate_least_workspace_bytes(T, E);
    if (!offsets || !row_token) return FP8Q_ERR_NULL;
    if (T > 0 && (!logits || !topk_idx || !topk_weight || !row_of || (need > 0 && !workspace))) return FP8Q_ERR_NULL;
    if (!aligned4(offsets) || !aligned4(row_token) || !aligned4(load) || !aligned4(bias)) return FP8Q_ERR_ALIGN;
    if (T > 0 && (!aligned_elem(logits, dtype) || !aligned4(topk_idx) || !aligned4(topk_weight) ||
                  !aligned4(row_of) || (need > 0 && !aligned4(workspace))))
        return FP8Q_ERR_ALIGN;
    if (workspace_bytes < need) return FP8Q_ERR_WORKSPACE;
    int rc = check_device();
    if (rc) return rc;
    const fp8q::GateShape g = {logits, bias, ld, T, (int)E, (int)k, (int)n_group, (int)topk_group, (int)group_top,
                               scale, dtype == FP8Q_OUT_BF16, score == FP8Q_SCORE_SOFTMAX, renormalize != 0};
    return finish(fp8q::launch_moe_gate_topk(g, topk_idx, topk_weight, offsets, row_of, row_token, rows, load,
                                             workspace, workspace_bytes, static_cast<hipStream_t>(stream)));
}

int fp8q_moe_gate_backward(const void *logits, int dtype, int64_t ld, int64_t T, int64_t E, int64_t k, int score,
                           int renormalize, float scale, const int32_t *topk_idx, const float *grad_weight,
                           void *grad_logits, void *stream) {
    if (T < 0 || T > kMaxGateTokens || E < 1 || E > fp8q::kMoeMaxExperts || k < 1 || k > E || k > fp8q::kMoeMaxK || ld < E)
        return FP8Q_ERR_SHAPE;
    if (dtype != FP8Q_OUT_BF16 && dtype != FP8Q_OUT_F32) return FP8Q_ERR_DTYPE;
    if ((score != FP8Q_SCORE_SIGMOID && score != FP8Q_SCORE_SOFTMAX) || (renormalize != 0 && renormalize != 1))
        return FP8Q_ERR_OPTION;
    if (T == 0) return FP8Q_OK;
    if (!logits || !topk_idx || !grad_weight || !grad_logits) return FP8Q_ERR_NULL;
    if (!aligned_elem(logits, dtype) || !aligned4(topk_idx) || !aligned4(grad_weight) ||
        !aligned_elem(grad_logits, dtype))
        return FP8Q_ERR_ALIGN;
    int rc = check_device();
    if (rc) return rc;
    const fp8q::GateShape g = {logits, nullptr, ld, T, (int)E, (int)k, 1, 1, 1, scale, dtype == FP8Q_OUT_BF16,
                               score == FP8Q_SCORE_SOFTMAX, renormalize != 0};
    return finish(fp8q::launch_moe_gate_backward(g, topk_idx, grad_weight, grad_logits,
                                                 static_cast<hipStream_t>(stream)));
}

int fp8q_moe_combine(const void *c, int dtype, int64_t rows, int64_t H, const int32_t *row_of, const float *weight,
                     int64_t T, int64_t k, const void *add, void *y, void *stream) {
    if (T < 0 || T > 0x7FFFFFFF || H < 0 || H % 8 || H > 0x7FFFFFFF || rows < 0 || rows > 0x7FFFFFFF || k < 1 ||
        k > fp8q::kMoeMaxK)
        return FP8Q_ERR_SHAPE;
    if (dtype != FP8Q_OUT_BF16 && dtype != FP8Q_OUT_F32) return FP8Q_ERR_DTYPE;
    if (T == 0 || H == 0) return FP8Q_OK;
    if ((rows > 0 && !c) || !row_of || !weight || !y) return FP8Q_ERR_NULL;
    if (!aligned16(c) || !aligned4(row_of) || !aligned4(weight) || !aligned16(add) || !aligned16(y))
        return FP8Q_ERR_ALIGN;
    if (fp8q::moe_combine_blocks(T, H, dtype == FP8Q_OUT_BF16) > kMaxGrid256) return FP8Q_ERR_SHAPE;
    int rc = check_device();
    if (rc) return rc;
    return finish(fp8q::launch_moe_combine(c, dtype == FP8Q_OUT_BF16, rows, H, row_of, weight, T, (int)k, add, y,
                                           static_cast<hipStream_t>(stream)));
}

int fp8q_moe_combine_backward(const void *grad_y, const void *c, int dtype, int64_t rows, int64_t H,
                              const int32_t *row_of, const float *weight, int64_t T, int64_t k,
                              const int32_t *row_token, const int32_t *offsets, int64_t E, void *grad_c,
                              float *grad_weight, void *stream) {
    if (T < 0 || T > 0x7FFFFFFF || H < 0 || H % 8 || H > 0x7FFFFFFF || rows < 0 || rows > 0x7FFFFFFF || k < 1 ||
        k > fp8q::kMoeMaxK || E < 1 || E > 0x7FFFFFFF)
        return FP8Q_ERR_SHAPE;
    if (dtype != FP8Q_OUT_BF16 && dtype != FP8Q_OUT_F32) return FP8Q_ERR_DTYPE;
    if (T == 0 && (rows == 0 || H == 0)) return FP8Q_OK;
    if (T > 0 && (!row_of || !weight || !grad_weight || (H > 0 && !grad_y))) return FP8Q_ERR_NULL;
    if (rows > 0 && (!row_token || !offsets || (H > 0 && (!c || !grad_c)))) return FP8Q_ERR_NULL;
    if (!aligned16(grad_y) || !aligned16(c) || !aligned16(grad_c) || !aligned4(row_of) || !aligned4(weight) ||
        !aligned4(grad_weight) || !aligned4(row_token) || !aligned4(offsets))
        return FP8Q_ERR_ALIGN;
    if (T + rows / 16 + 1 > kMaxGrid256) return FP8Q_ERR_SHAPE;  // a workgroup per token and per 16 rows
    int rc = check_device();
    if (rc) return rc;
    return finish(fp8q::launch_moe_combine_backward(grad_y, c, dtype == FP8Q_OUT_BF16, rows, H, row_of, weight, T,
                                                    (int)k, row_token, offsets, E, grad_c, grad_weight,
                                                    static_cast<hipStream_t>(stream)));
}

int fp8q_quant_int8(const uint16_t *x, int64_t ld, int64_t M, int64_t K, int8_t *q, float *s, void *stream) {
    if (M < 0 || K < 0 || K % 16 || ld < K || ld % 8) return FP8Q_ERR_SHAPE;
    if (M == 0) return FP8Q_OK;
    if (!s || (K > 0 && (!x || !q))) return FP8Q_ERR_NULL;  // K == 0: only the (zero) scales are written
    if (!aligned4(s) || (K > 0 && (!aligned16(x) || !aligned16(q)))) return FP8Q_ERR_ALIGN;
    if (M > kMaxGrid256) return FP8Q_ERR_SHAPE;  // one workgroup per row
    int rc = check_device();
    if (rc) return rc;
    return finish(fp8q::launch_quant_int8(x, ld, M, K, reinterpret_cast<uint8_t *>(q), s,
                                          static_cast<hipStream_t>(stream)));
}

int fp8q_gemm_int8(const int8_t *qa, const float *sa, const int8_t *qw, const float *sw, void *c, int out_dtype,
                   int64_t M, int64_t N, int64_t K, void *stream) {
    if (M < 0 || N < 0 || N % 8 || K < 16 || K > kMaxInt8K || K % 16) return FP8Q_ERR_SHAPE;
    if (out_dtype != FP8Q_OUT_BF16 && out_dtype != FP8Q_OUT_F32) return FP8Q_ERR_DTYPE;
    if (M == 0 || N == 0) return FP8Q_OK;
    if (!qa || !sa || !qw || !sw || !c) return FP8Q_ERR_NULL;
    if (!aligned16(qa) || !aligned4(sa) || !aligned16(qw) || !aligned4(sw) || !aligned16(c)) return FP8Q_ERR_ALIGN;
    const int64_t blocks = fp8q::gemm_int8_blocks(M, N, 0);
    if (blocks < 0 || blocks > kMaxGrid512) return FP8Q_ERR_SHAPE;
    int rc = check_device();
    if (rc) return rc;
    return finish(fp8q::launch_gemm_int8(reinterpret_cast<const uint8_t *>(qa), sa,
                                         reinterpret_cast<const uint8_t *>(qw), sw, c, out_dtype == FP8Q_OUT_BF16, M,
                                         N, K, static_cast<hipStream_t>(stream)));
}

int fp8q_grouped_gemm_int8(const int8_t *qa, const float *sa, const int8_t *qw, const float *sw, void *c,
                           int out_dtype, const int32_t *off, int64_t E, int64_t M_total, int64_t N, int64_t K,
                           void *stream) {
    if (E < 1 || E > 0x7FFFFFFF || M_total < 0 || M_total > 0x7FFFFFFF || M_total % 128 || N < 0 || N % 8 || K < 16 ||
        K > kMaxInt8K || K % 16)
        return FP8Q_ERR_SHAPE;
    if (out_dtype != FP8Q_OUT_BF16 && out_dtype != FP8Q_OUT_F32) return FP8Q_ERR_DTYPE;
    if (M_total == 0 || N == 0) return FP8Q_OK;
    if (!qa || !sa || !qw || !sw || !c || !off) return FP8Q_ERR_NULL;
    if (!aligned16(qa) || !aligned4(sa) || !aligned16(qw) || !aligned4(sw) || !aligned16(c) || !aligned4(off))
        return FP8Q_ERR_ALIGN;
    const int64_t blocks = fp8q::gemm_int8_blocks(M_total, N, E);
    if (blocks < 0 || blocks > kMaxGrid512) return FP8Q_ERR_SHAPE;
    int rc = check_device();
    if (rc) return rc;
    return finish(fp8q::launch_grouped_gemm_int8(reinterpret_cast<const uint8_t *>(qa), sa, M_total, nullptr,
                                                 reinterpret_cast<const uint8_t *>(qw), sw, c,
                                                 out_dtype == FP8Q_OUT_BF16, off, E, M_total, N, K,
                                                 static_cast<hipStream_t>(stream)));
}

int fp8q_grouped_gemm_int8_gather(const int8_t *q, const float *s, int64_t T, const int32_t *row_token,
                                  const int8_t *qw, const float *sw, void *c, int out_dtype, const int32_t *off,
                                  int64_t E, int64_t M_total, int64_t N, int64_t K, void *stream) {
    if (E < 1 || E > 0x7FFFFFFF || M_total < 0 || M_total > 0x7FFFFFFF || M_total % 128 || N < 0 || N % 8 || K < 16 ||
        K > kMaxInt8K || K % 16 || T < 0)
        return FP8Q_ERR_SHAPE;
    if (T > (int64_t)0x7FFFFFFF / K) return FP8Q_ERR_SHAPE;  // token offsets are 32-bit
    if (out_dtype != FP8Q_OUT_BF16 && out_dtype != FP8Q_OUT_F32) return FP8Q_ERR_DTYPE;
    if (M_total == 0 || N == 0) return FP8Q_OK;
    if (!row_token || !qw || !sw || !c || !off || (T > 0 && (!q || !s))) return FP8Q_ERR_NULL;
    if (!aligned4(row_token) || !aligned16(qw) || !aligned4(sw) || !aligned16(c) || !aligned4(off) ||
        (T > 0 && (!aligned16(q) || !aligned4(s))))
        return FP8Q_ERR_ALIGN;
    const int64_t blocks = fp8q::gemm_int8_blocks(M_total, N, E);
    if (blocks < 0 || blocks > kMaxGrid512) return FP8Q_ERR_SHAPE;
    int rc = check_device();
    if (rc) return rc;
    return finish(fp8q::launch_grouped_gemm_int8(reinterpret_cast<const uint8_t *>(q), s, T, row_token,
                                                 reinterpret_cast<const uint8_t *>(qw), sw, c,
                                                 out_dtype == FP8Q_OUT_BF16, off, E, M_total, N, K,
                                                 static_cast<hipStream_t>(stream)));
}

// Whether the bytes of `out`, contiguous rows, meet any of `in`'s rows: M of K 2-byte elements, ld elements apart.
static bool meets_rows(const void *out, const void *in, int64_t ld, int64_t M, int64_t K) {
    const int64_t o = (int64_t)reinterpret_cast<uintptr_t>(out), i = (int64_t)reinterpret_cast<uintptr_t>(in);
    const int64_t pitch = ld < (int64_t(1) << 60) ? 2 * ld : int64_t(1) << 61, row = 2 * K, end = o + M * row;
    if (i >= end) return false;
    // the last row that begins before the end of `out` (a row that ends behind its beginning, or none does)
    const int64_t last = (end - i - 1) / pitch < M - 1 ? (end - i - 1) / pitch : M - 1;
    return i + last * pitch + row > o;
}

// Whether a kernel that reads rows of `in` and writes the same rows of `out`, a workgroup a row, would write over rows that others
// still read: they share memory and are not one array.
static bool writes_over(const void *out, const void *in, int64_t ld, int64_t M, int64_t K) {
    if (out == in && (ld == K || M == 1)) return false;
    return meets_rows(out, in, ld, M, K);
}

int fp8q_rmsnorm_quant_act_1x128(const uint16_t *x, int64_t ldx, const uint16_t *residual, int64_t ldr, const void *w,
                                 int w_dtype, float eps, int pow2, int64_t M, int64_t K, uint16_t *h, uint16_t *y,
                                 uint8_t *q, float *s, float *rstd, void *stream) {
    if (M < 0 || M >= kMaxNormRows || K < 0 || K > 0x7FFFFFFF || K % 128 || ldx < K || ldx % 8 ||
        (residual && (ldr < K || ldr % 8)))
        return FP8Q_ERR_SHAPE;
    if (w_dtype != FP8Q_OUT_BF16 && w_dtype != FP8Q_OUT_F32) return FP8Q_ERR_DTYPE;
    if (!(eps > 0.0f && eps <= 3.402823466e38f) || (pow2 != 0 && pow2 != 1)) return FP8Q_ERR_OPTION;
    if (M == 0 || K == 0) return FP8Q_OK;
    if (!x || !w || !q != !s || (residual && !h) || (!q && !y && !rstd && !h)) return FP8Q_ERR_NULL;
    if (!residual && h) return FP8Q_ERR_OPTION;  // there is no sum to write
    if (!aligned16(x) || !aligned16(residual) || !aligned16(w) || !aligned16(h) || !aligned16(y) || !aligned16(q) ||
        !aligned4(s) || !aligned4(rstd))
        return FP8Q_ERR_ALIGN;
    for (const uint16_t *out : {h, y})
        if (out && (writes_over(out, x, ldx, M, K) || (residual && writes_over(out, residual, ldr, M, K))))
            return FP8Q_ERR_OPTION;
    if (h && y && meets_rows(y, h, K, M, K)) return FP8Q_ERR_OPTION;
    int rc = check_device();
    if (rc) return rc;
    return finish(fp8q::launch_rmsnorm_quant_act_1x128(x, ldx, residual, ldr, w, w_dtype == FP8Q_OUT_BF16, eps,
                                                       pow2 != 0, M, K, h, y, q, s, rstd,
                                                       static_cast<hipStream_t>(stream)));
}

int64_t fp8q_rmsnorm_backward_workspace_bytes(int64_t M, int64_t K) {
    if (M < 0 || M >= kMaxNormRows || K < 0 || K % 128 || K > fp8q::kMaxNormGradK) return -1;
    return fp8q::rmsnorm_backward_workspace_bytes(M, K);
}

int fp8q_rmsnorm_backward(const uint16_t *gy, int64_t ldg, const uint16_t *h, int64_t ldh, const void *w, int w_dtype,
                          const float *rstd, const uint16_t *gres, int64_t M, int64_t K, uint16_t *gx, float *gw,
                          void *workspace, int64_t workspace_bytes, void *stream) {
    const int64_t need = fp8q_rmsnorm_backward_workspace_bytes(M, K);
    if (need < 0 || ldg < K || ldg % 8 || ldh < K || ldh % 8) return FP8Q_ERR_SHAPE;
    if (w_dtype != FP8Q_OUT_BF16 && w_dtype != FP8Q_OUT_F32) return FP8Q_ERR_DTYPE;
    if (K == 0 || (M == 0 && !gw)) return FP8Q_OK;
    if (M > 0 && (!gy || !h || !w || !rstd || !gx || (gw && need > 0 && !workspace)))
        return FP8Q_ERR_NULL;
    if (!aligned16(gy) || !aligned16(h) || !aligned16(w) || !aligned4(rstd) || !aligned16(gres) || !aligned16(gx) ||
        !aligned16(gw) || !aligned16(workspace))
        return FP8Q_ERR_ALIGN;
    if (M > 0 && (gx == gy || gx == h)) return FP8Q_ERR_OPTION;  // other workgroups may still read them
    if (gw && workspace_bytes < need) return FP8Q_ERR_WORKSPACE;
    if (M > 0 && (meets_rows(gx, gy, ldg, M, K) || meets_rows(gx, h, ldh, M, K) || (gres && writes_over(gx, gres, K, M, K))))
        return FP8Q_ERR_OPTION;
    int rc = check_device();
    if (rc) return rc;
    return finish(fp8q::launch_rmsnorm_backward(gy, ldg, h, ldh, w, w_dtype == FP8Q_OUT_BF16, rstd, gres, M, K, gx, gw,
                                                static_cast<float *>(workspace), static_cast<hipStream_t>(stream)));
}

// Tiles of 128 x 128, or -1 where there are 2^23 and more.
static int64_t square_tiles(int64_t rows, int64_t K) {
    const int64_t mt = (rows + 127) / 128, kt = K / 128;
    if (mt > 0 && kt >= (kMaxGrid512 + mt) / mt) return -1;
    return mt * kt < kMaxGrid512 ? mt * kt : -1;
}

static int transpose_128x1(const void *x, const float *s, bool codes, int64_t ld, int64_t T, int64_t K,
                           const int32_t *row_token, int64_t rows, uint8_t *qt, uint8_t *et, void *stream) {
    if (T < 0 || T > 0x7FFFFFFF || rows < 0 || rows > 0x7FFFFFFF || K < 0 || K % 128 || (!row_token && rows != T && rows != 0) ||
        ld < K || ld % 8 || square_tiles(rows, K) < 0)
        return FP8Q_ERR_SHAPE;
    if (rows == 0 || K == 0) return FP8Q_OK;
    if ((T > 0 && (!x || (codes && !s))) || !qt || !et) return FP8Q_ERR_NULL;
    if (!aligned16(x) || !aligned4(s) || !aligned4(row_token) || !aligned16(qt) || !aligned16(et)) return FP8Q_ERR_ALIGN;
    int rc = check_device();
    if (rc) return rc;
    return finish(fp8q::launch_transpose_128x1(x, s, codes, ld, T, K, row_token, rows, qt, et,
                                               static_cast<hipStream_t>(stream)));
}

int fp8q_transpose_act_128x1(const uint8_t *q, const float *s, int64_t T, int64_t K, const int32_t *row_token,
                             int64_t rows, uint8_t *qt, uint8_t *et, void *stream) {
    return transpose_128x1(q, s, true, K, T, K, row_token, rows, qt, et, stream);
}

int fp8q_quant_act_128x1(const uint16_t *x, int64_t ld, int64_t T, int64_t K, const int32_t *row_token, int64_t rows,
                         uint8_t *qt, uint8_t *et, void *stream) {
    return transpose_128x1(x, nullptr, false, ld, T, K, row_token, rows, qt, et, stream);
}

int fp8q_swiglu_backward_quant(const uint8_t *q, const float *s, const uint16_t *gh, int64_t ldg, int64_t M, int64_t F,
                               uint8_t *gq, float *gs, uint8_t *gqt, uint8_t *get, uint8_t *hqt, uint8_t *het,
                               void *stream) {
    if (M < 0 || M > 0x7FFFFFFF || F < 0 || F > kMaxWgrad || F % 128 || ldg < F || ldg > kMaxK || ldg % 8 ||
        square_tiles(M, F) < 0)
        return FP8Q_ERR_SHAPE;
    if (M == 0 || F == 0) return FP8Q_OK;
    if (!q || !s || !gh || !gq || !gs || !gqt || !get || !hqt || !het) return FP8Q_ERR_NULL;
    if (!aligned16(q) || !aligned4(s) || !aligned16(gh) || !aligned16(gq) || !aligned4(gs) || !aligned16(gqt) ||
        !aligned16(get) || !aligned16(hqt) || !aligned16(het))
        return FP8Q_ERR_ALIGN;
    int rc = check_device();
    if (rc) return rc;
    return finish(fp8q::launch_swiglu_backward_quant(q, s, gh, ldg, M, F, gq, gs, gqt, get, hqt, het,
                                                     static_cast<hipStream_t>(stream)));
}

static bool wgrad_sizes(int64_t M, int64_t N, int64_t K) {
    if (M < 0 || M % 128 || M > kMaxK || N < 0 || N > kMaxWgrad || N % 16 || K < 0 || K > kMaxWgrad || K % 16) return false;
    return M / 128 * (N > K ? N : K) <= int64_t(1) << 30;  // scale bytes are addressed with 32-bit offsets
}

int64_t fp8q_gemm_wgrad_workspace_bytes(int64_t M, int64_t N, int64_t K, int out_dtype) {
    if (!wgrad_sizes(M, N, K)) return -1;
    if (out_dtype != FP8Q_OUT_BF16 && out_dtype != FP8Q_OUT_F32) return -1;
    const int64_t blocks = fp8q::gemm_wgrad_blocks(N, K, 1);
    if (blocks < 0 || blocks > kMaxGrid512) return -1;
    return fp8q::gemm_wgrad_workspace_bytes(M, N, K, out_dtype == FP8Q_OUT_BF16);
}

static int wgrad(const uint8_t *gt, const uint8_t *eg, const uint8_t *xt, const uint8_t *ex, void *dw, int out_dtype,
                 int accumulate, bool grouped, const int32_t *off, int64_t E, int64_t M, int64_t N, int64_t K,
                 void *workspace, int64_t workspace_bytes, void *stream) {
    if (E < 1 || E > 0x7FFFFFFF || !wgrad_sizes(M, N, K)) return FP8Q_ERR_SHAPE;
    const int64_t blocks = fp8q::gemm_wgrad_blocks(N, K, E);
    if (blocks < 0 || blocks > kMaxGrid512) return FP8Q_ERR_SHAPE;
    if (out_dtype != FP8Q_OUT_BF16 && out_dtype != FP8Q_OUT_F32) return FP8Q_ERR_DTYPE;
    if (accumulate != 0 && accumulate != 1) return FP8Q_ERR_OPTION;
    if (N == 0 || K == 0 || (M == 0 && accumulate)) return FP8Q_OK;
    const int64_t need = grouped ? 0 : fp8q::gemm_wgrad_workspace_bytes(M, N, K, out_dtype == FP8Q_OUT_BF16);
    if (!dw || (M > 0 && (!gt || !eg || !xt || !ex)) || (grouped && !off) || (need > 0 && !workspace))
        return FP8Q_ERR_NULL;
    if (!aligned16(gt) || !aligned16(eg) || !aligned16(xt) || !aligned16(ex) || !aligned16(dw) || !aligned4(off) ||
        !aligned16(workspace))
        return FP8Q_ERR_ALIGN;
    if (workspace_bytes < need) return FP8Q_ERR_WORKSPACE;
    int rc = check_device();
    if (rc) return rc;
    return finish(fp8q::launch_gemm_wgrad(gt, eg, xt, ex, dw, out_dtype == FP8Q_OUT_BF16, accumulate != 0, off, E, M, N,
                                          K, static_cast<float *>(workspace), static_cast<hipStream_t>(stream)));
}

int fp8q_gemm_wgrad(const uint8_t *gt, const uint8_t *eg, const uint8_t *xt, const uint8_t *ex, void *dw, int out_dtype,
                    int accumulate, int64_t M, int64_t N, int64_t K, void *workspace, int64_t workspace_bytes,
                    void *stream) {
    return wgrad(gt, eg, xt, ex, dw, out_dtype, accumulate, false, nullptr, 1, M, N, K, workspace, workspace_bytes, stream);
}

int fp8q_grouped_gemm_wgrad(const uint8_t *gt, const uint8_t *eg, const uint8_t *xt, const uint8_t *ex, void *dw,
                            int out_dtype, int accumulate, const int32_t *off, int64_t E, int64_t M_total, int64_t N,
                            int64_t K, void *stream) {
    return wgrad(gt, eg, xt, ex, dw, out_dtype, accumulate, true, off, E, M_total, N, K, nullptr, 0, stream);
}

}  // extern "C"
