// Host-side launchers of the fp8q gfx950 kernels.  Arguments are validated by the C-ABI layer
// (fp8q_api.hip) before any of these is called; each returns the launch status.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8q {

hipError_t launch_quant_act_1x128(const uint16_t *x, int64_t M, int64_t K, uint8_t *q, float *s, hipStream_t stream);
hipError_t launch_quant_w_128x128(const uint16_t *w, int64_t N, int64_t K, uint8_t *q, float *s, hipStream_t stream);
hipError_t launch_swiglu_quant_act_1x128(const uint16_t *x, const uint16_t *y, int64_t ld, int64_t M, int64_t K,
                                         uint8_t *q, float *s, hipStream_t stream);
hipError_t launch_quant_act_dual(const uint16_t *x, int64_t M, int64_t K, uint8_t *q, float *s, uint8_t *qt,
                                 float *st, hipStream_t stream);
hipError_t launch_swiglu_bf16(const uint16_t *x, const uint16_t *y, int64_t ld, int64_t M, int64_t K, uint16_t *h,
                              hipStream_t stream);
hipError_t launch_quant_act_fp4_1x128(const uint16_t *x, int64_t M, int64_t K, uint8_t *q, float *s,
                                      hipStream_t stream);
hipError_t launch_quant_w_fp4_128x128(const uint16_t *w, int64_t N, int64_t K, uint8_t *q, float *s,
                                      hipStream_t stream);
hipError_t launch_quant_act_e5m6_1x128(const uint16_t *x, int64_t M, int64_t K, uint8_t *q, float *s,
                                       hipStream_t stream);
hipError_t launch_quant_w_per_channel(const uint16_t *w, int64_t N, int64_t K, uint8_t *q, float *s,
                                      hipStream_t stream);
hipError_t launch_dequant_w_128x128(const uint8_t *q, const float *s, int64_t N, int64_t K, uint16_t *w,
                                    hipStream_t stream);
hipError_t launch_gemm_blockscaled(const uint8_t *qa, const float *sa, const uint8_t *qw, const float *sw, void *c,
                                   bool out_bf16, int64_t M, int64_t N, int64_t K, hipStream_t stream);
hipError_t launch_grouped_gemm_blockscaled(const uint8_t *qa, const float *sa, const uint8_t *qw, const float *sw,
                                           void *c, bool out_bf16, const int32_t *off, int64_t E, int64_t M_total,
                                           int64_t N, int64_t K, hipStream_t stream);
hipError_t launch_grouped_gemm_gather(const uint8_t *q, const float *s, int64_t T, const int32_t *row_token,
                                      const uint8_t *qw, const float *sw, void *c, bool out_bf16,
                                      const int32_t *off, int64_t E, int64_t M_total, int64_t N, int64_t K,
                                      hipStream_t stream);
// MoE routing: experts at most kMoeMaxExperts, k at most kMoeMaxK.
constexpr int kMoeMaxExperts = 1024;
constexpr int kMoeMaxK = 16;
int64_t moe_route_workspace_bytes(int64_t T, int64_t E);
// Bytes of the routing's fixed device workspace (one per GPU) used by the entry point that allocates nothing.
constexpr int64_t kRouteScratchBytes = int64_t(4) << 20;
// Device address of that workspace on device `dev`, which must be the current device (looked up on the first
// call per device, then cached).
hipError_t route_scratch(int dev, int32_t **ptr);
hipError_t launch_moe_route_topk(const float *logits, int64_t T, int E, int k, int32_t *topk_idx,
                                 int32_t *offsets, int32_t *row_of, int32_t *row_token, int64_t rows,
                                 int32_t *workspace, hipStream_t stream);
hipError_t launch_moe_gather_fp8(const uint8_t *q, const float *s, int64_t T, int64_t K, int k,
                                 const int32_t *row_of, const int32_t *row_token, const int32_t *offsets, int E,
                                 int64_t rows, uint8_t *qa, float *sa, hipStream_t stream);
// MoE gating (sizes as in the header; n_group at most kMoeMaxGroups).
constexpr int kMoeMaxGroups = 64;
struct GateShape {
    const void *logits;
    const float *bias;  // or null
    int64_t ld, T;
    int E, k, n_group, topk_group, group_top;
    float scale;
    bool bf16, softmax, renorm;
};
int64_t moe_gate_workspace_bytes(int64_t T, int64_t E);        // to run at its best
int64_t moe_gate_least_workspace_bytes(int64_t T, int64_t E);  // to run at all; never less for more tokens
hipError_t launch_moe_gate_topk(const GateShape &g, int32_t *topk_idx, float *topk_weight, int32_t *offsets,
                                int32_t *row_of, int32_t *row_token, int64_t rows, int32_t *load, void *workspace,
                                int64_t workspace_bytes, hipStream_t stream);
hipError_t launch_moe_gate_backward(const GateShape &g, const int32_t *topk_idx, const float *grad_weight,
                                    void *grad_logits, hipStream_t stream);
hipError_t launch_moe_combine(const void *c, bool bf16, int64_t rows, int64_t H, const int32_t *row_of,
                              const float *weight, int64_t T, int k, const void *add, void *y, hipStream_t stream);
// Number of workgroups of the combination (for grid-size validation).
int64_t moe_combine_blocks(int64_t T, int64_t H, bool bf16);
hipError_t launch_moe_combine_backward(const void *grad_y, const void *c, bool bf16, int64_t rows, int64_t H,
                                       const int32_t *row_of, const float *weight, int64_t T, int k,
                                       const int32_t *row_token, const int32_t *offsets, int64_t E, void *grad_c,
                                       float *grad_weight, hipStream_t stream);
hipError_t launch_quant_int8(const uint16_t *x, int64_t ld, int64_t M, int64_t K, uint8_t *q, float *s,
                             hipStream_t stream);
hipError_t launch_gemm_int8(const uint8_t *qa, const float *sa, const uint8_t *qw, const float *sw, void *c,
                            bool out_bf16, int64_t M, int64_t N, int64_t K, hipStream_t stream);
// row_token null: qa has one row per row of c (T is not used); else it picks each row's token of qa [T, K].
hipError_t launch_grouped_gemm_int8(const uint8_t *qa, const float *sa, int64_t T, const int32_t *row_token,
                                    const uint8_t *qw, const float *sw, void *c, bool out_bf16, const int32_t *off,
                                    int64_t E, int64_t M_total, int64_t N, int64_t K, hipStream_t stream);
// Upper bound on the workgroups of an INT8 product (E == 0: dense); -1 past 2^40.
int64_t gemm_int8_blocks(int64_t M, int64_t N, int64_t E);
// Multiprocessor count of the current device (cached).
int cu_count();
// The norm in front of an FP8 Linear and its gradients; residual, gres, h, y, q (with s), rstd and gw may be null.
hipError_t launch_rmsnorm_quant_act_1x128(const uint16_t *x, int64_t ldx, const uint16_t *residual, int64_t ldr,
                                          const void *w, bool w_bf16, float eps, bool pow2, int64_t M, int64_t K,
                                          uint16_t *h, uint16_t *y, uint8_t *q, float *s, float *rstd,
                                          hipStream_t stream);
int64_t rmsnorm_backward_workspace_bytes(int64_t M, int64_t K);
constexpr int64_t kMaxNormGradK = 20480;
hipError_t launch_rmsnorm_backward(const uint16_t *gy, int64_t ldg, const uint16_t *h, int64_t ldh, const void *w,
                                   bool w_bf16, const float *rstd, const uint16_t *gres, int64_t M, int64_t K,
                                   uint16_t *gx, float *gw, float *workspace, hipStream_t stream);
// Transposed copies in groups of 128 tokens with power-of-two scales, from an 8-bit checkpoint (codes and s) or from bf16
// rows ld elements apart; row_token null: rows == T.
hipError_t launch_transpose_128x1(const void *x, const float *s, bool codes, int64_t ld, int64_t T, int64_t K,
                                  const int32_t *row_token, int64_t rows, uint8_t *qt, uint8_t *et, hipStream_t stream);
hipError_t launch_swiglu_backward_quant(const uint8_t *q, const float *s, const uint16_t *gh, int64_t ldg, int64_t M,
                                        int64_t F, uint8_t *gq, float *gs, uint8_t *gqt, uint8_t *get, uint8_t *hqt,
                                        uint8_t *het, hipStream_t stream);
// Weight gradients from transposed copies; off null: one product over all M columns (E is 1).
int64_t gemm_wgrad_workspace_bytes(int64_t M, int64_t N, int64_t K, bool out_bf16);
// Upper bound on the workgroups of E weight gradients; -1 past 2^40.
int64_t gemm_wgrad_blocks(int64_t N, int64_t K, int64_t E);
hipError_t launch_gemm_wgrad(const uint8_t *gt, const uint8_t *eg, const uint8_t *xt, const uint8_t *ex, void *dw,
                             bool out_bf16, bool accumulate, const int32_t *off, int64_t E, int64_t M, int64_t N,
                             int64_t K, float *workspace, hipStream_t stream);
// Number of workgroups the dense GEMM launches for an M x N output (for grid-size validation).
int64_t gemm_blocks(int64_t M, int64_t N);
// Number of workgroups a grouped GEMM launches for M rows, N columns and E experts; -1 when that count
// would pass 2^40 or E is past 2^31 (for grid-size validation).
int64_t grouped_gemm_blocks(int64_t M, int64_t N, int64_t E);

}  // namespace fp8q
