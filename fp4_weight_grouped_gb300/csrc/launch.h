// Internal launchers behind the C ABI (host side).  Arguments are already
// validated by api.cu; each launcher only enqueues kernels on `stream`.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/moe_mxfp4.h"

namespace moe {

// Kernel launches per grouped GEMM call: one per band class (bands of up to 32
// rows, and longer bands).
constexpr int kGemmLaunches = 2;

size_t route_sort_scratch_bytes(int T, int k, int E);

moe_status launch_route_sort(const int32_t *ids, int T, int k, int E, int32_t *group_sizes,
                             int32_t *offsets, int32_t *sorted_slot, int32_t *slot_to_row,
                             const uint16_t *x, int hidden, uint16_t *x_sorted, int x_k8,
                             void *scratch, int *status, cudaStream_t stream, int *launches,
                             uint16_t *x_tok = nullptr);

moe_status launch_route_sort_noalloc(const int32_t *ids, int T, int k, int E,
                                     int32_t *group_sizes, int32_t *offsets,
                                     int32_t *sorted_slot, int32_t *slot_to_row,
                                     const uint16_t *x, int hidden, uint16_t *x_sorted, int x_k8,
                                     cudaStream_t stream, int *launches);

moe_status launch_grouped_gemm(const uint16_t *act, int rows, int K, const uint8_t *codes,
                               const uint8_t *scales, const int32_t *group_sizes, int E, int N,
                               void *out, int out_bf16, int act_k8, int *status,
                               uint64_t wait_limit_ns, cudaStream_t stream, int num_sms);

// MXFP4 with one E8M0 scale per scale_block (32 or 512) consecutive k.
moe_status launch_grouped_gemm_block(const uint16_t *act, int rows, int K, int scale_block,
                                     const uint8_t *codes, const uint8_t *scales,
                                     const int32_t *group_sizes, int E, int N, void *out,
                                     int out_bf16, int act_k8, int *status, uint64_t wait_limit_ns,
                                     cudaStream_t stream, int num_sms);

// Fused w13 + SwiGLU: N = 2 * I weight rows ([gate | up]) -> h bf16 [rows, I].
moe_status launch_grouped_gemm_swiglu(const uint16_t *act, int rows, int K, const uint8_t *codes,
                                      const uint8_t *scales, const int32_t *group_sizes, int E,
                                      int N, uint16_t *h, int act_k8, int h_k8, int *status,
                                      uint64_t wait_limit_ns, cudaStream_t stream, int num_sms);

// Fused w13 + SwiGLU with the routing permutation in the activation load:
// sorted row r reads row sorted_slot[r] / top_k of x_k8 [act_rows, K]
// (K8-interleaved token activations).
moe_status launch_grouped_gemm_swiglu_gather(const uint16_t *x_k8, int act_rows, int top_k,
                                             const int32_t *sorted_slot, int rows, int K,
                                             const uint8_t *codes, const uint8_t *scales,
                                             const int32_t *group_sizes, int E, int N, uint16_t *h,
                                             int h_k8, int *status, uint64_t wait_limit_ns,
                                             cudaStream_t stream, int num_sms);

// Grouped GEMM writing sorted row r to output row out_row[r].
moe_status launch_grouped_gemm_scatter(const uint16_t *act, int rows, int K, const uint8_t *codes,
                                       const uint8_t *scales, const int32_t *group_sizes, int E,
                                       int N, const int32_t *out_row, void *out, int out_bf16,
                                       int act_k8, int *status, uint64_t wait_limit_ns,
                                       cudaStream_t stream, int num_sms);

moe_status launch_grouped_gemm_nvfp4(const uint16_t *act, int rows, int K, const uint8_t *codes,
                                     const uint8_t *scales16, const float *weight_scale_2,
                                     const int32_t *group_sizes, int E, int N, void *out,
                                     int out_bf16, int act_k8, int *status,
                                     uint64_t wait_limit_ns, cudaStream_t stream, int num_sms);

// CTA-pair use for bands over 32 rows: 0 automatic, 1 never, 2 whenever the
// shape allows (process-wide).
void set_gemm_pairing(int mode);
void set_fp4_pairing(int mode);   // the W4A4 products' copy of it

moe_status launch_decode_expert(const uint8_t *codes, const uint8_t *scales, int N, int K, int e,
                                uint16_t *out, int *status, cudaStream_t stream);

moe_status launch_mxfp4_to_nvfp4(const uint8_t *scales, int E, int N, int K, uint8_t *e4m3,
                                 float *weight_scale_2, unsigned long long *out_of_range,
                                 int *kmax_scratch, int *status, uint64_t wait_limit_ns,
                                 cudaStream_t stream, int num_sms, int *launches);

moe_status launch_bounded_wait(uint64_t limit_ns, int *status, cudaStream_t stream);

moe_status launch_swiglu(const void *gu, int in_bf16, long long rows, int I, uint16_t *h,
                         int h_k8, cudaStream_t stream, int num_sms);

// x_k8 [rows, hidden] = x with every 8 bf16 in the K8-interleaved order.
moe_status launch_interleave_k8(const uint16_t *x, long long rows, int hidden, uint16_t *x_k8,
                                cudaStream_t stream, int num_sms);

// slot_order: y row of slot s is s (s2r only marks the slots that count).
moe_status launch_combine(const float *y, const int32_t *s2r, const float *w, int T, int k, int N,
                          void *out, int out_bf16, cudaStream_t stream, int num_sms,
                          int slot_order = 0);

// Grouped product of 4-bit activations and 4-bit weights.  swiglu: N = 2 * I weight
// rows ([gate | up]), `out` = h codes [rows, I / 2] with `out_scales`.
struct Fp4Gemm {
    const uint8_t *a_codes, *a_scales, *w_codes, *w_scales;
    const float *a_scale_2, *w_scale_2, *h_scale_2;   // NVFP4 only
    const int32_t *group_sizes;
    int rows, K, E, N;
    void *out;
    uint8_t *out_scales;
    int out_bf16;
    int *status;
    uint64_t wait_limit_ns;
};
moe_status launch_fp4_gemm(const Fp4Gemm &g, bool nv, bool swiglu, cudaStream_t stream, int num_sms, int *launches);

// Rows of x (row r, or row row_index[r] / index_div) to 4-bit codes and block
// scales; `values` (optional) receives what they stand for.
struct Fp4Quant {
    const void *x;
    int in_bf16;
    int64_t x_rows, x_stride;
    int K;
    const int32_t *row_index;
    int index_div;
    int64_t rows;
    bool nv;
    const float *tensor_scale;
    uint8_t *codes, *scales;
    void *values;
    int values_bf16;
    int *status;
    // Instead of row_index: row r (a token) goes to rows slot_to_row[r k + j] < out_rows, j < k.
    const int32_t *slot_to_row;
    int k;
    int64_t out_rows;
};
moe_status launch_fp4_quantize(const Fp4Quant &q, cudaStream_t stream, int num_sms);

// Gradient of the combine: dy and dw (either may be null).
struct CombineGrad {
    const void *dout, *y;
    int dout_bf16, y_bf16, dy_bf16;
    const int32_t *s2r;
    const float *w;
    int T, k, N;
    void *dy;
    float *dw;
};
moe_status launch_combine_backward(const CombineGrad &c, cudaStream_t stream, int num_sms);

moe_status launch_gather_backward(const void *dxs, int in_bf16, const int32_t *s2r, int T, int k, int N, void *dx,
                                  int out_bf16, cudaStream_t stream, int num_sms);

// Router gate (ids, weights written) and its gradient (ids, dw read, dlogits written).
struct Gate {
    const void *logits;
    int bf16;
    int64_t stride;
    int T, E, k, renorm;
    int32_t *ids;
    float *weights;
    const float *dw;
    void *dlogits;
};
moe_status launch_topk_gate(const Gate &g, bool backward, cudaStream_t stream);

// Products of a few rows with weights that each row chooses: 4-bit or bf16, plain or SwiGLU
// (N = I columns of h, weights of 2 I rows an expert).
struct Matvec {
    enum Format { kMx, kNv, kBf16 };
    const uint16_t *x;
    int64_t x_stride;
    int index_div;
    const int32_t *row_expert;
    int rows, K, E, N;
    const void *weights;
    const uint8_t *scales;
    const float *weight_scale_2;
    Format format;
    bool swiglu;
    void *out;
    int out_bf16;
    int *status;
    uint64_t wait_limit_ns;
    bool chained;                 // x comes from the launch before: may start under its end
};
moe_status launch_matvec(const Matvec &m, cudaStream_t stream, int num_sms);

// out[t] = sum_j w[t, j] y[t k + j] over the slots whose id is in [0, E).
moe_status launch_weigh(const float *y, const int32_t *ids, const float *w, int T, int k, int N, int E, void *out,
                        int out_bf16, cudaStream_t stream);

// Global norm of n tensors and, with `out`, clipping by it.
struct GradList {
    const void *const *in;
    void *const *out;             // null: the norm alone
    const int64_t *sizes;
    const int32_t *dtypes;
    int n;
    double max_norm, eps;
    float *norm;
    void *partial;                // grad_partial_bytes
};
size_t grad_partial_bytes(int num_sms);
moe_status check_grad_spans(const GradList &g);
moe_status launch_grad_clip(const GradList &g, cudaStream_t stream, int num_sms, int *launches);

// Dense gated feed-forward block: forward (h, gu if given, out written) and what the backward reads of it.
struct Ffn {
    const uint16_t *x;
    int64_t x_stride;
    int T, hidden, inter;
    const uint16_t *w13, *w2;
    uint16_t *gu, *h;
    void *out;
    int out_bf16;
    int *status;
    uint64_t wait_limit_ns;
};
// Gradients; dx, dw13 and dw2 may each be null.
struct FfnGrad {
    const uint16_t *dout;
    uint16_t *dgu, *dx;
    void *dw13, *dw2;
    int dw_f32;
};
moe_status launch_ffn_forward(const Ffn &f, cudaStream_t stream, int num_sms, int *launches);
moe_status launch_ffn_backward(const Ffn &f, const FfnGrad &d, cudaStream_t stream, int num_sms, int *launches);

}  // namespace moe
