// C ABI of the library: argument validation, device checks and launches.
// See include/moe_mxfp4.h for the contract of every entry point.
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/moe_mxfp4.h"
#include "launch.h"

namespace {

constexpr uint64_t kWaitLimitNs = 2000000000ull;   // 2 s per pipeline wait
constexpr int kMaxE = 1024;
constexpr size_t kStatusBytes = 256;

thread_local int32_t g_last_launches = 0;

// Per device: 0 not yet looked up, -1 not compute capability 10.3, else its
// SM count.  Host threads may race on the first lookup; each stores the same
// value, published with release and read with acquire.
std::atomic<int> g_dev_sms[64];

// Current device must be compute capability 10.3 (GB300).
moe_status current_device(int *num_sms) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MOE_ERR_CUDA;
    int sms = g_dev_sms[dev].load(std::memory_order_acquire);
    if (sms == 0) {
        int major = 0, minor = 0, count = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&count, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return MOE_ERR_CUDA;
        sms = (major == 10 && minor == 3 && count > 0) ? count : -1;
        g_dev_sms[dev].store(sms, std::memory_order_release);
    }
    if (sms < 0) return MOE_ERR_UNSUPPORTED;
    *num_sms = sms;
    return MOE_OK;
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int *status_word(void *workspace) { return static_cast<int *>(workspace); }

moe_status check_gemm_args(const uint16_t *act, int layout, int64_t rows, int32_t K, const uint8_t *codes,
                           const uint8_t *scales, const int32_t *group_sizes, int32_t E, int32_t N,
                           const void *out, moe_dtype out_dtype, const void *workspace,
                           size_t workspace_bytes) {
    if (rows < 0 || rows > INT32_MAX || K <= 0 || K % 32 != 0 || N <= 0 || E <= 0 || E > kMaxE)
        return MOE_ERR_INVALID_ARG;
    if (static_cast<int64_t>(E) * N > INT32_MAX) return MOE_ERR_INVALID_ARG;
    if (out_dtype != MOE_F32 && out_dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
    if (layout != MOE_ACT_ROW_MAJOR && layout != MOE_ACT_K8_INTERLEAVED) return MOE_ERR_INVALID_ARG;
    if (!codes || !scales || !group_sizes || !workspace || workspace_bytes < kStatusBytes)
        return MOE_ERR_INVALID_ARG;
    if (rows > 0 && (!act || !out)) return MOE_ERR_INVALID_ARG;
    if (!aligned(act, 16) || !aligned(codes, 16) || !aligned(workspace, 16))
        return MOE_ERR_INVALID_ARG;
    if (!aligned(out, out_dtype == MOE_F32 ? 4 : 2)) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

moe_status check_route_args(const int32_t *ids, int32_t T, int32_t k, int32_t E,
                            const int32_t *gs, const int32_t *off, const int32_t *ss,
                            const int32_t *s2r, const uint16_t *x, int32_t hidden,
                            const uint16_t *xs, int layout, const void *workspace,
                            size_t workspace_bytes) {
    if (T < 0 || E <= 0 || E > kMaxE || k <= 0 || k > E) return MOE_ERR_INVALID_ARG;
    if (static_cast<int64_t>(T) * k > INT32_MAX) return MOE_ERR_INVALID_ARG;
    if (!gs || !off || !workspace) return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!ids || !ss || !s2r)) return MOE_ERR_INVALID_ARG;
    if ((x == nullptr) != (xs == nullptr)) return MOE_ERR_INVALID_ARG;
    if (layout != MOE_ACT_ROW_MAJOR && layout != MOE_ACT_K8_INTERLEAVED &&
        layout != MOE_ACT_K8_TOKEN_ORDER)
        return MOE_ERR_INVALID_ARG;
    if (x && (hidden <= 0 || hidden % 8 != 0 || !aligned(x, 16) || !aligned(xs, 16)))
        return MOE_ERR_INVALID_ARG;
    if (!aligned(workspace, 16) || workspace_bytes < moe_workspace_bytes(T, k, E))
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

// Rows of 4-bit codes: the kernels count stages of up to 1,024 k, rounded up, in 32 bits.
constexpr int32_t kMaxFp4K = INT32_MAX - 1023;

bool known_dtype(int d) { return d == MOE_F32 || d == MOE_BF16; }

moe_status check_fp4_gemm_args(const uint8_t *act_codes, const uint8_t *act_scales, const float *act_scale_2,
                               int64_t rows, int32_t K, const uint8_t *codes, const uint8_t *scales,
                               const float *weight_scale_2, int format, const int32_t *group_sizes, int32_t E,
                               int64_t N, const void *workspace, size_t workspace_bytes) {
    if (format != MOE_FP4_MX && format != MOE_FP4_NV) return MOE_ERR_INVALID_ARG;
    // A tile may start its loads up to 256 rows past the last row (they read as
    // zeros): its coordinates stay 32-bit.
    constexpr int64_t kMaxRows = INT32_MAX - 512;
    if (rows < 0 || rows > kMaxRows || K <= 0 || K > kMaxFp4K || K % 32 != 0 || N <= 0 || E <= 0 || E > kMaxE)
        return MOE_ERR_INVALID_ARG;
    if (static_cast<int64_t>(E) * N > kMaxRows) return MOE_ERR_INVALID_ARG;
    if (!codes || !scales || !group_sizes || !workspace || workspace_bytes < kStatusBytes)
        return MOE_ERR_INVALID_ARG;
    if (rows > 0 && (!act_codes || !act_scales)) return MOE_ERR_INVALID_ARG;
    if (!aligned(act_codes, 16) || !aligned(codes, 16) || !aligned(workspace, 16)) return MOE_ERR_INVALID_ARG;
    if (format == MOE_FP4_NV && (!act_scale_2 || !weight_scale_2 || !aligned(act_scale_2, 4) ||
                                 !aligned(weight_scale_2, 4)))
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

moe::Fp4Gemm fp4_gemm(const uint8_t *act_codes, const uint8_t *act_scales, const float *act_scale_2, int64_t rows,
                      int32_t K, const uint8_t *codes, const uint8_t *scales, const float *weight_scale_2,
                      const int32_t *group_sizes, int32_t E, int32_t N, void *workspace) {
    moe::Fp4Gemm g = {};
    g.a_codes = act_codes;
    g.a_scales = act_scales;
    g.a_scale_2 = act_scale_2;
    g.w_codes = codes;
    g.w_scales = scales;
    g.w_scale_2 = weight_scale_2;
    g.group_sizes = group_sizes;
    g.rows = static_cast<int>(rows);
    g.K = K;
    g.E = E;
    g.N = N;
    g.status = status_word(workspace);
    g.wait_limit_ns = kWaitLimitNs;
    return g;
}

moe_status check_gate_args(const void *logits, int dtype, int64_t stride, int32_t T, int32_t E, int32_t k) {
    if (T < 0 || E <= 0 || E > kMaxE || k <= 0 || k > E || !known_dtype(dtype) || stride < 0)
        return MOE_ERR_INVALID_ARG;
    if (static_cast<int64_t>(T) * k > INT32_MAX) return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!logits || !aligned(logits, dtype == MOE_F32 ? 4 : 2))) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

moe_status check_matvec_args(const uint16_t *x, int64_t x_stride, int32_t index_div, int32_t rows, int32_t K,
                             const uint8_t *codes, const uint8_t *scales, const float *weight_scale_2, int format,
                             int32_t E, int64_t N, int64_t columns, const void *out, const void *workspace,
                             size_t workspace_bytes) {
    if (rows < 0 || K <= 0 || K % 32 != 0 || E <= 0 || E > kMaxE || N <= 0 || index_div < 1 || x_stride < 0)
        return MOE_ERR_INVALID_ARG;
    if (static_cast<int64_t>(E) * N > INT32_MAX || static_cast<int64_t>(rows) * columns > INT32_MAX)
        return MOE_ERR_INVALID_ARG;
    if (columns > MOE_MATVEC_MAX_COLUMNS) return MOE_ERR_INVALID_ARG;      // the last item's columns lie up to 510 past them
    if (format != MOE_FP4_MX && format != MOE_FP4_NV) return MOE_ERR_INVALID_ARG;
    if (!codes || !scales || !workspace || workspace_bytes < kStatusBytes || !aligned(codes, 16) || !aligned(workspace, 16))
        return MOE_ERR_INVALID_ARG;
    if (format == MOE_FP4_NV && (!weight_scale_2 || !aligned(weight_scale_2, 4))) return MOE_ERR_INVALID_ARG;
    if (rows > 0 && (!x || !out || !aligned(x, 2))) return MOE_ERR_INVALID_ARG;
    if (rows > MOE_MATVEC_MAX_ROWS || K > MOE_MATVEC_MAX_K) return MOE_ERR_CAPACITY;
    return MOE_OK;
}

moe::Matvec matvec(const uint16_t *x, int64_t x_stride, int32_t index_div, const int32_t *row_expert, int32_t rows,
                   int32_t K, const uint8_t *codes, const uint8_t *scales, const float *weight_scale_2, int format,
                   int32_t E, int32_t N, bool swiglu, void *out, int out_bf16, void *workspace, bool chained = false) {
    return {x, x_stride, index_div, row_expert, rows, K, E, N, codes, scales, weight_scale_2,
            format == MOE_FP4_NV ? moe::Matvec::kNv : moe::Matvec::kMx, swiglu, out, out_bf16, status_word(workspace),
            kWaitLimitNs, chained};
}

moe_status check_ffn_args(const uint16_t *x, int64_t x_stride, int32_t T, int32_t hidden, int32_t inter,
                          const uint16_t *w13, const uint16_t *w2, const void *workspace, size_t workspace_bytes) {
    constexpr int32_t kMost = 1 << 30;
    if (T < 0 || T >= kMost || hidden <= 0 || hidden >= kMost || hidden % 8 || inter <= 0 || inter >= kMost / 2 || inter % 8)
        return MOE_ERR_INVALID_ARG;
    if (T > 1 && (x_stride < hidden || x_stride % 8)) return MOE_ERR_INVALID_ARG;
    if (!w13 || !w2 || !aligned(w13, 16) || !aligned(w2, 16) || !workspace || workspace_bytes < kStatusBytes ||
        !aligned(workspace, 16))
        return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!x || !aligned(x, 16))) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

// Whether the sums' lengths are ones that the tensor cores' f32 is good for; behind the other checks.
moe_status check_ffn_sums(int32_t hidden, int32_t inter, int32_t tokens) {
    return hidden > MOE_FFN_MAX_SUM || inter > MOE_FFN_MAX_SUM / 2 || tokens > MOE_FFN_MAX_SUM ? MOE_ERR_CAPACITY : MOE_OK;
}

moe_status grad_call(const void *const *grads, const int64_t *sizes, const int32_t *dtypes, int32_t n, float max_norm,
                     float eps, void *const *outs, float *norm, void *workspace, size_t workspace_bytes,
                     void *stream) {
    if (n < 0 || (n > 0 && (!grads || !sizes || !dtypes)) || !norm || !aligned(norm, 4)) return MOE_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < MOE_GRAD_WORKSPACE_BYTES || !aligned(workspace, 16)) return MOE_ERR_INVALID_ARG;
    if (!(max_norm >= 0.0f) || !(eps >= 0.0f) || eps > 3.402823466e38f) return MOE_ERR_INVALID_ARG;
    for (int32_t i = 0; i < n; ++i) {
        if (sizes[i] < 0 || sizes[i] > (INT64_MAX >> 4) || !known_dtype(dtypes[i])) return MOE_ERR_INVALID_ARG;
        const uintptr_t a = dtypes[i] == MOE_F32 ? 4 : 2;
        if (sizes[i] > 0 && (!grads[i] || !aligned(grads[i], a) || (outs && (!outs[i] || !aligned(outs[i], a)))))
            return MOE_ERR_INVALID_ARG;
    }
    moe::GradList g = {grads, outs, sizes, dtypes, n, max_norm, eps, norm,
                       static_cast<uint8_t *>(workspace) + kStatusBytes};
    moe_status st = moe::check_grad_spans(g);
    if (st != MOE_OK) return st;
    int sms = 0;
    if ((st = current_device(&sms)) != MOE_OK) return st;
    if (moe::grad_partial_bytes(sms) + kStatusBytes > MOE_GRAD_WORKSPACE_BYTES) return MOE_ERR_UNSUPPORTED;
    int launches = 0;
    st = moe::launch_grad_clip(g, static_cast<cudaStream_t>(stream), sms, &launches);
    g_last_launches = launches;
    return st;
}

}  // namespace

extern "C" {

const char *moe_status_string(moe_status s) {
    switch (s) {
        case MOE_OK: return "MOE_OK";
        case MOE_ERR_INVALID_ARG: return "MOE_ERR_INVALID_ARG";
        case MOE_ERR_UNSUPPORTED: return "MOE_ERR_UNSUPPORTED";
        case MOE_ERR_CUDA: return "MOE_ERR_CUDA";
        case MOE_ERR_DATA: return "MOE_ERR_DATA";
        case MOE_ERR_TIMEOUT: return "MOE_ERR_TIMEOUT";
        case MOE_ERR_CAPACITY: return "MOE_ERR_CAPACITY";
    }
    return "MOE_ERR_UNKNOWN";
}

size_t moe_workspace_bytes(int32_t T, int32_t k, int32_t E) {
    if (T < 0 || k < 0 || E < 0) return kStatusBytes;
    return kStatusBytes + moe::route_sort_scratch_bytes(T, k, E);
}

moe_status moe_clear_status(void *workspace, void *stream) {
    if (!workspace) return MOE_ERR_INVALID_ARG;
    g_last_launches = 0;
    return cudaMemsetAsync(workspace, 0, sizeof(int), static_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

moe_status moe_read_status(const void *workspace, void *stream) {
    if (!workspace) return MOE_ERR_INVALID_ARG;
    int v = 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cudaMemcpyAsync(&v, workspace, sizeof(int), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return MOE_ERR_CUDA;
    return static_cast<moe_status>(v);
}

moe_status moe_route_sort(const int32_t *topk_ids, int32_t T, int32_t k, int32_t E,
                          int32_t *group_sizes, int32_t *group_offsets, int32_t *sorted_slot,
                          int32_t *slot_to_row, const uint16_t *x, int32_t hidden,
                          uint16_t *x_sorted, moe_act_layout x_sorted_layout, void *workspace,
                          size_t workspace_bytes, void *stream) {
    moe_status st = check_route_args(topk_ids, T, k, E, group_sizes, group_offsets, sorted_slot,
                                     slot_to_row, x, hidden, x_sorted, x_sorted_layout, workspace,
                                     workspace_bytes);
    if (st != MOE_OK) return st;
    int sms = 0;
    if ((st = current_device(&sms)) != MOE_OK) return st;
    int launches = 0;
    const bool tokens = x_sorted_layout == MOE_ACT_K8_TOKEN_ORDER;
    st = moe::launch_route_sort(topk_ids, T, k, E, group_sizes, group_offsets, sorted_slot,
                                slot_to_row, x, hidden, tokens ? nullptr : x_sorted,
                                x_sorted_layout == MOE_ACT_K8_INTERLEAVED,
                                static_cast<uint8_t *>(workspace) + kStatusBytes,
                                status_word(workspace), static_cast<cudaStream_t>(stream),
                                &launches, tokens ? x_sorted : nullptr);
    g_last_launches = launches;
    return st;
}

moe_status moe_route_sort_noalloc(const int32_t *topk_ids, int32_t T, int32_t k, int32_t E,
                                  int32_t *group_sizes, int32_t *group_offsets,
                                  int32_t *sorted_slot, int32_t *slot_to_row, const uint16_t *x,
                                  int32_t hidden, uint16_t *x_sorted,
                                  moe_act_layout x_sorted_layout, void *stream) {
    // The checks of moe_route_sort that do not concern the workspace.
    if (T < 0 || E <= 0 || E > kMaxE || k <= 0 || k > E) return MOE_ERR_INVALID_ARG;
    if (static_cast<int64_t>(T) * k > INT32_MAX) return MOE_ERR_INVALID_ARG;
    if (!group_sizes || !group_offsets) return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!topk_ids || !sorted_slot || !slot_to_row)) return MOE_ERR_INVALID_ARG;
    if ((x == nullptr) != (x_sorted == nullptr)) return MOE_ERR_INVALID_ARG;
    if (x_sorted_layout != MOE_ACT_ROW_MAJOR && x_sorted_layout != MOE_ACT_K8_INTERLEAVED)
        return MOE_ERR_INVALID_ARG;
    if (x && (hidden <= 0 || hidden % 8 != 0 || !aligned(x, 16) || !aligned(x_sorted, 16)))
        return MOE_ERR_INVALID_ARG;
    if (moe::route_sort_scratch_bytes(T, k, E) > MOE_ROUTE_SORT_NOALLOC_SCRATCH_BYTES)
        return MOE_ERR_CAPACITY;
    int sms = 0;
    moe_status st = current_device(&sms);
    if (st != MOE_OK) return st;
    int launches = 0;
    st = moe::launch_route_sort_noalloc(topk_ids, T, k, E, group_sizes, group_offsets,
                                        sorted_slot, slot_to_row, x, hidden, x_sorted,
                                        x_sorted_layout == MOE_ACT_K8_INTERLEAVED,
                                        static_cast<cudaStream_t>(stream), &launches);
    g_last_launches = launches;
    return st;
}

moe_status moe_mxfp4_grouped_gemm(const uint16_t *act, moe_act_layout act_layout, int64_t rows,
                                  int32_t K, const uint8_t *codes, const uint8_t *scales,
                                  const int32_t *group_sizes, int32_t E, int32_t N, void *out,
                                  moe_dtype out_dtype, void *workspace, size_t workspace_bytes,
                                  void *stream) {
    moe_status st = check_gemm_args(act, act_layout, rows, K, codes, scales, group_sizes, E, N,
                                    out, out_dtype, workspace, workspace_bytes);
    if (st != MOE_OK) return st;
    int sms = 0;
    if ((st = current_device(&sms)) != MOE_OK) return st;
    st = moe::launch_grouped_gemm(act, static_cast<int>(rows), K, codes, scales, group_sizes, E, N,
                                  out, out_dtype == MOE_BF16, act_layout == MOE_ACT_K8_INTERLEAVED,
                                  status_word(workspace), kWaitLimitNs,
                                  static_cast<cudaStream_t>(stream), sms);
    g_last_launches = rows > 0 ? moe::kGemmLaunches : 0;
    return st;
}

moe_status moe_mxfp4_grouped_gemm_block(const uint16_t *act, moe_act_layout act_layout,
                                        int64_t rows, int32_t K, int32_t scale_block,
                                        const uint8_t *codes, const uint8_t *scales,
                                        const int32_t *group_sizes, int32_t E, int32_t N,
                                        void *out, moe_dtype out_dtype, void *workspace,
                                        size_t workspace_bytes, void *stream) {
    if ((scale_block != 32 && scale_block != 512) || K <= 0 || K % scale_block != 0)
        return MOE_ERR_INVALID_ARG;
    moe_status st = check_gemm_args(act, act_layout, rows, K, codes, scales, group_sizes, E, N,
                                    out, out_dtype, workspace, workspace_bytes);
    if (st != MOE_OK) return st;
    int sms = 0;
    if ((st = current_device(&sms)) != MOE_OK) return st;
    st = moe::launch_grouped_gemm_block(act, static_cast<int>(rows), K, scale_block, codes, scales,
                                        group_sizes, E, N, out, out_dtype == MOE_BF16,
                                        act_layout == MOE_ACT_K8_INTERLEAVED,
                                        status_word(workspace), kWaitLimitNs,
                                        static_cast<cudaStream_t>(stream), sms);
    g_last_launches = rows > 0 ? moe::kGemmLaunches : 0;
    return st;
}

moe_status moe_mxfp4_grouped_gemm_swiglu(const uint16_t *act, moe_act_layout act_layout,
                                         int64_t rows, int32_t K, const uint8_t *codes,
                                         const uint8_t *scales, const int32_t *group_sizes,
                                         int32_t E, int32_t I, uint16_t *h,
                                         moe_act_layout h_layout, void *workspace,
                                         size_t workspace_bytes, void *stream) {
    if (I <= 0 || I % 16 != 0 || static_cast<int64_t>(I) * 2 > INT32_MAX) return MOE_ERR_INVALID_ARG;
    moe_status st = check_gemm_args(act, act_layout, rows, K, codes, scales, group_sizes, E, 2 * I,
                                    h, MOE_BF16, workspace, workspace_bytes);
    if (st != MOE_OK) return st;
    if (h_layout != MOE_ACT_ROW_MAJOR && (h_layout != MOE_ACT_K8_INTERLEAVED || I % 8 != 0))
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    if ((st = current_device(&sms)) != MOE_OK) return st;
    st = moe::launch_grouped_gemm_swiglu(act, static_cast<int>(rows), K, codes, scales, group_sizes,
                                         E, 2 * I, h, act_layout == MOE_ACT_K8_INTERLEAVED,
                                         h_layout == MOE_ACT_K8_INTERLEAVED,
                                         status_word(workspace), kWaitLimitNs,
                                         static_cast<cudaStream_t>(stream), sms);
    g_last_launches = rows > 0 ? moe::kGemmLaunches : 0;
    return st;
}

moe_status moe_mxfp4_grouped_gemm_swiglu_gather(const uint16_t *x_k8, int32_t T, int32_t top_k,
                                                const int32_t *sorted_slot, int64_t rows, int32_t K,
                                                const uint8_t *codes, const uint8_t *scales,
                                                const int32_t *group_sizes, int32_t E, int32_t I,
                                                uint16_t *h, moe_act_layout h_layout,
                                                void *workspace, size_t workspace_bytes,
                                                void *stream) {
    if (I <= 0 || I % 16 != 0 || static_cast<int64_t>(I) * 2 > INT32_MAX) return MOE_ERR_INVALID_ARG;
    if (T < 0 || top_k <= 0 || (rows > 0 && (T == 0 || !sorted_slot))) return MOE_ERR_INVALID_ARG;
    moe_status st = check_gemm_args(x_k8, MOE_ACT_K8_INTERLEAVED, rows, K, codes, scales,
                                    group_sizes, E, 2 * I, h, MOE_BF16, workspace, workspace_bytes);
    if (st != MOE_OK) return st;
    if (h_layout != MOE_ACT_ROW_MAJOR && (h_layout != MOE_ACT_K8_INTERLEAVED || I % 8 != 0))
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    if ((st = current_device(&sms)) != MOE_OK) return st;
    st = moe::launch_grouped_gemm_swiglu_gather(x_k8, T, top_k, sorted_slot, static_cast<int>(rows), K,
                                                codes, scales, group_sizes, E, 2 * I, h,
                                                h_layout == MOE_ACT_K8_INTERLEAVED,
                                                status_word(workspace), kWaitLimitNs,
                                                static_cast<cudaStream_t>(stream), sms);
    g_last_launches = rows > 0 ? moe::kGemmLaunches : 0;
    return st;
}

moe_status moe_mxfp4_grouped_gemm_scatter(const uint16_t *act, moe_act_layout act_layout,
                                          int64_t rows, int32_t K, const uint8_t *codes,
                                          const uint8_t *scales, const int32_t *group_sizes,
                                          int32_t E, int32_t N, const int32_t *out_row, void *out,
                                          moe_dtype out_dtype, void *workspace,
                                          size_t workspace_bytes, void *stream) {
    moe_status st = check_gemm_args(act, act_layout, rows, K, codes, scales, group_sizes, E, N,
                                    out, out_dtype, workspace, workspace_bytes);
    if (st != MOE_OK) return st;
    if (rows > 0 && !out_row) return MOE_ERR_INVALID_ARG;
    int sms = 0;
    if ((st = current_device(&sms)) != MOE_OK) return st;
    st = moe::launch_grouped_gemm_scatter(act, static_cast<int>(rows), K, codes, scales, group_sizes,
                                          E, N, out_row, out, out_dtype == MOE_BF16,
                                          act_layout == MOE_ACT_K8_INTERLEAVED,
                                          status_word(workspace), kWaitLimitNs,
                                          static_cast<cudaStream_t>(stream), sms);
    g_last_launches = rows > 0 ? moe::kGemmLaunches : 0;
    return st;
}

moe_status moe_nvfp4_grouped_gemm(const uint16_t *act, moe_act_layout act_layout, int64_t rows,
                                  int32_t K, const uint8_t *codes, const uint8_t *scales16,
                                  const float *weight_scale_2, const int32_t *group_sizes,
                                  int32_t E, int32_t N, void *out, moe_dtype out_dtype,
                                  void *workspace, size_t workspace_bytes, void *stream) {
    moe_status st = check_gemm_args(act, act_layout, rows, K, codes, scales16, group_sizes, E, N,
                                    out, out_dtype, workspace, workspace_bytes);
    if (st != MOE_OK) return st;
    if (!weight_scale_2 || !aligned(weight_scale_2, 4)) return MOE_ERR_INVALID_ARG;
    int sms = 0;
    if ((st = current_device(&sms)) != MOE_OK) return st;
    st = moe::launch_grouped_gemm_nvfp4(act, static_cast<int>(rows), K, codes, scales16,
                                        weight_scale_2, group_sizes, E, N, out,
                                        out_dtype == MOE_BF16,
                                        act_layout == MOE_ACT_K8_INTERLEAVED,
                                        status_word(workspace), kWaitLimitNs,
                                        static_cast<cudaStream_t>(stream), sms);
    g_last_launches = rows > 0 ? moe::kGemmLaunches : 0;
    return st;
}

moe_status moe_swiglu(const void *gu, moe_dtype in_dtype, int64_t rows, int32_t I, uint16_t *h,
                      moe_act_layout h_layout, void *stream) {
    if (rows < 0 || I <= 0 || (in_dtype != MOE_F32 && in_dtype != MOE_BF16))
        return MOE_ERR_INVALID_ARG;
    if (h_layout != MOE_ACT_ROW_MAJOR && (h_layout != MOE_ACT_K8_INTERLEAVED || I % 8 != 0))
        return MOE_ERR_INVALID_ARG;
    if (rows > 0 && (!gu || !h || !aligned(gu, 16) || !aligned(h, 16))) return MOE_ERR_INVALID_ARG;
    int sms = 0;
    moe_status st = current_device(&sms);
    if (st != MOE_OK) return st;
    st = moe::launch_swiglu(gu, in_dtype == MOE_BF16, rows, I, h,
                            h_layout == MOE_ACT_K8_INTERLEAVED, static_cast<cudaStream_t>(stream),
                            sms);
    g_last_launches = rows > 0 ? 1 : 0;
    return st;
}

moe_status moe_combine(const float *y, const int32_t *slot_to_row, const float *topk_w,
                       int32_t T, int32_t k, int32_t N, void *out, moe_dtype out_dtype,
                       void *stream) {
    if (T < 0 || k <= 0 || N <= 0 || (out_dtype != MOE_F32 && out_dtype != MOE_BF16))
        return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!y || !slot_to_row || !topk_w || !out || !aligned(y, 16) || !aligned(out, 16)))
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    moe_status st = current_device(&sms);
    if (st != MOE_OK) return st;
    st = moe::launch_combine(y, slot_to_row, topk_w, T, k, N, out, out_dtype == MOE_BF16,
                             static_cast<cudaStream_t>(stream), sms);
    g_last_launches = T > 0 ? 1 : 0;
    return st;
}

moe_status moe_combine_slots(const float *y, const int32_t *slot_to_row, const float *topk_w,
                             int32_t T, int32_t k, int32_t N, void *out, moe_dtype out_dtype,
                             void *stream) {
    if (T < 0 || k <= 0 || N <= 0 || (out_dtype != MOE_F32 && out_dtype != MOE_BF16))
        return MOE_ERR_INVALID_ARG;
    if (static_cast<int64_t>(T) * k > INT32_MAX) return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!y || !slot_to_row || !topk_w || !out || !aligned(y, 16) || !aligned(out, 16)))
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    moe_status st = current_device(&sms);
    if (st != MOE_OK) return st;
    st = moe::launch_combine(y, slot_to_row, topk_w, T, k, N, out, out_dtype == MOE_BF16,
                             static_cast<cudaStream_t>(stream), sms, 1);
    g_last_launches = T > 0 ? 1 : 0;
    return st;
}

moe_status moe_act_interleave_k8(const uint16_t *x, int64_t rows, int32_t hidden, uint16_t *x_k8,
                                 void *stream) {
    if (rows < 0 || hidden <= 0 || hidden % 8 != 0) return MOE_ERR_INVALID_ARG;
    if (rows > 0 && (!x || !x_k8 || !aligned(x, 16) || !aligned(x_k8, 16)))
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    moe_status st = current_device(&sms);
    if (st != MOE_OK) return st;
    st = moe::launch_interleave_k8(x, rows, hidden, x_k8, static_cast<cudaStream_t>(stream), sms);
    g_last_launches = rows > 0 ? 1 : 0;
    return st;
}

moe_status moe_layer_forward(const uint16_t *x, const int32_t *topk_ids, const float *topk_w,
                             int32_t T, int32_t k, int32_t E, int32_t hidden, int32_t inter,
                             const uint8_t *w13_codes, const uint8_t *w13_scales,
                             const uint8_t *w2_codes, const uint8_t *w2_scales, float *out,
                             int32_t *group_sizes, int32_t *group_offsets, int32_t *sorted_slot,
                             int32_t *slot_to_row, uint16_t *x_sorted, uint16_t *h, float *y2,
                             void *workspace, size_t workspace_bytes, void *stream) {
    if (hidden <= 0 || inter <= 0 || hidden % 32 || inter % 32) return MOE_ERR_INVALID_ARG;
    if (static_cast<int64_t>(inter) * 2 > INT32_MAX) return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!x || !out || !x_sorted || !h || !y2 || !topk_w)) return MOE_ERR_INVALID_ARG;
    const int64_t rows = static_cast<int64_t>(T) * k;
    moe_status st = check_route_args(topk_ids, T, k, E, group_sizes, group_offsets, sorted_slot,
                                     slot_to_row, x, hidden, x_sorted, MOE_ACT_K8_INTERLEAVED,
                                     workspace, workspace_bytes);
    if (st != MOE_OK) return st;
    if ((st = check_gemm_args(x_sorted, MOE_ACT_K8_INTERLEAVED, rows, hidden, w13_codes,
                              w13_scales, group_sizes, E, 2 * inter, h, MOE_BF16, workspace,
                              workspace_bytes)) != MOE_OK ||
        (st = check_gemm_args(h, MOE_ACT_K8_INTERLEAVED, rows, inter, w2_codes, w2_scales,
                              group_sizes, E, hidden, y2, MOE_F32, workspace, workspace_bytes)) !=
            MOE_OK)
        return st;
    if (T > 0 && (!aligned(h, 16) || !aligned(y2, 16) || !aligned(out, 16)))
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    if ((st = current_device(&sms)) != MOE_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int launches = 0, n = 0;
    int *status = status_word(workspace);
    st = moe::launch_route_sort(topk_ids, T, k, E, group_sizes, group_offsets, sorted_slot,
                                slot_to_row, x, hidden, x_sorted, 1,
                                static_cast<uint8_t *>(workspace) + kStatusBytes, status, s, &n);
    launches += n;
    if (st == MOE_OK && rows > 0) {   // w13 with SwiGLU in its epilogue: h, never y13
        st = moe::launch_grouped_gemm_swiglu(x_sorted, static_cast<int>(rows), hidden, w13_codes,
                                             w13_scales, group_sizes, E, 2 * inter, h, 1, 1,
                                             status, kWaitLimitNs, s, sms);
        launches += moe::kGemmLaunches;
    }
    if (st == MOE_OK && rows > 0) {
        st = moe::launch_grouped_gemm(h, static_cast<int>(rows), inter, w2_codes, w2_scales,
                                      group_sizes, E, hidden, y2, 0, 1, status, kWaitLimitNs, s,
                                      sms);
        launches += moe::kGemmLaunches;
    }
    if (st == MOE_OK && T > 0) {
        st = moe::launch_combine(y2, slot_to_row, topk_w, T, k, hidden, out, 0, s, sms);
        ++launches;
    }
    g_last_launches = launches;
    return st;
}

moe_status moe_set_gemm_pairing(int32_t mode) {
    if (mode < MOE_PAIRING_AUTO || mode > MOE_PAIRING_ON) return MOE_ERR_INVALID_ARG;
    moe::set_gemm_pairing(mode);
    moe::set_fp4_pairing(mode);
    return MOE_OK;
}

moe_status moe_mxfp4_decode_expert(const uint8_t *codes, const uint8_t *scales, int32_t E,
                                   int32_t N, int32_t K, int32_t e, uint16_t *out,
                                   void *workspace, size_t workspace_bytes, void *stream) {
    if (!codes || !scales || !out || !workspace || workspace_bytes < kStatusBytes || E <= 0 ||
        N <= 0 || K <= 0 || K % 32 || e < 0 || e >= E || !aligned(out, 4))
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    moe_status st = current_device(&sms);
    if (st != MOE_OK) return st;
    st = moe::launch_decode_expert(codes, scales, N, K, e, out, status_word(workspace),
                                   static_cast<cudaStream_t>(stream));
    g_last_launches = 1;
    return st;
}

size_t moe_nvfp4_cast_workspace_bytes(int32_t E) {
    return E <= 0 ? kStatusBytes : kStatusBytes + ((static_cast<size_t>(E) * sizeof(int) + 255) & ~size_t(255));
}

moe_status moe_mxfp4_to_nvfp4(const uint8_t *scales, int32_t E, int32_t N, int32_t K,
                              uint8_t *e4m3_scales, float *weight_scale_2, uint64_t *out_of_range,
                              void *workspace, size_t workspace_bytes, void *stream) {
    if (!scales || !e4m3_scales || !weight_scale_2 || !out_of_range || !workspace || E <= 0 ||
        E > 65535 || N <= 0 || K <= 0 || K % 32 || !aligned(workspace, 16) ||
        !aligned(weight_scale_2, 4) || !aligned(out_of_range, 8) ||
        workspace_bytes < moe_nvfp4_cast_workspace_bytes(E))
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    moe_status st = current_device(&sms);
    if (st != MOE_OK) return st;
    int launches = 0;
    st = moe::launch_mxfp4_to_nvfp4(
        scales, E, N, K, e4m3_scales, weight_scale_2,
        reinterpret_cast<unsigned long long *>(out_of_range),
        reinterpret_cast<int *>(static_cast<uint8_t *>(workspace) + kStatusBytes),
        status_word(workspace), kWaitLimitNs, static_cast<cudaStream_t>(stream), sms, &launches);
    g_last_launches = launches;
    return st;
}

moe_status moe_topk_gate(const void *logits, moe_dtype dtype, int64_t stride, int32_t T, int32_t E,
                         int32_t k, int32_t renorm, int32_t *topk_ids, float *topk_w, void *stream) {
    moe_status st = check_gate_args(logits, dtype, stride, T, E, k);
    if (st != MOE_OK) return st;
    if (T > 0 && (!topk_ids || !topk_w)) return MOE_ERR_INVALID_ARG;
    int sms = 0;
    if ((st = current_device(&sms)) != MOE_OK) return st;
    moe::Gate g = {logits, dtype == MOE_BF16, stride, T, E, k, renorm != 0, topk_ids, topk_w, nullptr, nullptr};
    st = moe::launch_topk_gate(g, false, static_cast<cudaStream_t>(stream));
    g_last_launches = T > 0 ? 1 : 0;
    return st;
}

moe_status moe_topk_gate_backward(const void *logits, moe_dtype dtype, int64_t stride, int32_t T,
                                  int32_t E, int32_t k, int32_t renorm, const int32_t *topk_ids,
                                  const float *topk_dw, void *dlogits, void *stream) {
    moe_status st = check_gate_args(logits, dtype, stride, T, E, k);
    if (st != MOE_OK) return st;
    if (T > 0 && (!topk_ids || !topk_dw || !dlogits || !aligned(dlogits, dtype == MOE_F32 ? 4 : 2)))
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    if ((st = current_device(&sms)) != MOE_OK) return st;
    moe::Gate g = {logits, dtype == MOE_BF16, stride, T, E, k, renorm != 0,
                   const_cast<int32_t *>(topk_ids), nullptr, topk_dw, dlogits};
    st = moe::launch_topk_gate(g, true, static_cast<cudaStream_t>(stream));
    g_last_launches = T > 0 ? 1 : 0;
    return st;
}

moe_status moe_fp4_quantize(const void *x, moe_dtype dtype, int64_t x_rows, int64_t x_stride, int32_t K,
                            const int32_t *row_index, int32_t index_div, int64_t rows,
                            moe_fp4_format format, const float *tensor_scale, uint8_t *codes,
                            uint8_t *scales, void *values, moe_dtype values_dtype, void *workspace,
                            size_t workspace_bytes, void *stream) {
    if (!known_dtype(dtype) || (format != MOE_FP4_MX && format != MOE_FP4_NV) || K <= 0 || K > kMaxFp4K || K % 32 != 0 ||
        x_rows < 0 || x_rows > INT32_MAX || x_stride < 0 || rows < 0 || rows > INT32_MAX || index_div < 1)
        return MOE_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < kStatusBytes || !aligned(workspace, 16)) return MOE_ERR_INVALID_ARG;
    if (values && (!known_dtype(values_dtype) || !aligned(values, 16))) return MOE_ERR_INVALID_ARG;
    if (format == MOE_FP4_NV && (!tensor_scale || !aligned(tensor_scale, 4))) return MOE_ERR_INVALID_ARG;
    if (rows > 0 && (!codes || !scales || !aligned(codes, 16))) return MOE_ERR_INVALID_ARG;
    if (rows > 0 && x_rows > 0 && (!x || !aligned(x, dtype == MOE_F32 ? 4 : 2))) return MOE_ERR_INVALID_ARG;
    if (!row_index && rows > x_rows) return MOE_ERR_INVALID_ARG;
    int sms = 0;
    moe_status st = current_device(&sms);
    if (st != MOE_OK) return st;
    moe::Fp4Quant q = {x, dtype == MOE_BF16, x_rows, x_stride, K, row_index, index_div, rows,
                       format == MOE_FP4_NV, tensor_scale, codes, scales, values,
                       values_dtype == MOE_BF16, status_word(workspace)};
    st = moe::launch_fp4_quantize(q, static_cast<cudaStream_t>(stream), sms);
    g_last_launches = rows > 0 ? 1 : 0;
    return st;
}

moe_status moe_fp4_grouped_gemm(const uint8_t *act_codes, const uint8_t *act_scales,
                                const float *act_scale_2, int64_t rows, int32_t K, const uint8_t *codes,
                                const uint8_t *scales, const float *weight_scale_2,
                                moe_fp4_format format, const int32_t *group_sizes, int32_t E, int32_t N,
                                void *out, moe_dtype out_dtype, void *workspace, size_t workspace_bytes,
                                void *stream) {
    moe_status st = check_fp4_gemm_args(act_codes, act_scales, act_scale_2, rows, K, codes, scales,
                                        weight_scale_2, format, group_sizes, E, N, workspace, workspace_bytes);
    if (st != MOE_OK) return st;
    if (!known_dtype(out_dtype) || (rows > 0 && !out) || !aligned(out, out_dtype == MOE_F32 ? 4 : 2))
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    if ((st = current_device(&sms)) != MOE_OK) return st;
    moe::Fp4Gemm g = fp4_gemm(act_codes, act_scales, act_scale_2, rows, K, codes, scales, weight_scale_2,
                              group_sizes, E, N, workspace);
    g.out = out;
    g.out_bf16 = out_dtype == MOE_BF16;
    int launches = 0;
    st = moe::launch_fp4_gemm(g, format == MOE_FP4_NV, false, static_cast<cudaStream_t>(stream), sms, &launches);
    g_last_launches = launches;
    return st;
}

moe_status moe_fp4_grouped_gemm_swiglu(const uint8_t *act_codes, const uint8_t *act_scales,
                                       const float *act_scale_2, int64_t rows, int32_t K,
                                       const uint8_t *codes, const uint8_t *scales,
                                       const float *weight_scale_2, moe_fp4_format format,
                                       const int32_t *group_sizes, int32_t E, int32_t I,
                                       const float *h_scale_2, uint8_t *h_codes, uint8_t *h_scales,
                                       void *workspace, size_t workspace_bytes, void *stream) {
    if (I <= 0 || I % 32 != 0) return MOE_ERR_INVALID_ARG;
    moe_status st = check_fp4_gemm_args(act_codes, act_scales, act_scale_2, rows, K, codes, scales,
                                        weight_scale_2, format, group_sizes, E, 2 * static_cast<int64_t>(I),
                                        workspace, workspace_bytes);
    if (st != MOE_OK) return st;
    if (rows > 0 && (!h_codes || !h_scales || !aligned(h_codes, 16))) return MOE_ERR_INVALID_ARG;
    if (format == MOE_FP4_NV && (!h_scale_2 || !aligned(h_scale_2, 4))) return MOE_ERR_INVALID_ARG;
    int sms = 0;
    if ((st = current_device(&sms)) != MOE_OK) return st;
    moe::Fp4Gemm g = fp4_gemm(act_codes, act_scales, act_scale_2, rows, K, codes, scales, weight_scale_2,
                              group_sizes, E, 2 * I, workspace);
    g.out = h_codes;
    g.out_scales = h_scales;
    g.h_scale_2 = h_scale_2;
    int launches = 0;
    st = moe::launch_fp4_gemm(g, format == MOE_FP4_NV, true, static_cast<cudaStream_t>(stream), sms, &launches);
    g_last_launches = launches;
    return st;
}

moe_status moe_layer_forward_fp4(
    const uint16_t *x, const int32_t *topk_ids, const float *topk_w, int32_t T, int32_t k, int32_t E,
    int32_t hidden, int32_t inter, moe_fp4_format format, const uint8_t *w13_codes,
    const uint8_t *w13_scales, const float *w13_scale_2, const uint8_t *w2_codes, const uint8_t *w2_scales,
    const float *w2_scale_2, const float *x_scale_2, const float *h_scale_2, float *out,
    int32_t *group_sizes, int32_t *group_offsets, int32_t *sorted_slot, int32_t *slot_to_row,
    uint8_t *x_codes, uint8_t *x_scales, uint8_t *h_codes, uint8_t *h_scales, float *y2, void *workspace,
    size_t workspace_bytes, void *stream) {
    // Every check of every stage first: a call that fails enqueues nothing.
    if (hidden <= 0 || hidden % 32 || inter <= 0 || inter % 32) return MOE_ERR_INVALID_ARG;
    moe_status st = check_route_args(topk_ids, T, k, E, group_sizes, group_offsets, sorted_slot, slot_to_row,
                                     nullptr, 0, nullptr, MOE_ACT_ROW_MAJOR, workspace, workspace_bytes);
    if (st != MOE_OK) return st;
    const int64_t rows = static_cast<int64_t>(T) * k;
    if ((st = check_fp4_gemm_args(x_codes, x_scales, x_scale_2, rows, hidden, w13_codes, w13_scales, w13_scale_2,
                                  format, group_sizes, E, 2 * static_cast<int64_t>(inter), workspace,
                                  workspace_bytes)) != MOE_OK ||
        (st = check_fp4_gemm_args(h_codes, h_scales, h_scale_2, rows, inter, w2_codes, w2_scales, w2_scale_2,
                                  format, group_sizes, E, hidden, workspace, workspace_bytes)) != MOE_OK)
        return st;
    if (T > 0 && (!x || !topk_w || !y2 || !out || !aligned(x, 2) || !aligned(y2, 16) || !aligned(out, 16)))
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    if ((st = current_device(&sms)) != MOE_OK) return st;
    const bool nv = format == MOE_FP4_NV;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int launches = 0;
    st = moe::launch_route_sort(topk_ids, T, k, E, group_sizes, group_offsets, sorted_slot, slot_to_row, nullptr, 0,
                                nullptr, 0, static_cast<uint8_t *>(workspace) + kStatusBytes,
                                status_word(workspace), s, &launches);
    if (st == MOE_OK && rows > 0) {
        moe::Fp4Quant q = {x, 1, T, hidden, hidden, nullptr, 1, T, nv, x_scale_2, x_codes, x_scales,
                           nullptr, 0, status_word(workspace), slot_to_row, k, rows};
        moe::Fp4Gemm g13 = fp4_gemm(x_codes, x_scales, x_scale_2, rows, hidden, w13_codes, w13_scales, w13_scale_2,
                                    group_sizes, E, 2 * inter, workspace);
        g13.out = h_codes;
        g13.out_scales = h_scales;
        g13.h_scale_2 = h_scale_2;
        moe::Fp4Gemm g2 = fp4_gemm(h_codes, h_scales, h_scale_2, rows, inter, w2_codes, w2_scales, w2_scale_2,
                                   group_sizes, E, hidden, workspace);
        g2.out = y2;
        if ((st = moe::launch_fp4_quantize(q, s, sms)) == MOE_OK) ++launches;
        int n = 0;
        if (st == MOE_OK) {
            st = moe::launch_fp4_gemm(g13, nv, true, s, sms, &n);
            launches += n;
        }
        if (st == MOE_OK) {
            st = moe::launch_fp4_gemm(g2, nv, false, s, sms, &n);
            launches += n;
        }
        if (st == MOE_OK && (st = moe::launch_combine(y2, slot_to_row, topk_w, T, k, hidden, out, 0, s, sms)) == MOE_OK)
            ++launches;
    }
    g_last_launches = launches;
    return st;
}

moe_status moe_combine_backward(const void *dout, moe_dtype dout_dtype, const void *y, moe_dtype y_dtype,
                                const int32_t *slot_to_row, const float *topk_w, int32_t T, int32_t k,
                                int32_t N, void *dy, moe_dtype dy_dtype, float *topk_dw, void *stream) {
    if (T < 0 || k <= 0 || N <= 0 || static_cast<int64_t>(T) * k > INT32_MAX) return MOE_ERR_INVALID_ARG;
    if (!known_dtype(dout_dtype) || !known_dtype(y_dtype) || !known_dtype(dy_dtype)) return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!dout || !slot_to_row || !topk_w || (topk_dw && !y) || (!dy && !topk_dw))) return MOE_ERR_INVALID_ARG;
    if (!aligned(dout, 16) || !aligned(y, 16) || !aligned(dy, 16)) return MOE_ERR_INVALID_ARG;
    int sms = 0;
    moe_status st = current_device(&sms);
    if (st != MOE_OK) return st;
    moe::CombineGrad c = {dout, y, dout_dtype == MOE_BF16, y_dtype == MOE_BF16, dy_dtype == MOE_BF16,
                          slot_to_row, topk_w, T, k, N, dy, topk_dw};
    st = moe::launch_combine_backward(c, static_cast<cudaStream_t>(stream), sms);
    g_last_launches = T > 0 ? 1 : 0;
    return st;
}

moe_status moe_gather_backward(const void *dx_sorted, moe_dtype in_dtype, const int32_t *slot_to_row,
                               int32_t T, int32_t k, int32_t hidden, void *dx, moe_dtype out_dtype,
                               void *stream) {
    if (T < 0 || k <= 0 || hidden <= 0 || static_cast<int64_t>(T) * k > INT32_MAX || !known_dtype(in_dtype) ||
        !known_dtype(out_dtype))
        return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!dx_sorted || !slot_to_row || !dx || !aligned(dx_sorted, 16) || !aligned(dx, 16)))
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    moe_status st = current_device(&sms);
    if (st != MOE_OK) return st;
    st = moe::launch_gather_backward(dx_sorted, in_dtype == MOE_BF16, slot_to_row, T, k, hidden, dx,
                                     out_dtype == MOE_BF16, static_cast<cudaStream_t>(stream), sms);
    g_last_launches = T > 0 ? 1 : 0;
    return st;
}

moe_status moe_fp4_matvec(const uint16_t *x, int64_t x_stride, int32_t index_div, const int32_t *row_expert,
                          int32_t rows, int32_t K, const uint8_t *codes, const uint8_t *scales,
                          const float *weight_scale_2, moe_fp4_format format, int32_t E, int32_t N, void *out,
                          moe_dtype out_dtype, void *workspace, size_t workspace_bytes, void *stream) {
    if (!known_dtype(out_dtype) || !aligned(out, out_dtype == MOE_F32 ? 4 : 2) || !aligned(row_expert, 4))
        return MOE_ERR_INVALID_ARG;
    moe_status st = check_matvec_args(x, x_stride, index_div, rows, K, codes, scales, weight_scale_2, format, E, N, N,
                                      out, workspace, workspace_bytes);
    if (st != MOE_OK) return st;
    int sms = 0;
    if ((st = current_device(&sms)) != MOE_OK) return st;
    st = moe::launch_matvec(matvec(x, x_stride, index_div, row_expert, rows, K, codes, scales, weight_scale_2, format, E,
                                   N, false, out, out_dtype == MOE_BF16, workspace),
                            static_cast<cudaStream_t>(stream), sms);
    g_last_launches = rows > 0 ? 1 : 0;
    return st;
}

moe_status moe_fp4_matvec_swiglu(const uint16_t *x, int64_t x_stride, int32_t index_div, const int32_t *row_expert,
                                 int32_t rows, int32_t K, const uint8_t *codes, const uint8_t *scales,
                                 const float *weight_scale_2, moe_fp4_format format, int32_t E, int32_t I,
                                 uint16_t *h, void *workspace, size_t workspace_bytes, void *stream) {
    if (!aligned(h, 2) || !aligned(row_expert, 4)) return MOE_ERR_INVALID_ARG;
    moe_status st = check_matvec_args(x, x_stride, index_div, rows, K, codes, scales, weight_scale_2, format, E,
                                      2 * static_cast<int64_t>(I), I, h, workspace, workspace_bytes);
    if (st != MOE_OK) return st;
    int sms = 0;
    if ((st = current_device(&sms)) != MOE_OK) return st;
    st = moe::launch_matvec(matvec(x, x_stride, index_div, row_expert, rows, K, codes, scales, weight_scale_2, format, E,
                                   I, true, h, 1, workspace),
                            static_cast<cudaStream_t>(stream), sms);
    g_last_launches = rows > 0 ? 1 : 0;
    return st;
}

moe_status moe_layer_decode(const uint16_t *x, const int32_t *topk_ids, const float *topk_w, int32_t T, int32_t k,
                            int32_t E, int32_t hidden, int32_t inter, moe_fp4_format format, const uint8_t *w13_codes,
                            const uint8_t *w13_scales, const float *w13_scale_2, const uint8_t *w2_codes,
                            const uint8_t *w2_scales, const float *w2_scale_2, uint16_t *h, float *y2, void *out,
                            moe_dtype out_dtype, void *workspace, size_t workspace_bytes, void *stream) {
    if (T < 0 || k <= 0 || !known_dtype(out_dtype) || !aligned(out, out_dtype == MOE_F32 ? 4 : 2) || !aligned(h, 2) ||
        !aligned(y2, 4) || !aligned(topk_ids, 4) || !aligned(topk_w, 4))
        return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!topk_ids || !topk_w || !out)) return MOE_ERR_INVALID_ARG;
    const int64_t slots = static_cast<int64_t>(T) * k;
    const int32_t rows = static_cast<int32_t>(slots < INT32_MAX ? slots : INT32_MAX);
    moe_status st = check_matvec_args(x, hidden, k, rows, hidden, w13_codes, w13_scales, w13_scale_2, format, E,
                                      2 * static_cast<int64_t>(inter), inter, h, workspace, workspace_bytes);
    if (st == MOE_OK || st == MOE_ERR_CAPACITY) {
        const moe_status s2 = check_matvec_args(h, inter, 1, rows, inter, w2_codes, w2_scales, w2_scale_2, format, E,
                                                hidden, hidden, y2, workspace, workspace_bytes);
        if (s2 != MOE_OK && (st == MOE_OK || s2 == MOE_ERR_INVALID_ARG)) st = s2;
    }
    if (st != MOE_OK) return st;
    int sms = 0;
    if ((st = current_device(&sms)) != MOE_OK) return st;
    g_last_launches = 0;
    if (rows == 0) return MOE_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    st = moe::launch_matvec(matvec(x, hidden, k, topk_ids, rows, hidden, w13_codes, w13_scales, w13_scale_2, format, E,
                                   inter, true, h, 1, workspace),
                            s, sms);
    if (st == MOE_OK)
        st = moe::launch_matvec(matvec(h, inter, 1, topk_ids, rows, inter, w2_codes, w2_scales, w2_scale_2, format, E,
                                       hidden, false, y2, 0, workspace, true),
                                s, sms);
    if (st == MOE_OK) st = moe::launch_weigh(y2, topk_ids, topk_w, T, k, hidden, E, out, out_dtype == MOE_BF16, s);
    g_last_launches = 3;
    return st;
}

moe_status moe_ffn_forward(const uint16_t *x, int64_t x_stride, int32_t T, int32_t hidden, int32_t inter,
                           const uint16_t *w13, const uint16_t *w2, uint16_t *gu, uint16_t *h, void *out,
                           moe_dtype out_dtype, void *workspace, size_t workspace_bytes, void *stream) {
    moe_status st = check_ffn_args(x, x_stride, T, hidden, inter, w13, w2, workspace, workspace_bytes);
    if (st != MOE_OK) return st;
    if (!known_dtype(out_dtype) || (T > 0 && (!h || !out)) || !aligned(gu, 16) || !aligned(h, 16) || !aligned(out, 16))
        return MOE_ERR_INVALID_ARG;
    if ((st = check_ffn_sums(hidden, inter, 0)) != MOE_OK) return st;
    int sms = 0;
    if ((st = current_device(&sms)) != MOE_OK) return st;
    const moe::Ffn f = {x, T > 1 ? x_stride : hidden, T, hidden, inter, w13, w2, gu, h, out, out_dtype == MOE_BF16,
                        status_word(workspace), kWaitLimitNs};
    int launches = 0;
    st = moe::launch_ffn_forward(f, static_cast<cudaStream_t>(stream), sms, &launches);
    g_last_launches = launches;
    return st;
}

moe_status moe_ffn_backward(const uint16_t *dout, const uint16_t *x, int64_t x_stride, int32_t T, int32_t hidden,
                            int32_t inter, const uint16_t *w13, const uint16_t *w2, const uint16_t *h,
                            const uint16_t *gu, uint16_t *dgu, uint16_t *dx, void *dw13, void *dw2,
                            moe_dtype dw_dtype, void *workspace, size_t workspace_bytes, void *stream) {
    moe_status st = check_ffn_args(x, x_stride, T, hidden, inter, w13, w2, workspace, workspace_bytes);
    if (st != MOE_OK) return st;
    if (!known_dtype(dw_dtype)) return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!dout || (dw2 && !h) || ((dx || dw13) && (!gu || !dgu)))) return MOE_ERR_INVALID_ARG;
    if (!aligned(dout, 16) || !aligned(h, 16) || !aligned(gu, 16) || !aligned(dgu, 16) || !aligned(dx, 16) ||
        !aligned(dw13, 16) || !aligned(dw2, 16))
        return MOE_ERR_INVALID_ARG;
    if ((st = check_ffn_sums(hidden, inter, dw13 || dw2 ? T : 0)) != MOE_OK) return st;
    int sms = 0;
    if ((st = current_device(&sms)) != MOE_OK) return st;
    const moe::Ffn f = {x, T > 1 ? x_stride : hidden, T, hidden, inter, w13, w2, const_cast<uint16_t *>(gu),
                        const_cast<uint16_t *>(h), nullptr, 0, status_word(workspace), kWaitLimitNs};
    const moe::FfnGrad d = {dout, dgu, dx, dw13, dw2, dw_dtype == MOE_F32};
    int launches = 0;
    st = moe::launch_ffn_backward(f, d, static_cast<cudaStream_t>(stream), sms, &launches);
    g_last_launches = launches;
    return st;
}

moe_status moe_grad_norm(const void *const *grads, const int64_t *sizes, const int32_t *dtypes, int32_t n, float *norm,
                         void *workspace, size_t workspace_bytes, void *stream) {
    return grad_call(grads, sizes, dtypes, n, 0.0f, 0.0f, nullptr, norm, workspace, workspace_bytes, stream);
}

moe_status moe_grad_clip(const void *const *grads, const int64_t *sizes, const int32_t *dtypes, int32_t n,
                         float max_norm, float eps, void *const *outs, float *norm, void *workspace,
                         size_t workspace_bytes, void *stream) {
    void *const *in_place = const_cast<void *const *>(grads);
    return grad_call(grads, sizes, dtypes, n, max_norm, eps, outs ? outs : in_place, norm, workspace, workspace_bytes,
                     stream);
}

moe_status moe_debug_bounded_wait(uint64_t limit_ns, void *workspace, size_t workspace_bytes,
                                  void *stream) {
    if (!workspace || workspace_bytes < kStatusBytes || limit_ns < 1000 ||
        limit_ns > 5000000000ull)
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    moe_status st = current_device(&sms);
    if (st != MOE_OK) return st;
    st = moe::launch_bounded_wait(limit_ns, status_word(workspace),
                                  static_cast<cudaStream_t>(stream));
    g_last_launches = 1;
    return st;
}

int32_t moe_last_launch_count(void) { return g_last_launches; }

}  // extern "C"
