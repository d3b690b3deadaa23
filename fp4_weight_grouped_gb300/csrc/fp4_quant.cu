// Quantisation of activation rows to MXFP4 or NVFP4 (the rules are in
// fp4_common.cuh), with the routing permutation in the load.
//
// A lane owns 16 consecutive elements: an NV block, or half an MX block, whose other
// half one shuffle reaches.  A warp takes 512 elements of one row at a time, so its
// loads, code words and values are contiguous.  Magnitudes are compared as integers,
// for bf16 two in a word.  Bound: HBM.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fp4_common.cuh"
#include "launch.h"
#include "vec_io.cuh"

namespace moe {
namespace quant {

constexpr int kThreads = 256;

// Sixteen elements at p as f32, and the largest magnitude's f32 bits.
__device__ __forceinline__ uint32_t load16(const float *p, int vec, float (&v)[16]) {
    if (vec) {
        float a[8], b[8];
        load_row<8>(p, a);
        load_row<8>(p + 8, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) { v[e] = a[e]; v[8 + e] = b[e]; }
    } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = __ldg(p + e);
    }
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 16; ++e) m = max(m, __float_as_uint(v[e]) & 0x7FFFFFFFu);
    return m;
}

__device__ __forceinline__ uint32_t load16(const __nv_bfloat16 *p, int vec, float (&v)[16]) {
    uint32_t w[8];
    if (vec) {
        const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p)), b = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    } else {
        const uint16_t *u = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __ldg(u + 2 * i) | static_cast<uint32_t>(__ldg(u + 2 * i + 1)) << 16;
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
        v[2 * i] = bf16_low(w[i]);
        v[2 * i + 1] = bf16_high(w[i]);
    }
    return max(m & 0xFFFF0000u, m << 16);
}

// Sixteen values, to be evicted first: they are not read again here, and x's rows,
// which are (once for each choice of a token), stay in L2.
__device__ __forceinline__ void store_stream(void *p, const uint32_t (&w)[8]) {
    __stcs(static_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2], w[3]));
    __stcs(static_cast<uint4 *>(p) + 1, make_uint4(w[4], w[5], w[6], w[7]));
}

__device__ __forceinline__ void store16(float *p, const float (&v)[16]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(v[8 * h + e]);
        store_stream(p + 8 * h, w);
    }
}

__device__ __forceinline__ void store16(__nv_bfloat16 *p, const float (&v)[16]) {
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = bf16_pair(v[2 * e], v[2 * e + 1]);
    store_stream(p, w);
}

// A warp's task is `span` consecutive 512-element segments of one row (so that the
// index arithmetic, as long as a segment's, is paid once a task).
template <typename T, bool kNv, typename V>
__global__ void __launch_bounds__(kThreads)
    quantize_kernel(const T *x, int64_t x_rows, int64_t x_stride, int x_vec, int K, int span, const int32_t *row_index,
                    int index_div, int64_t rows, const float *tensor_scale, uint8_t *codes, uint8_t *scales,
                    V *values, int *status) {
    const int lane = threadIdx.x & 31;
    const int tasks = (K + 512 * span - 1) / (512 * span);      // a row
    const int64_t total = rows * tasks;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    float g = 1.0f;
    if constexpr (kNv) {
        g = __ldg(tensor_scale);
        if (!(g > 0.0f && g < __uint_as_float(kF32Inf))) set_status(status, MOE_ERR_DATA);
    }
    const float g6 = 6.0f * g;
    for (int64_t i = blockIdx.x * static_cast<int64_t>(kThreads / 32) + (threadIdx.x >> 5); i < total; i += step) {
        const int64_t r = tasks == 1 ? i : i / tasks;
        const int k_first = static_cast<int>(i - r * tasks) * span * 512, k_end = min(K, k_first + span * 512);
        int64_t src = r;
        bool have = true;
        if (row_index) {
            const int32_t idx = __ldg(row_index + r);
            src = idx / index_div;
            have = idx >= 0 && src < x_rows;
            if (!have && lane == 0) set_status(status, MOE_ERR_DATA);
        }
        const T *from = x + src * x_stride;
        uint8_t *to = codes + r * (K / 2), *to_scale = scales + r * (K / (kNv ? 16 : 32));
        V *to_value = values ? values + r * K : nullptr;
        for (int k1 = k_first; k1 < k_end; k1 += 512) {
            const int k0 = k1 + lane * 16;
            float v[16] = {};
            uint32_t m = 0;
            if (have && k0 < K) m = load16(from + k0, x_vec, v);
            if constexpr (!kNv) m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            if (k0 >= K) continue;
            uint32_t byte;
            float inv, unit;
            if constexpr (kNv) {
                byte = nv_scale_byte(m, g6);
                inv = nv_inverse(byte, g);
                unit = e4m3_value(byte);
            } else {
                byte = mx_scale_byte(m);
                inv = mx_inverse(byte);
                unit = mx_scale_value(byte);
            }
            uint32_t w[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float q[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) q[e] = v[8 * h + e] * inv;
                w[h] = byte == (kNv ? 0x7Fu : 255u) ? 0u : e2m1x8(q);
            }
            *reinterpret_cast<uint2 *>(to + k0 / 2) = make_uint2(w[0], w[1]);
            if (kNv || (k0 & 16) == 0) to_scale[k0 / (kNv ? 16 : 32)] = static_cast<uint8_t>(byte);
            if (to_value) {
                // The values the codes stand for: exact in bf16 for MX; in f32 one
                // rounding (the product with g) for NV.
                float o[16];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float e8[8];
                    e2m1x8_values(w[h], e8);
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[8 * h + e] = kNv ? e8[e] * unit * g : e8[e] * unit;
                }
                store16(to_value + k0, o);
            }
        }
    }
}

}  // namespace quant

namespace {

template <typename T, bool kNv, typename V>
void start(const Fp4Quant &q, V *values, cudaStream_t stream, int num_sms) {
    // Whole rows a warp where that leaves two tasks a warp of the grid, else segments.
    const int segs = (q.K + 511) / 512;
    const int span = q.rows >= static_cast<int64_t>(num_sms) * 64 * 2 ? segs : 1;
    const int64_t warps = q.rows * ((segs + span - 1) / span);
    int64_t blocks = (warps + 7) / 8;
    const int64_t cap = static_cast<int64_t>(num_sms) * 8;
    if (blocks > cap) blocks = cap;
    const T *x = static_cast<const T *>(q.x);
    const int x_vec = (reinterpret_cast<uintptr_t>(x) & 15) == 0 && (q.x_stride * sizeof(T)) % 16 == 0;
    quant::quantize_kernel<T, kNv, V><<<static_cast<int>(blocks), quant::kThreads, 0, stream>>>(
        x, q.x_rows, q.x_stride, x_vec, q.K, span, q.row_index, q.index_div, q.rows, q.tensor_scale, q.codes, q.scales,
        values, q.status);
}

template <typename T, bool kNv>
void start_values(const Fp4Quant &q, cudaStream_t stream, int num_sms) {
    if (q.values_bf16)
        start<T, kNv, __nv_bfloat16>(q, static_cast<__nv_bfloat16 *>(q.values), stream, num_sms);
    else
        start<T, kNv, float>(q, static_cast<float *>(q.values), stream, num_sms);
}

}  // namespace

moe_status launch_fp4_quantize(const Fp4Quant &q, cudaStream_t stream, int num_sms) {
    if (q.rows == 0) return MOE_OK;
    if (q.in_bf16) {
        if (q.nv) start_values<__nv_bfloat16, true>(q, stream, num_sms);
        else start_values<__nv_bfloat16, false>(q, stream, num_sms);
    } else {
        if (q.nv) start_values<float, true>(q, stream, num_sms);
        else start_values<float, false>(q, stream, num_sms);
    }
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
