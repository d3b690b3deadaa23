// Quantisation of activation rows to MXFP4 or NVFP4 (the rules are in
// fp4_common.cuh), with the routing permutation in the load.
//
// A thread owns 8 consecutive elements; a block of 32 (16) elements is 4 (2)
// lanes, whose maximum two (one) shuffles find.  A warp takes 256 elements of
// one row at a time, so its loads, code words and values are contiguous.  Bound:
// HBM; an element costs about ten instructions.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fp4_common.cuh"
#include "launch.h"
#include "vec_io.cuh"

namespace moe {
namespace quant {

constexpr int kThreads = 256;

template <typename T, bool kNv, typename V>
__global__ void __launch_bounds__(kThreads)
    quantize_kernel(const T *x, int64_t x_rows, int64_t x_stride, int x_vec, int K, const int32_t *row_index,
                    int index_div, int64_t rows, const float *tensor_scale, uint8_t *codes, uint8_t *scales,
                    V *values, int *status) {
    constexpr int kBlock = kNv ? 16 : 32;
    const int lane = threadIdx.x & 31;
    const int segs = (K + 255) / 256;
    const int64_t total = rows * segs;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    float g = 1.0f;
    if constexpr (kNv) {
        g = __ldg(tensor_scale);
        if (!(g > 0.0f && g < __uint_as_float(kF32Inf))) set_status(status, MOE_ERR_DATA);
    }
    const float g6 = 6.0f * g;
    for (int64_t i = blockIdx.x * static_cast<int64_t>(kThreads / 32) + (threadIdx.x >> 5); i < total; i += step) {
        const int64_t r = i / segs;
        const int k0 = static_cast<int>(i - r * segs) * 256 + lane * 8;
        int64_t src = r;
        bool have = true;
        if (row_index) {
            const int32_t idx = __ldg(row_index + r);
            src = idx / index_div;
            have = idx >= 0 && src < x_rows;
            if (!have && lane == 0) set_status(status, MOE_ERR_DATA);
        }
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (have && k0 < K) {
            const T *p = x + src * x_stride + k0;
            if (x_vec) {
                load_row<8>(p, v);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float one[1];
                    load_row<1>(p + e, one);
                    v[e] = one[0];
                }
            }
        }
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[e]) & 0x7FFFFFFFu);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        if constexpr (!kNv) m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        uint32_t byte;
        float inv, unit;
        bool nan;
        if constexpr (kNv) {
            byte = nv_scale_byte(m, g6);
            inv = nv_inverse(byte, g);
            unit = e4m3_value(byte);
            nan = byte == 0x7Fu;
        } else {
            byte = mx_scale_byte(m);
            inv = mx_inverse(byte);
            unit = mx_scale_value(byte);
            nan = byte == 255u;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = nan ? 0.0f : v[e] * inv;
        const uint32_t w = e2m1x8(v);
        if (k0 >= K) continue;
        *reinterpret_cast<uint32_t *>(codes + r * (K / 2) + k0 / 2) = w;
        if (k0 % kBlock == 0) scales[r * (K / kBlock) + k0 / kBlock] = static_cast<uint8_t>(byte);
        if (values) {
            // The values the codes stand for: exact in bf16 for MX; in f32 one
            // rounding (the product with g) for NV.
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t c = (w >> (4 * e)) & 15u, mag = c & 7u;
                // e2m1 magnitude from its bits: (mag < 2) 0, 0.5; else 1.f * 2^(e - 1)
                const float a = mag < 2u ? 0.5f * static_cast<float>(mag)
                                         : __uint_as_float((mag << 22) + (126u << 23));
                const float s = c & 8u ? -a : a;
                o[e] = s * unit;
                if constexpr (kNv) o[e] *= g;
            }
            store_row<8>(values + r * K + k0, o);
        }
    }
}

}  // namespace quant

namespace {

template <typename T, bool kNv, typename V>
void start(const Fp4Quant &q, V *values, cudaStream_t stream, int num_sms) {
    const int64_t warps = q.rows * ((q.K + 255) / 256);
    int64_t blocks = (warps + 7) / 8;
    const int64_t cap = static_cast<int64_t>(num_sms) * 8;
    if (blocks > cap) blocks = cap;
    const T *x = static_cast<const T *>(q.x);
    const int x_vec = (reinterpret_cast<uintptr_t>(x) & 15) == 0 && (q.x_stride * sizeof(T)) % 16 == 0;
    quant::quantize_kernel<T, kNv, V><<<static_cast<int>(blocks), quant::kThreads, 0, stream>>>(
        x, q.x_rows, q.x_stride, x_vec, q.K, q.row_index, q.index_div, q.rows, q.tensor_scale, q.codes, q.scales,
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
