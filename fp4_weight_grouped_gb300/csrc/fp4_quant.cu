// Quantisation of activation rows to MXFP4 or NVFP4 (the rules are in
// fp4_common.cuh), with the routing permutation in the load.
//
// A lane owns 16 consecutive elements: an NV block, or half an MX block, whose other
// half one shuffle reaches.  A warp takes 512 elements of one row at a time, so its
// loads, code words and values are contiguous.  Magnitudes are compared as integers,
// for bf16 two in a word.
//
// Bound: HBM writes where values are asked for, instruction issue where not.  Measured,
// 49,152 rows of 4,096 bf16 gathered from 8,192 tokens: MXFP4 codes alone 64 us, NVFP4
// 70 us (three quarters of all issue slots, 2.7 TB/s; see kScatter for the layer's way); with bf16 values 124 us (578 MB;
// filling as many bytes as it writes takes 112 us); without the gather 83 us (6.1 TB/s).
// 3,001 rows of 2,080 f32 to NVFP4 with values: 9.4 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fp4_common.cuh"
#include "launch.h"
#include "vec_io.cuh"

namespace moe {
namespace quant {

constexpr int kThreads = 256;

// Sixteen elements as they lie in memory: 8 (bf16) or 16 (f32) words.
template <typename T>
struct Raw {
    static constexpr int kWords = 4 * sizeof(T);
    uint32_t w[kWords];
};

// 32 bytes in one instruction: a lane's 16 bf16 are one sector, which two 16-byte
// loads (or stores) would ask for twice.
__device__ __forceinline__ void load32(const void *p, uint32_t *w) {
    asm("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
        : "l"(p));
}

// align: 32 or 16, that of x's address and rows, or 0.
template <typename T>
__device__ __forceinline__ void load16(const T *p, int align, Raw<T> &r) {
    constexpr int n = Raw<T>::kWords;
    if (align == 32) {
#pragma unroll
        for (int i = 0; i < n; i += 8) load32(reinterpret_cast<const uint32_t *>(p) + i, r.w + i);
    } else if (align == 16) {
#pragma unroll
        for (int i = 0; i < n; i += 4) {
            const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p) + i / 4);
            r.w[i] = a.x; r.w[i + 1] = a.y; r.w[i + 2] = a.z; r.w[i + 3] = a.w;
        }
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < n; ++i) r.w[i] = __ldg(reinterpret_cast<const uint32_t *>(p) + i);
    } else {
        const uint16_t *u = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
        for (int i = 0; i < n; ++i) r.w[i] = __ldg(u + 2 * i) | static_cast<uint32_t>(__ldg(u + 2 * i + 1)) << 16;
    }
}

// The largest magnitude's f32 bits.
__device__ __forceinline__ uint32_t largest16(const Raw<float> &r) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 16; ++e) m = max(m, r.w[e] & 0x7FFFFFFFu);
    return m;
}

__device__ __forceinline__ uint32_t largest16(const Raw<__nv_bfloat16> &r) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, r.w[i] & 0x7FFF7FFFu);
    return max(m & 0xFFFF0000u, m << 16);
}

// Values, to be evicted first: they are not read again here, and x's rows, which are
// (once for each choice of a token), stay in L2.
__device__ __forceinline__ void store_stream(void *p, const uint32_t (&w)[8], bool wide) {
    if (wide) {
        asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
                     "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        __stcs(static_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2], w[3]));
        __stcs(static_cast<uint4 *>(p) + 1, make_uint4(w[4], w[5], w[6], w[7]));
    }
}

__device__ __forceinline__ void store16(float *p, const float (&v)[16], bool wide) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(v[8 * h + e]);
        store_stream(p + 8 * h, w, wide);
    }
}

__device__ __forceinline__ void store16(__nv_bfloat16 *p, const float (&v)[16], bool wide) {
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = bf16_pair(v[2 * e], v[2 * e + 1]);
    store_stream(p, w, wide);
}

// The elements times a block's inverse scale.
__device__ __forceinline__ void scaled16(const Raw<float> &r, float inv, float (&q)[16]) {
#pragma unroll
    for (int e = 0; e < 16; ++e) q[e] = __uint_as_float(r.w[e]) * inv;
}

__device__ __forceinline__ void scaled16(const Raw<__nv_bfloat16> &r, float inv, float (&q)[16]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        q[2 * i] = bf16_low(r.w[i]) * inv;
        q[2 * i + 1] = bf16_high(r.w[i]) * inv;
    }
}

// A row without a source: zeros.
template <bool kNv, typename V>
__device__ __noinline__ void zero_row(int k_first, int k_end, uint8_t *to, uint8_t *to_scale, V *to_value) {
    for (int k = k_first + (threadIdx.x & 31) * 16; k < k_end; k += 512) {
        *reinterpret_cast<uint2 *>(to + k / 2) = make_uint2(0u, 0u);
        to_scale[k / (kNv ? 16 : 32)] = 0;
        if (to_value)
            for (int e = 0; e < 16; ++e) to_value[k + e] = V(0.0f);
    }
}

// A warp's task is `span` consecutive 512-element segments of one row (so that the
// index arithmetic, as long as a segment's, is paid once a task); a segment's loads are
// issued before the one in front of it is worked on.  Lanes past the row's end work on
// its last block again and store what its own lanes store, so nothing in the loop
// branches by lane.  kValues: `values` is there.
//
// kScatter: the rows are tokens, and codes and scales go to the k rows of each token's
// slots, so that a token is loaded and quantised once, not k times (a whole W4A4 layer of
// 8,192 tokens, top-6: MXFP4 963 -> 937 us, NVFP4 1,010 -> 979 us).
template <typename T, bool kNv, typename V, bool kValues, bool kScatter>
__global__ void __launch_bounds__(kThreads)
    quantize_kernel(const T *x, int64_t x_rows, int64_t x_stride, int x_align, int K, int span,
                    const int32_t *row_index, int index_div, int64_t rows, const float *tensor_scale, uint8_t *codes, uint8_t *scales,
                    V *values, int values_wide, int *status, const int32_t *slot_to_row, int k, int64_t out_rows) {
    const int lane = threadIdx.x & 31;
    const int tasks = (K + 512 * span - 1) / (512 * span);      // a row
    const int64_t total = rows * tasks;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    const int k_last = K - 32 + (lane & 1) * 16;
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
        }
        const T *from = x + src * x_stride;
        uint8_t *to = codes + r * (K / 2), *to_scale = scales + r * (K / (kNv ? 16 : 32));
        V *to_value = kValues ? values + r * K : nullptr;
        if (!have) {                                            // warp-uniform
            if (lane == 0) set_status(status, MOE_ERR_DATA);
            zero_row<kNv, V>(k_first, k_end, to, to_scale, to_value);
            continue;
        }
        int k0 = min(k_first + lane * 16, k_last);
        Raw<T> next;
        load16(from + k0, x_align, next);
        for (int k1 = k_first; k1 < k_end; k1 += 512) {
            const Raw<T> now = next;
            const int at = k0;
            if (k1 + 512 < k_end) {
                k0 = min(k0 + 512, k_last);
                load16(from + k0, x_align, next);
            }
            uint32_t m = largest16(now);
            if constexpr (!kNv) m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
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
            float v[16];
            scaled16(now, inv, v);
            uint32_t w[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float q[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) q[e] = v[8 * h + e];
                w[h] = byte == (kNv ? 0x7Fu : 255u) ? 0u : e2m1x8(q);
            }
            if constexpr (kScatter) {
#pragma unroll 4
                for (int j = 0; j < k; ++j) {
                    const int32_t d = __ldg(slot_to_row + r * k + j);
                    if (d < 0 || d >= out_rows) continue;       // a slot without a row
                    *reinterpret_cast<uint2 *>(codes + static_cast<int64_t>(d) * (K / 2) + at / 2) = make_uint2(w[0], w[1]);
                    if (kNv || (lane & 1) == 0)
                        scales[static_cast<int64_t>(d) * (K / (kNv ? 16 : 32)) + at / (kNv ? 16 : 32)] =
                            static_cast<uint8_t>(byte);
                }
                continue;
            }
            *reinterpret_cast<uint2 *>(to + at / 2) = make_uint2(w[0], w[1]);
            if (kNv || (lane & 1) == 0) to_scale[at / (kNv ? 16 : 32)] = static_cast<uint8_t>(byte);
            if constexpr (kValues) {
                // The values the codes stand for: exact in bf16 for MX; for NV one
                // rounding to f32 (the product with g), and one more where V is bf16.
                float o[16];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float e8[8];
                    e2m1x8_values(w[h], e8);
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[8 * h + e] = kNv ? e8[e] * unit * g : e8[e] * unit;
                }
                store16(to_value + at, o, values_wide);
            }
        }
    }
}

}  // namespace quant

namespace {

template <typename T, bool kNv, typename V, bool kValues, bool kScatter>
void start(const Fp4Quant &q, V *values, cudaStream_t stream, int num_sms) {
    // Whole rows a warp where there are two rows a warp that fits the SM, else segments.
    // 24 blocks an SM: 4 or 5 are resident, and the rest go to whichever is done first (the
    // case above, 8 / 16 / 24 / 64 blocks: 73 / 70 / 68 / 70 us).
    const int segs = (q.K + 511) / 512;
    const int span = q.rows >= static_cast<int64_t>(num_sms) * 64 * 2 ? segs : 1;
    const int64_t warps = q.rows * ((segs + span - 1) / span);
    int64_t blocks = (warps + 7) / 8;
    const int64_t cap = static_cast<int64_t>(num_sms) * 24;
    if (blocks > cap) blocks = cap;
    const T *x = static_cast<const T *>(q.x);
    const uintptr_t x_at = reinterpret_cast<uintptr_t>(x) | static_cast<uintptr_t>(q.x_stride * sizeof(T));
    const int x_align = x_at % 32 == 0 ? 32 : x_at % 16 == 0 ? 16 : 0;
    const int wide = reinterpret_cast<uintptr_t>(values) % 32 == 0;   // K % 32 = 0: every row then
    quant::quantize_kernel<T, kNv, V, kValues, kScatter><<<static_cast<int>(blocks), quant::kThreads, 0, stream>>>(
        x, q.x_rows, q.x_stride, x_align, q.K, span, q.row_index, q.index_div, q.rows, q.tensor_scale, q.codes,
        q.scales, values, wide, q.status, q.slot_to_row, q.k, q.out_rows);
}

template <typename T, bool kNv>
void start_values(const Fp4Quant &q, cudaStream_t stream, int num_sms) {
    if (q.slot_to_row)
        start<T, kNv, float, false, true>(q, nullptr, stream, num_sms);
    else if (!q.values)
        start<T, kNv, float, false, false>(q, nullptr, stream, num_sms);
    else if (q.values_bf16)
        start<T, kNv, __nv_bfloat16, true, false>(q, static_cast<__nv_bfloat16 *>(q.values), stream, num_sms);
    else
        start<T, kNv, float, true, false>(q, static_cast<float *>(q.values), stream, num_sms);
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
