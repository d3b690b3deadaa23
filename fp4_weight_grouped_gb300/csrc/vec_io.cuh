// Vector loads and stores of f32 / bf16 rows as f32 registers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

__device__ __forceinline__ float bf16_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&b);
}

// V consecutive elements at p; V = 8 or 4 need p aligned to 16 bytes or to the
// vector, whichever is less.
template <int V>
__device__ __forceinline__ void load_row(const float *p, float (&v)[V]) {
    if constexpr (V == 1) {
        v[0] = __ldg(p);
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 a = __ldg(reinterpret_cast<const float4 *>(p + i));
            v[i] = a.x; v[i + 1] = a.y; v[i + 2] = a.z; v[i + 3] = a.w;
        }
    }
}

template <int V>
__device__ __forceinline__ void load_row(const __nv_bfloat16 *p, float (&v)[V]) {
    if constexpr (V == 1) {
        v[0] = __bfloat162float(__ldg(p));
    } else if constexpr (V == 4) {
        const uint2 a = __ldg(reinterpret_cast<const uint2 *>(p));
        v[0] = bf16_low(a.x); v[1] = bf16_high(a.x); v[2] = bf16_low(a.y); v[3] = bf16_high(a.y);
    } else {
        const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p));
        v[0] = bf16_low(a.x); v[1] = bf16_high(a.x); v[2] = bf16_low(a.y); v[3] = bf16_high(a.y);
        v[4] = bf16_low(a.z); v[5] = bf16_high(a.z); v[6] = bf16_low(a.w); v[7] = bf16_high(a.w);
    }
}

template <int V>
__device__ __forceinline__ void store_row(float *p, const float (&v)[V]) {
    if constexpr (V == 1) {
        *p = v[0];
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 4)
            *reinterpret_cast<float4 *>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
}

template <int V>
__device__ __forceinline__ void store_row(__nv_bfloat16 *p, const float (&v)[V]) {
    if constexpr (V == 1) {
        *p = __float2bfloat16_rn(v[0]);
    } else if constexpr (V == 4) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
    } else {
        *reinterpret_cast<uint4 *>(p) = make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]),
                                                   bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
    }
}

}  // namespace moe
