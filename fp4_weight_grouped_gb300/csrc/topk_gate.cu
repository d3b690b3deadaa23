// Router gate: the k largest of E logits a token and their softmax weights, and
// the gradient with respect to the logits.
//
//   ids   the k largest logits in descending order; equal logits (and -0, +0) by
//         ascending expert; a NaN ranks with -inf.
//   w     softmax over all E logits taken at the chosen ones, or (renorm) softmax
//         over the chosen k alone.  A row without a finite maximum because every
//         logit that counts is -inf has weights 0.
//   dl    with dot = sum_j w_j dw_j:  p_e (dw_e - dot) over all E experts (dw_e =
//         0 where e was not chosen), or (renorm) w_j (dw_j - dot) at the chosen
//         ones and 0 elsewhere.
//
// One warp a token, the row in registers (expert lane + 32 i in register i), f32
// throughout.  A selection step is one redux for the largest key and one for
// the lowest expert that has it.
//
// Bound: launches for few tokens, instruction issue for many.  Measured, bf16, 256 experts,
// k = 6, renorm, forward / gradient: 64 tokens 3.1 / 2.1 us, two launches' time; 8,192 tokens
// 8.8 / 3.4; from 32,768 tokens on 0.8 / 0.25 ns a token (26.8 / 7.7 us).  The forward takes
// 651 instructions a token (ncu: 57% of issue slots while active, the selection's reductions
// and compares waiting for their pipe), the gradient 192, against 1.3 us of bytes for both at
// 8,192 tokens.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "launch.h"
#include "vec_io.cuh"

namespace moe {
namespace gate {

constexpr int kThreads = 128;
constexpr uint32_t kAll = 0xffffffffu;

// Unsigned key with the order of the logits; never 0.
__device__ __forceinline__ uint32_t key_of(float v) {
    if (v != v) v = -CUDART_INF_F;
    const uint32_t u = __float_as_uint(v + 0.0f);   // -0 + 0 = +0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

// e^(v - m), 0 for v = -inf (also where m is -inf).
__device__ __forceinline__ float exp_of(float v, float m) { return v == -CUDART_INF_F ? 0.0f : expf(v - m); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    return v;
}

template <typename T>
__device__ __forceinline__ float load_one(const T *p) {
    float v[1];
    load_row<1>(p, v);
    return v[0];
}

template <typename T, int R>
__global__ void __launch_bounds__(kThreads)
    gate_kernel(const T *logits, int64_t stride, int n, int E, int k, int renorm, int32_t *ids, float *weights) {
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (t >= n) return;
    const T *row = logits + t * stride;
    float v[R];
    uint32_t key[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int e = lane + 32 * i;
        v[i] = e < E ? load_one(row + e) : -CUDART_INF_F;
        key[i] = e < E ? key_of(v[i]) : 0u;
    }
    uint32_t best = 0, at = 0;
    auto scan = [&] {
        best = key[0];
        at = 0;
#pragma unroll
        for (int i = 1; i < R; ++i)
            if (key[i] > best) { best = key[i]; at = i; }
    };
    scan();
    const float m = value_of(__reduce_max_sync(kAll, best));
    float sum = 0.0f;
    if (!renorm) {
#pragma unroll
        for (int i = 0; i < R; ++i) sum += exp_of(v[i], m);
        sum = warp_sum(sum);
    }
    int32_t *out_id = ids + static_cast<int64_t>(t) * k;
    float *out_w = weights + static_cast<int64_t>(t) * k;
    for (int j = 0; j < k; ++j) {
        const uint32_t top = __reduce_max_sync(kAll, best);
        const uint32_t e = __reduce_min_sync(kAll, best == top ? lane + 32u * at : 0xFFFFFFFFu);
        if (lane == 0) out_id[j] = static_cast<int32_t>(e);
        if (static_cast<int>(e & 31u) == lane) {
#pragma unroll
            for (int i = 0; i < R; ++i) key[i] = i == static_cast<int>(e >> 5) ? 0u : key[i];
            scan();
        }
    }
    // The weights, a chosen expert a lane: its logit comes from memory again (a
    // register picked by a run-time index would put the row into local memory).
    __syncwarp();
    float total = 0.0f;
    for (int j = lane; j < k; j += 32) {
        const float x = exp_of(load_one(row + out_id[j]), m);
        if (renorm) { out_w[j] = x; total += x; }
        else out_w[j] = sum == 0.0f ? 0.0f : x / sum;
    }
    if (renorm) {
        total = warp_sum(total);
        for (int j = lane; j < k; j += 32) out_w[j] = total == 0.0f ? 0.0f : out_w[j] / total;
    }
}

// Gradient for k <= 32: chosen expert j and its dw in lane j.  An id that appears
// more than once is the lowest such lane's, with the sum of their dw in lane order;
// one outside [0, E) is nobody's.
template <typename T, int R>
__global__ void __launch_bounds__(kThreads)
    gate_backward_small_kernel(const T *logits, int64_t stride, int n, int E, int k, int renorm, const int32_t *ids,
                               const float *dw, T *dlogits) {
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (t >= n) return;
    const T *row = logits + t * stride;
    T *out = dlogits + static_cast<int64_t>(t) * E;
    int id = -1;
    float d = 0.0f;
    if (lane < k) {
        id = __ldg(ids + static_cast<int64_t>(t) * k + lane);
        d = __ldg(dw + static_cast<int64_t>(t) * k + lane);
        if (static_cast<unsigned>(id) >= static_cast<unsigned>(E)) id = -1;
    }
    const uint32_t same = __match_any_sync(kAll, id);
    const bool mine = id >= 0 && __ffs(same) - 1 == lane;
    if (__any_sync(kAll, id >= 0 && (same & (same - 1)) != 0)) {
        float sum = 0.0f;
        for (int l = 0; l < 32; ++l) {
            const float x = __shfl_sync(kAll, d, l);
            if (same >> l & 1u) sum += x;
        }
        d = sum;
    }
    float l = mine ? load_one(row + id) : -CUDART_INF_F;
    float v[R];
    float m = l;                  // fmaxf skips NaN, as the forward's keys do
    if (!renorm) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int e = lane + 32 * i;
            v[i] = e < E ? load_one(row + e) : -CUDART_INF_F;
            m = fmaxf(m, v[i]);
        }
    }
    if (m != m) m = -CUDART_INF_F;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
    l = exp_of(l, m);
    float sum = renorm ? l : 0.0f;
    if (!renorm) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            v[i] = exp_of(v[i], m);
            sum += v[i];
        }
    }
    sum = warp_sum(sum);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    l *= inv;
    const float dot = warp_sum(mine ? l * d : 0.0f);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int e = lane + 32 * i;
        // (renorm: p is 0 here, and a NaN among the chosen reaches every expert)
        const float g[1] = {0.0f - (renorm ? 0.0f : v[i]) * inv * dot};
        if (e < E) store_row<1>(out + e, g);
    }
    __syncwarp();                 // the chosen experts' gradients replace what was just stored
    const float g[1] = {l * (d - dot)};
    if (mine) store_row<1>(out + id, g);
}

// Gradient for any k.
template <typename T, int R>
__global__ void __launch_bounds__(kThreads)
    gate_backward_kernel(const T *logits, int64_t stride, int n, int E, int k, int renorm, const int32_t *ids,
                         const float *dw, T *dlogits) {
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (t >= n) return;
    const T *row = logits + t * stride;
    const int32_t *id = ids + static_cast<int64_t>(t) * k;
    const float *d = dw + static_cast<int64_t>(t) * k;
    float p[R], grad[R];
    float m = -CUDART_INF_F, sum = 0.0f;
    // Gradient of the weights spread over the experts (ids outside [0, E) add
    // nothing), and with renorm the mask of the chosen ones.
    uint32_t chosen = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int e = lane + 32 * i;
        p[i] = e < E ? load_one(row + e) : -CUDART_INF_F;
        grad[i] = 0.0f;
    }
    for (int j = 0; j < k; ++j) {
        const int e = __ldg(id + j);
        const float dj = __ldg(d + j);
        if (static_cast<unsigned>(e) < static_cast<unsigned>(E) && (e & 31) == lane) {
            chosen |= 1u << (e >> 5);
#pragma unroll
            for (int i = 0; i < R; ++i) grad[i] += i == (e >> 5) ? dj : 0.0f;
        }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if (renorm && !(chosen >> i & 1u)) p[i] = -CUDART_INF_F;
        m = fmaxf(m, p[i]);          // skips NaN, as the forward's keys do
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
#pragma unroll
    for (int i = 0; i < R; ++i) {
        p[i] = exp_of(p[i], m);
        sum += p[i];
    }
    sum = warp_sum(sum);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        p[i] *= inv;
        dot = fmaf(p[i], grad[i], dot);
    }
    dot = warp_sum(dot);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int e = lane + 32 * i;
        const float g[1] = {p[i] * (grad[i] - dot)};
        if (e < E) store_row<1>(dlogits + static_cast<int64_t>(t) * E + e, g);
    }
}

template <typename T, int R>
void start(const Gate &g, bool backward, cudaStream_t stream) {
    const int blocks = static_cast<int>((static_cast<int64_t>(g.T) + kThreads / 32 - 1) / (kThreads / 32));
    const T *l = static_cast<const T *>(g.logits);
    if (backward && g.k <= 32)
        gate_backward_small_kernel<T, R><<<blocks, kThreads, 0, stream>>>(l, g.stride, g.T, g.E, g.k, g.renorm, g.ids,
                                                                         g.dw, static_cast<T *>(g.dlogits));
    else if (backward)
        gate_backward_kernel<T, R><<<blocks, kThreads, 0, stream>>>(l, g.stride, g.T, g.E, g.k, g.renorm, g.ids, g.dw,
                                                                   static_cast<T *>(g.dlogits));
    else
        gate_kernel<T, R><<<blocks, kThreads, 0, stream>>>(l, g.stride, g.T, g.E, g.k, g.renorm, g.ids, g.weights);
}

template <typename T>
void start_width(const Gate &g, bool backward, cudaStream_t stream) {
    // Registers a lane: the smallest power of two that holds the row.
    if (g.E <= 32) start<T, 1>(g, backward, stream);
    else if (g.E <= 64) start<T, 2>(g, backward, stream);
    else if (g.E <= 128) start<T, 4>(g, backward, stream);
    else if (g.E <= 256) start<T, 8>(g, backward, stream);
    else if (g.E <= 512) start<T, 16>(g, backward, stream);
    else start<T, 32>(g, backward, stream);
}

}  // namespace gate

moe_status launch_topk_gate(const Gate &g, bool backward, cudaStream_t stream) {
    if (g.T == 0) return MOE_OK;
    if (g.bf16) gate::start_width<__nv_bfloat16>(g, backward, stream);
    else gate::start_width<float>(g, backward, stream);
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
