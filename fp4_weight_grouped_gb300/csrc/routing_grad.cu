// Gradients of the weighted unsort (moe_combine) and of the sort's gather.
//
//   out[t] = sum_j w[t, j] y[row(t, j)]    =>  dy[row(t, j)] = w[t, j] dout[t]
//                                              dw[t, j] = <dout[t], y[row(t, j)]>
//   x_sorted[row(t, j)] = x[t]             =>  dx[t] = sum_j dx_sorted[row(t, j)]
//
// row(t, j) = slot_to_row[t k + j]; a slot without a row (-1) takes part in
// nothing and its dw is 0.  Every output element has one writer and every sum
// one fixed order (no atomics): results repeat bit for bit.
//
// Bound: HBM.  Measured, T = 8,192, k = 6, N = 4,096, bf16, both gradients (a combine's and
// a gather's): 269 us for 1.75 GB, 6.5 TB/s, 95% of the measured copy rate; T = 250,
// N = 1,028: 5.9 us, two launches' latency.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "launch.h"
#include "vec_io.cuh"

namespace moe {
namespace grad {

constexpr int kThreads = 256;

// One warp a slot: it reads dout[t] (the k warps of a token share it through
// L1 / L2), reads y's row, writes dy's row and sums the products in f32.
template <typename G, typename Y, typename D, int V>
__global__ void __launch_bounds__(kThreads)
    combine_backward_kernel(const G *dout, const Y *y, const int32_t *s2r, const float *w, int64_t slots, int k,
                            int N, D *dy, float *dw) {
    const int lane = threadIdx.x & 31;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    for (int64_t s = blockIdx.x * static_cast<int64_t>(kThreads / 32) + (threadIdx.x >> 5); s < slots; s += step) {
        const int32_t r = __ldg(s2r + s);
        if (r < 0 || r >= slots) {
            if (dw && lane == 0) dw[s] = 0.0f;
            continue;
        }
        const G *g = dout + (s / k) * static_cast<int64_t>(N);
        const Y *yr = y + static_cast<int64_t>(r) * N;
        D *dr = dy + static_cast<int64_t>(r) * N;
        const float wj = __ldg(w + s);
        float acc = 0.0f;
#pragma unroll 4
        for (int c = lane * V; c < N; c += 32 * V) {
            float a[V];
            load_row<V>(g + c, a);
            if (dw) {
                float b[V];
                load_row<V>(yr + c, b);
#pragma unroll
                for (int i = 0; i < V; ++i) acc = fmaf(a[i], b[i], acc);
            }
            if (dy) {
#pragma unroll
                for (int i = 0; i < V; ++i) a[i] *= wj;
                store_row<V>(dr + c, a);
            }
        }
        if (dw) {
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, d);
            if (lane == 0) dw[s] = acc;
        }
    }
}

// The same with `lanes` threads a slot: a power of two below 32 where a row has fewer
// vectors than a warp has lanes (T = 8,192, k = 6, bf16, both gradients: N = 4 in 5.0 us
// for 14.5 with a warp a slot, N = 132 in 15.7 for 18.1), the whole block where few slots
// have long rows (T = 16, k = 8, N = 4,096: 6.1 us for 8.3).
template <typename G, typename Y, typename D, int V>
__global__ void __launch_bounds__(kThreads)
    combine_backward_lanes_kernel(const G *dout, const Y *y, const int32_t *s2r, const float *w, int64_t slots, int k,
                                  int N, int lanes, D *dy, float *dw) {
    __shared__ float part[kThreads / 32];
    const int sub = threadIdx.x & (lanes - 1), a_block = kThreads / lanes;
    const int64_t step = static_cast<int64_t>(gridDim.x) * a_block;
    for (int64_t s0 = blockIdx.x * static_cast<int64_t>(a_block); s0 < slots; s0 += step) {   // block-uniform
        const int64_t s = s0 + threadIdx.x / lanes;
        const int32_t r = s < slots ? __ldg(s2r + s) : -1;
        float acc = 0.0f;
        if (r >= 0 && r < slots) {
            const int64_t t = slots <= INT32_MAX ? static_cast<uint32_t>(s) / static_cast<uint32_t>(k) : s / k;
            const G *g = dout + t * N;
            const Y *yr = y + static_cast<int64_t>(r) * N;
            D *dr = dy + static_cast<int64_t>(r) * N;
            const float wj = __ldg(w + s);
#pragma unroll 4
            for (int c = sub * V; c < N; c += lanes * V) {
                float a[V];
                load_row<V>(g + c, a);
                if (dw) {
                    float b[V];
                    load_row<V>(yr + c, b);
#pragma unroll
                    for (int i = 0; i < V; ++i) acc = fmaf(a[i], b[i], acc);
                }
                if (dy) {
#pragma unroll
                    for (int i = 0; i < V; ++i) a[i] *= wj;
                    store_row<V>(dr + c, a);
                }
            }
        }
        if (dw) {
            for (int d = lanes < 32 ? lanes / 2 : 16; d > 0; d >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, d);
            if (lanes > 32) {
                if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = acc;
                __syncthreads();
                acc = 0.0f;
                for (int i = 0; i < kThreads / 32; ++i) acc += part[i];
                __syncthreads();                            // part is written again by the next slot
            }
            if (sub == 0 && s < slots) dw[s] = acc;         // 0 for a slot without a row
        }
    }
}

// A thread owns V columns of one token; the k rows are summed in ascending j.
template <typename G, typename D, int V>
__global__ void __launch_bounds__(kThreads)
    gather_backward_kernel(const G *dxs, const int32_t *s2r, int T, int k, int N, D *dx) {
    const int vecs = N / V;
    const int64_t rows = static_cast<int64_t>(T) * k, total = static_cast<int64_t>(T) * vecs;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
    for (int64_t i = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x; i < total; i += step) {
        const int64_t t = total <= INT32_MAX ? static_cast<uint32_t>(i) / static_cast<uint32_t>(vecs) : i / vecs;
        const int c = static_cast<int>(i - t * vecs) * V;
        float acc[V];
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = 0.0f;
#pragma unroll 4
        for (int j = 0; j < k; ++j) {
            const int32_t r = __ldg(s2r + t * k + j);
            if (r < 0 || r >= rows) continue;
            float a[V];
            load_row<V>(dxs + static_cast<int64_t>(r) * N + c, a);
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] += a[e];
        }
        store_row<V>(dx + t * N + c, acc);
    }
}

}  // namespace grad

namespace {

// A block a slot up to 4 slots an SM, for rows of 128 vectors or more: above either a warp a
// slot has enough in flight (bf16, k = 8, block / warp: 512 x 4,096 in 7.0 / 8.5 us, 1,024 x
// 4,096 in 8.9 / 8.8, 2,048 x 4,096 in 11.5 / 10.7; 512 x 512 in 6.3 / 6.0).
constexpr int kBlockSlotsPerSm = 4, kBlockVectors = 128;

template <typename G, typename Y, typename D>
void combine_backward(const CombineGrad &c, cudaStream_t stream, int num_sms) {
    const int64_t slots = static_cast<int64_t>(c.T) * c.k;
    const int V = c.N % 8 == 0 ? 8 : c.N % 4 == 0 ? 4 : 1;
    int lanes = 32;
    while (lanes > 1 && (lanes / 2) * V >= c.N) lanes /= 2;
    if (slots <= kBlockSlotsPerSm * static_cast<int64_t>(num_sms) && c.N >= kBlockVectors * V) lanes = grad::kThreads;
    const int a_block = grad::kThreads / lanes;
    const int64_t blocks = (slots + a_block - 1) / a_block, cap = static_cast<int64_t>(num_sms) * 8;
    const int grid = static_cast<int>(blocks < cap ? blocks : cap);
    const G *g = static_cast<const G *>(c.dout);
    const Y *y = static_cast<const Y *>(c.y);
    D *dy = static_cast<D *>(c.dy);
    auto launch = [&](auto v) {
        constexpr int kV = decltype(v)::value;
        if (lanes == 32)
            grad::combine_backward_kernel<G, Y, D, kV>
                <<<grid, grad::kThreads, 0, stream>>>(g, y, c.s2r, c.w, slots, c.k, c.N, dy, c.dw);
        else
            grad::combine_backward_lanes_kernel<G, Y, D, kV>
                <<<grid, grad::kThreads, 0, stream>>>(g, y, c.s2r, c.w, slots, c.k, c.N, lanes, dy, c.dw);
    };
    if (V == 8) launch(std::integral_constant<int, 8>());
    else if (V == 4) launch(std::integral_constant<int, 4>());
    else launch(std::integral_constant<int, 1>());
}

template <typename G, typename D>
void gather_backward(const void *dxs, const int32_t *s2r, int T, int k, int N, void *dx, cudaStream_t stream,
                     int num_sms) {
    const G *g = static_cast<const G *>(dxs);
    D *d = static_cast<D *>(dx);
    const int V = N % 8 == 0 ? 8 : N % 4 == 0 ? 4 : 1;
    const int64_t blocks = (static_cast<int64_t>(T) * (N / V) + grad::kThreads - 1) / grad::kThreads;
    const int64_t cap = static_cast<int64_t>(num_sms) * 8;
    const int grid = static_cast<int>(blocks < cap ? blocks : cap);
    if (V == 8) grad::gather_backward_kernel<G, D, 8><<<grid, grad::kThreads, 0, stream>>>(g, s2r, T, k, N, d);
    else if (V == 4) grad::gather_backward_kernel<G, D, 4><<<grid, grad::kThreads, 0, stream>>>(g, s2r, T, k, N, d);
    else grad::gather_backward_kernel<G, D, 1><<<grid, grad::kThreads, 0, stream>>>(g, s2r, T, k, N, d);
}

}  // namespace

moe_status launch_combine_backward(const CombineGrad &c, cudaStream_t stream, int num_sms) {
    if (c.T == 0) return MOE_OK;
    using B = __nv_bfloat16;
    switch ((c.dout_bf16 ? 4 : 0) | (c.y_bf16 ? 2 : 0) | (c.dy_bf16 ? 1 : 0)) {
        case 0: combine_backward<float, float, float>(c, stream, num_sms); break;
        case 1: combine_backward<float, float, B>(c, stream, num_sms); break;
        case 2: combine_backward<float, B, float>(c, stream, num_sms); break;
        case 3: combine_backward<float, B, B>(c, stream, num_sms); break;
        case 4: combine_backward<B, float, float>(c, stream, num_sms); break;
        case 5: combine_backward<B, float, B>(c, stream, num_sms); break;
        case 6: combine_backward<B, B, float>(c, stream, num_sms); break;
        default: combine_backward<B, B, B>(c, stream, num_sms); break;
    }
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status launch_gather_backward(const void *dxs, int in_bf16, const int32_t *s2r, int T, int k, int N, void *dx,
                                  int out_bf16, cudaStream_t stream, int num_sms) {
    if (T == 0) return MOE_OK;
    using B = __nv_bfloat16;
    if (in_bf16) {
        if (out_bf16) gather_backward<B, B>(dxs, s2r, T, k, N, dx, stream, num_sms);
        else gather_backward<B, float>(dxs, s2r, T, k, N, dx, stream, num_sms);
    } else {
        if (out_bf16) gather_backward<float, B>(dxs, s2r, T, k, N, dx, stream, num_sms);
        else gather_backward<float, float>(dxs, s2r, T, k, N, dx, stream, num_sms);
    }
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
