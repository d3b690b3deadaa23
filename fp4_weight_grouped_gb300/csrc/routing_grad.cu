// Gradients of the weighted unsort (moe_combine) and of the sort's gather.
//
//   out[t] = sum_j w[t, j] y[row(t, j)]    =>  dy[row(t, j)] = w[t, j] dout[t]
//                                              dw[t, j] = <dout[t], y[row(t, j)]>
//   x_sorted[row(t, j)] = x[t]             =>  dx[t] = sum_j dx_sorted[row(t, j)]
//
// row(t, j) = slot_to_row[t k + j]; a slot without a row (-1) takes part in
// nothing and its dw is 0.  Every output element has one writer and every sum
// one fixed order (no atomics): results repeat bit for bit.  Bound: HBM.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

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

// One warp a segment of 32 V columns of one token; the k rows are summed in
// ascending j.
template <typename G, typename D, int V>
__global__ void __launch_bounds__(kThreads)
    gather_backward_kernel(const G *dxs, const int32_t *s2r, int T, int k, int N, D *dx) {
    const int lane = threadIdx.x & 31;
    const int segs = (N + 32 * V - 1) / (32 * V);
    const int64_t rows = static_cast<int64_t>(T) * k, total = static_cast<int64_t>(T) * segs;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    for (int64_t i = blockIdx.x * static_cast<int64_t>(kThreads / 32) + (threadIdx.x >> 5); i < total; i += step) {
        const int64_t t = i / segs;
        const int c = (static_cast<int>(i - t * segs) * 32 + lane) * V;
        if (c >= N) continue;
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

int grid_for(int64_t warps, int num_sms) {
    int64_t blocks = (warps + 7) / 8;
    const int64_t cap = static_cast<int64_t>(num_sms) * 8;
    return static_cast<int>(blocks < cap ? blocks : cap);
}

template <typename G, typename Y, typename D>
void combine_backward(const CombineGrad &c, cudaStream_t stream, int num_sms) {
    const int64_t slots = static_cast<int64_t>(c.T) * c.k;
    const int grid = grid_for(slots, num_sms);
    const G *g = static_cast<const G *>(c.dout);
    const Y *y = static_cast<const Y *>(c.y);
    D *dy = static_cast<D *>(c.dy);
    if (c.N % 8 == 0)
        grad::combine_backward_kernel<G, Y, D, 8><<<grid, grad::kThreads, 0, stream>>>(g, y, c.s2r, c.w, slots, c.k, c.N, dy, c.dw);
    else if (c.N % 4 == 0)
        grad::combine_backward_kernel<G, Y, D, 4><<<grid, grad::kThreads, 0, stream>>>(g, y, c.s2r, c.w, slots, c.k, c.N, dy, c.dw);
    else
        grad::combine_backward_kernel<G, Y, D, 1><<<grid, grad::kThreads, 0, stream>>>(g, y, c.s2r, c.w, slots, c.k, c.N, dy, c.dw);
}

template <typename G, typename D>
void gather_backward(const void *dxs, const int32_t *s2r, int T, int k, int N, void *dx, cudaStream_t stream,
                     int num_sms) {
    const G *g = static_cast<const G *>(dxs);
    D *d = static_cast<D *>(dx);
    const int V = N % 8 == 0 ? 8 : N % 4 == 0 ? 4 : 1;
    const int grid = grid_for(static_cast<int64_t>(T) * ((N + 32 * V - 1) / (32 * V)), num_sms);
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
