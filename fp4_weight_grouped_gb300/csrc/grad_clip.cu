// Global norm of a list of gradient tensors, and clipping by it:
//
//   norm = sqrt(sum over all tensors of x^2),   out = x * min(1, max_norm / (norm + eps))
//
//  * Two kernels.  The first leaves one sum a block; every block of the second adds those
//    up again in the same order, so no counter or atomic decides an order and nothing has
//    to be cleared between calls.
//  * The tensors' addresses travel in the kernel's parameters, kCap a launch (longer lists
//    take several launches); a chunk of work finds its tensor by bisection.
//  * Squares are summed in f32 over the elements that a thread loads together and in f64
//    from there on.  Where such a sum is too small or large for f32 (elements under about
//    2^-50 or over 2^60) its squares are formed again in f64: the norm is right over the
//    whole range of the types.
//  * Bound by HBM: one read for the norm and a read and a write for the clipping.  The
//    second kernel goes through the chunks backwards, so what the first read last (the L2's
//    share) is not fetched again.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <new>

#include "device_common.cuh"
#include "launch.h"
#include "vec_io.cuh"

namespace moe {
namespace clip {

constexpr int kThreads = 256;
constexpr int kBlocksPerSm = 8;
constexpr int kVecs = 4;                  // 16-byte loads a thread has in flight

struct Tensor {
    const void *in;
    void *out;
    int64_t n;
    int32_t chunk0;                       // first chunk of the tensor in its launch
    int32_t bf16;
};

template <int kCap>
struct List {
    Tensor t[kCap];
    int count, chunks;
    int chunk;                            // elements a chunk, a multiple of 8
};

template <int kCap>
__device__ __forceinline__ int tensor_of(const List<kCap> &l, int chunk) {
    int lo = 0, hi = l.count - 1;         // the last tensor whose first chunk is not past it
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (l.t[mid].chunk0 <= chunk) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

template <typename T>
__device__ __forceinline__ float as_f32(T v) {
    if constexpr (sizeof(T) == 2) return __bfloat162float(v);
    else return v;
}

// f32 sums in this range hold their squares to f32 accuracy: what underflows (under 2^-126
// each) is below 2^-30 of it.
__device__ __forceinline__ bool sum_holds(float s) { return s > 0x1p-90f && s < 0x1p120f; }

template <int V>
__device__ __forceinline__ double squares(const float (&v)[V]) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) s = fmaf(v[i], v[i], s);
    if (sum_holds(s)) return s;
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) any |= __float_as_uint(v[i]) << 1;
    if (any == 0) return 0.0;
    double d = 0.0;
#pragma unroll 1
    for (int i = 0; i < V; ++i) d = fma(static_cast<double>(v[i]), static_cast<double>(v[i]), d);
    return d;
}

// Elements of [p, p + n) before the first 16-byte address.
template <typename T>
__device__ __forceinline__ int head_of(const T *p, int n) {
    return min(n, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / static_cast<int>(sizeof(T)));
}

template <typename T>
__device__ __forceinline__ double chunk_squares(const T *p, int n) {
    constexpr int V = 16 / sizeof(T);
    const int tid = threadIdx.x;
    double d = 0.0;
    const int head = head_of(p, n), vecs = (n - head) / V, tail = head + vecs * V;
    const T *q = p + head;
    int v = tid;
    for (; v + (kVecs - 1) * kThreads < vecs; v += kVecs * kThreads) {
        float x[kVecs][V];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) load_row<V>(q + static_cast<int64_t>(v + i * kThreads) * V, x[i]);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) d += squares(x[i]);
    }
    for (; v < vecs; v += kThreads) {
        float x[V];
        load_row<V>(q + static_cast<int64_t>(v) * V, x);
        d += squares(x);
    }
    // Up to V - 1 elements before and behind the vectors.
    const int at = tid < head ? tid : tail + tid - head;
    if (at < n && (tid < head || at >= tail)) {
        const double x = as_f32(p[at]);
        d = fma(x, x, d);
    }
    return d;
}

__device__ __forceinline__ double block_sum(double d, double *shared) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) d += __shfl_xor_sync(0xffffffffu, d, m);
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = d;
    __syncthreads();
    d = 0.0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) d += shared[w];
    return d;
}

template <int kCap>
__global__ void __launch_bounds__(kThreads) norm_kernel(const __grid_constant__ List<kCap> l, double *partial, int add) {
    __shared__ double shared[kThreads / 32];
    double d = 0.0;
    for (int c = blockIdx.x; c < l.chunks; c += gridDim.x) {
        const Tensor &t = l.t[tensor_of(l, c)];
        const int64_t at = static_cast<int64_t>(c - t.chunk0) * l.chunk;
        const int n = static_cast<int>(min(static_cast<int64_t>(l.chunk), t.n - at));
        if (t.bf16) d += chunk_squares(static_cast<const __nv_bfloat16 *>(t.in) + at, n);
        else d += chunk_squares(static_cast<const float *>(t.in) + at, n);
    }
    d = block_sum(d, shared);
    if (threadIdx.x == 0) partial[blockIdx.x] = add ? partial[blockIdx.x] + d : d;
}

// The sum of all partial sums, the same in every block.
__device__ __forceinline__ double total_of(const double *partial, int n, double *shared) {
    double d = 0.0;
    for (int i = threadIdx.x; i < n; i += kThreads) d += __ldcg(partial + i);
    return block_sum(d, shared);
}

template <typename T>
__device__ __forceinline__ void scale_chunk(const T *p, T *o, int n, float pre, float s) {
    constexpr int V = 16 / sizeof(T);
    const int tid = threadIdx.x;
    const bool together = ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(o)) & 15) == 0;
    const int head = together ? head_of(p, n) : 0, vecs = together ? (n - head) / V : 0, tail = head + vecs * V;
    const T *q = p + head;
    T *r = o + head;
    int v = tid;
    for (; v + (kVecs - 1) * kThreads < vecs; v += kVecs * kThreads) {
        float x[kVecs][V];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) load_row<V>(q + static_cast<int64_t>(v + i * kThreads) * V, x[i]);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
#pragma unroll
            for (int j = 0; j < V; ++j) x[i][j] = x[i][j] * pre * s;
            store_row<V>(r + static_cast<int64_t>(v + i * kThreads) * V, x[i]);
        }
    }
    for (; v < vecs; v += kThreads) {
        float x[V];
        load_row<V>(q + static_cast<int64_t>(v) * V, x);
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] = x[j] * pre * s;
        store_row<V>(r + static_cast<int64_t>(v) * V, x);
    }
    for (int i = tid; i < head; i += kThreads) {
        const float x[1] = {as_f32(p[i]) * pre * s};
        store_row<1>(o + i, x);
    }
    for (int i = tail + tid; i < n; i += kThreads) {
        const float x[1] = {as_f32(p[i]) * pre * s};
        store_row<1>(o + i, x);
    }
}

// The bits as they are (a NaN keeps its own).
template <typename T>
__device__ __forceinline__ void copy_chunk(const T *p, T *o, int n) {
    constexpr int V = 16 / sizeof(T);
    const int tid = threadIdx.x;
    const bool together = ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(o)) & 15) == 0;
    const int head = together ? head_of(p, n) : 0, vecs = together ? (n - head) / V : 0, tail = head + vecs * V;
    for (int v = tid; v < vecs; v += kThreads)
        reinterpret_cast<uint4 *>(o + head)[v] = __ldg(reinterpret_cast<const uint4 *>(p + head) + v);
    for (int i = tid; i < head; i += kThreads) o[i] = p[i];
    for (int i = tail + tid; i < n; i += kThreads) o[i] = p[i];
}

template <int kCap>
__global__ void __launch_bounds__(kThreads) scale_kernel(const __grid_constant__ List<kCap> l, const double *partial,
                                                         int n_partial, double max_norm, double eps, float *norm) {
    __shared__ double shared[kThreads / 32];
    const double total = sqrt(total_of(partial, n_partial, shared));
    if (blockIdx.x == 0 && threadIdx.x == 0 && norm) *norm = static_cast<float>(total);
    // A norm that is not finite clips nothing: the gradients are left (or copied) as they are.
    const bool clips = total < __longlong_as_double(0x7FF0000000000000ll) && max_norm < total + eps;
    // A scale near or below f32's smallest normal number (a norm past 2^100) would lose bits:
    // part of it is applied ahead, as a power of two.
    const double whole = clips ? max_norm / (total + eps) : 1.0;
    const float pre = whole < 0x1p-100 ? 0x1p-100f : 1.0f;
    const float s = static_cast<float>(whole < 0x1p-100 ? whole * 0x1p100 : whole);
    for (int i = blockIdx.x; i < l.chunks; i += gridDim.x) {
        const int c = l.chunks - 1 - i;
        const Tensor &t = l.t[tensor_of(l, c)];
        if (!clips && t.in == t.out) continue;
        const int64_t at = static_cast<int64_t>(c - t.chunk0) * l.chunk;
        const int n = static_cast<int>(min(static_cast<int64_t>(l.chunk), t.n - at));
        if (!clips) {
            if (t.bf16) copy_chunk(static_cast<const uint16_t *>(t.in) + at, static_cast<uint16_t *>(t.out) + at, n);
            else copy_chunk(static_cast<const uint32_t *>(t.in) + at, static_cast<uint32_t *>(t.out) + at, n);
            continue;
        }
        if (t.bf16) scale_chunk(static_cast<const __nv_bfloat16 *>(t.in) + at, static_cast<__nv_bfloat16 *>(t.out) + at, n, pre, s);
        else scale_chunk(static_cast<const float *>(t.in) + at, static_cast<float *>(t.out) + at, n, pre, s);
    }
}

__global__ void __launch_bounds__(kThreads) finish_kernel(const double *partial, int n_partial, float *norm) {
    __shared__ double shared[kThreads / 32];
    const double total = total_of(partial, n_partial, shared);
    if (threadIdx.x == 0) *norm = static_cast<float>(sqrt(total));
}

// Calls body(list, first) for every launch's worth of tensors.
template <int kCap, class Body>
moe_status for_lists(const GradList &g, int blocks, const Body &body) {
    int64_t all = 0;
    for (int i = 0; i < g.n; ++i) all += g.sizes[i];
    // Chunks small enough to spread over the blocks, large enough to stream.
    int chunk = 2048;
    while (chunk < 16384 && all / chunk > 4ll * blocks) chunk *= 2;
    List<kCap> l;
    for (int i = 0; i < g.n;) {
        const int first = i;
        l.count = 0;
        int64_t chunks = 0;
        l.chunk = chunk;
        for (; i < g.n && l.count < kCap; ++i) {
            if (g.sizes[i] == 0) continue;
            const int64_t c = (g.sizes[i] + chunk - 1) / chunk;
            if (chunks + c > INT32_MAX / 2) {
                if (l.count == 0) return MOE_ERR_CAPACITY;
                break;
            }
            l.t[l.count++] = {g.in[i], g.out ? g.out[i] : nullptr, g.sizes[i], static_cast<int32_t>(chunks),
                              g.dtypes[i] == MOE_BF16};
            chunks += c;
        }
        l.chunks = static_cast<int>(chunks);
        const moe_status st = body(l, first == 0);
        if (st != MOE_OK) return st;
    }
    return MOE_OK;
}

template <int kCap>
moe_status run(const GradList &g, cudaStream_t stream, int num_sms, int *launches) {
    const int blocks = num_sms * kBlocksPerSm;
    double *partial = static_cast<double *>(g.partial);
    moe_status st = for_lists<kCap>(g, blocks, [&](const List<kCap> &l, bool first) {
        norm_kernel<kCap><<<blocks, kThreads, 0, stream>>>(l, partial, !first);
        ++*launches;
        return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    });
    if (st != MOE_OK) return st;
    if (!g.out) {
        finish_kernel<<<1, kThreads, 0, stream>>>(partial, blocks, g.norm);
        ++*launches;
        return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    }
    return for_lists<kCap>(g, blocks, [&](const List<kCap> &l, bool first) {
        scale_kernel<kCap><<<blocks, kThreads, 0, stream>>>(l, partial, blocks, g.max_norm, g.eps, first ? g.norm : nullptr);
        ++*launches;
        return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    });
}

struct Span {
    uintptr_t from, to;
    bool written;
};

}  // namespace clip

size_t grad_partial_bytes(int num_sms) { return static_cast<size_t>(num_sms) * clip::kBlocksPerSm * sizeof(double); }

// Whether no output overlaps another tensor: neighbours in address order are enough once
// the furthest end so far is kept.
moe_status check_grad_spans(const GradList &g) {
    if (!g.out) return MOE_OK;
    bool sorted = true, in_place = true;
    uintptr_t end = 0;
    for (int i = 0; i < g.n; ++i) {
        if (g.sizes[i] == 0) continue;
        const uintptr_t a = reinterpret_cast<uintptr_t>(g.out[i]);
        in_place = in_place && g.out[i] == g.in[i];
        sorted = sorted && a >= end;
        end = a + static_cast<uintptr_t>(g.sizes[i]) * (g.dtypes[i] == MOE_BF16 ? 2 : 4);
    }
    if (sorted && in_place) return MOE_OK;
    clip::Span *s = new (std::nothrow) clip::Span[2 * static_cast<size_t>(g.n)];
    if (!s) return MOE_ERR_CAPACITY;
    size_t n = 0;
    for (int i = 0; i < g.n; ++i) {
        if (g.sizes[i] == 0) continue;
        const uintptr_t bytes = static_cast<uintptr_t>(g.sizes[i]) * (g.dtypes[i] == MOE_BF16 ? 2 : 4);
        const uintptr_t a = reinterpret_cast<uintptr_t>(g.in[i]), o = reinterpret_cast<uintptr_t>(g.out[i]);
        s[n++] = {o, o + bytes, true};
        if (a != o) s[n++] = {a, a + bytes, false};
    }
    std::sort(s, s + n, [](const clip::Span &a, const clip::Span &b) { return a.from < b.from; });
    uintptr_t any = 0, written = 0;
    bool ok = true;
    for (size_t i = 0; i < n; ++i) {
        if (s[i].from < (s[i].written ? any : written)) ok = false;
        any = std::max(any, s[i].to);
        if (s[i].written) written = std::max(written, s[i].to);
    }
    delete[] s;
    return ok ? MOE_OK : MOE_ERR_INVALID_ARG;
}

moe_status launch_grad_clip(const GradList &g, cudaStream_t stream, int num_sms, int *launches) {
    *launches = 0;
    bool empty = true;
    for (int i = 0; i < g.n && empty; ++i) empty = g.sizes[i] == 0;
    if (empty) {
        if (cudaMemsetAsync(g.norm, 0, sizeof(float), stream) != cudaSuccess) return MOE_ERR_CUDA;
        return MOE_OK;
    }
    // A short list's parameters are a few hundred bytes, a long one's 20 KB.
    return g.n <= 16 ? clip::run<16>(g, stream, num_sms, launches) : clip::run<640>(g, stream, num_sms, launches);
}

}  // namespace moe
