// Global norm of a list of gradient tensors, and clipping by it:
//
//   norm = sqrt(sum over all tensors of x^2),   out = x * min(1, max_norm / (norm + eps))
//
//  * Two kernels.  The first leaves one sum a block; every block of the second adds those
//    up again in the same order, so no counter or atomic decides an order and nothing has
//    to be cleared between calls.
//  * The tensors' addresses travel in the kernel's parameters, kCap a launch (longer lists
//    take several launches); a chunk of work finds its tensor by bisection.
//  * f64 additions are slow here (about two a cycle and SM): a thread adds the squares of the
//    elements that it loads together in f32, and those sums in an f32 pair (the sum and what
//    its roundings left out, by Knuth's two-sum); the block joins its pairs and only the
//    block's sum is f64.  A group of squares outside 2^-90 .. 2^80, where f32 would lose some
//    of them or the sums overflow, is formed again from scaled elements and travels beside the
//    pairs, in f64: the norm is right over the whole range of the types.
//  * Bound by HBM: one read for the norm and a read and a write for the clipping.  The
//    second kernel goes through the chunks backwards, so what the first read last (the L2's
//    share) is not fetched again.  1.3 GB in 120 tensors: 619 us, 6.3 TB/s of the three passes
//    (the norm alone 6.7); 0.8 M elements in 10 tensors: 8.8 us for the two launches.
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

constexpr int kThreads = 512;
constexpr int kBlocksPerSm = 3;           // few: every block of the second kernel adds up all sums
constexpr int kVecs = 4;                  // 16-byte loads a thread has in flight
constexpr int kMinChunk = 4096, kMaxChunk = 32768;

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

// A sum and what its roundings left out.
struct Pair {
    float hi, lo;
};

__device__ __forceinline__ void add(Pair &a, float b) {
    const float s = a.hi + b, t = s - a.hi;
    a.lo += (a.hi - (s - t)) + (b - t);
    a.hi = s;
}

// f32 sums in this range hold their squares to f32 accuracy (what underflows, under 2^-126
// each, is below 2^-30 of it), and 2^40 of them fit f32.
__device__ __forceinline__ bool sum_holds(float s) { return s > 0x1p-90f && s < 0x1p80f; }

template <int V>
__device__ __forceinline__ float squares(const float (&v)[V]) {
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int i = 0; i < V; i += 2) {
        a = fmaf(v[i], v[i], a);
        b = fmaf(v[i + 1], v[i + 1], b);
    }
    return a + b;
}

// The squares of n vectors, kThreads vectors apart, whatever their magnitude: of the elements
// times a power of two that brings the largest to 1 (or 4), in f32 as above, and back in the
// exponent of a double, by integers.
template <typename T>
__device__ __forceinline__ double scaled_squares(const T *p, int n) {
    constexpr int V = 16 / sizeof(T);
    uint32_t most = 0;
    for (int i = 0; i < n; ++i) {
        float x[V];
        load_row<V>(p + i * kThreads * V, x);
#pragma unroll
        for (int j = 0; j < V; ++j) most = max(most, __float_as_uint(x[j]) & 0x7FFFFFFFu);
    }
    if (most == 0) return 0.0;
    if (most >= 0x7F800000u) return __uint_as_float(most);           // an infinity or a NaN
    const int e = min(max(static_cast<int>(most >> 23), 1), 253);
    const float f = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
    float s = 0.f;
    for (int i = 0; i < n; ++i) {
        float x[V];
        load_row<V>(p + i * kThreads * V, x);
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] *= f;
        s += squares(x);
    }
    // s is in 2^-46 .. 2^9 (the largest element may be subnormal): a normal number
    const uint64_t b = __float_as_uint(s);
    return __longlong_as_double(static_cast<int64_t>((b << 29) + (static_cast<uint64_t>(1023 - 127 + 2 * (e - 127)) << 52)));
}

// A thread's groups of a chunk that f32 does not hold, a bit each.  Read again behind the chunk
// rather than kept in registers or worked out on the spot, either of which spills in the loop that
// every gradient goes through (1 GB in bf16 150 -> 197 us, in f32 150 -> 170).  Zeros and small
// elements are ordinary in gradients; element by element in f64 they took 13 times as long as
// others in bf16 and 7 times in f32.
template <typename T>
__device__ __noinline__ double far_squares(const T *q, int vecs, uint32_t groups) {
    constexpr int V = 16 / sizeof(T);
    double far = 0.0;
    for (int v = threadIdx.x; groups; groups >>= 1) {
        const int count = v + (kVecs - 1) * kThreads < vecs ? kVecs : 1;
        if (groups & 1) {
            const double d = scaled_squares(q + static_cast<int64_t>(v) * V, count);
            if (__double_as_longlong(d) != 0) far += d;
        }
        v += count * kThreads;
    }
    return far;
}

struct Sums {
    Pair near;
    double far;
};

// Elements of [p, p + n) before the first 16-byte address.
template <typename T>
__device__ __forceinline__ int head_of(const T *p, int n) {
    return min(n, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / static_cast<int>(sizeof(T)));
}

template <typename T>
__device__ __forceinline__ void chunk_squares(const T *p, int n, Sums &sums) {
    constexpr int V = 16 / sizeof(T);
    const int tid = threadIdx.x;
    const int head = head_of(p, n), vecs = (n - head) / V, tail = head + vecs * V;
    const T *q = p + head;
    uint32_t far = 0, bit = 1;                // at most kMaxChunk / (4 kThreads kVecs) + kVecs - 1 groups
    const auto take = [&](float s) {
        if (sum_holds(s)) add(sums.near, s);
        else far |= bit;
        bit <<= 1;
    };
    int v = tid;
    for (; v + (kVecs - 1) * kThreads < vecs; v += kVecs * kThreads) {
        float x[kVecs][V];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) load_row<V>(q + static_cast<int64_t>(v + i * kThreads) * V, x[i]);
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kVecs; i += 2) s += squares(x[i]) + squares(x[i + 1]);
        take(s);
    }
    for (; v < vecs; v += kThreads) {
        float x[V];
        load_row<V>(q + static_cast<int64_t>(v) * V, x);
        take(squares(x));
    }
    if (far) sums.far += far_squares(q, vecs, far);
    // Up to V - 1 elements before and behind the vectors.
    const int at = tid < head ? tid : tail + tid - head;
    if (at < n) {
        const float x = as_f32(p[at]), s = x * x;
        if (sum_holds(s)) add(sums.near, s);
        else sums.far = fma(static_cast<double>(x), static_cast<double>(x), sums.far);
    }
}

// The sum of n doubles, in lane 0 of the warp that asks: the same in every block.
__device__ __forceinline__ double total_of(const double *partial, int n) {
    double d = 0.0;
    for (int i = threadIdx.x & 31; i < n; i += 32) d += __ldcg(partial + i);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) d += __shfl_xor_sync(0xffffffffu, d, m);
    return d;
}

template <int kCap>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    norm_kernel(const __grid_constant__ List<kCap> l, double *partial, int add_to) {
    __shared__ Pair pairs[kThreads / 32];
    __shared__ double far[kThreads / 32];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    Sums sums = {};
    for (int c = blockIdx.x; c < l.chunks; c += gridDim.x) {
        const Tensor &t = l.t[tensor_of(l, c)];
        const int64_t at = static_cast<int64_t>(c - t.chunk0) * l.chunk;
        const int n = static_cast<int>(min(static_cast<int64_t>(l.chunk), t.n - at));
        if (t.bf16) chunk_squares(static_cast<const __nv_bfloat16 *>(t.in) + at, n, sums);
        else chunk_squares(static_cast<const float *>(t.in) + at, n, sums);
    }
    const auto join = [](Pair &a, int m) {
        const float hi = __shfl_xor_sync(0xffffffffu, a.hi, m), lo = __shfl_xor_sync(0xffffffffu, a.lo, m);
        add(a, hi);
        a.lo += lo;
    };
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) join(sums.near, m);
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) pairs[warp] = sums.near;
    const bool any_far = __syncthreads_or(sums.far != 0.0);       // a NaN is not 0
    if (any_far) {
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) sums.far += __shfl_xor_sync(0xffffffffu, sums.far, m);
        if ((threadIdx.x & 31) == 0) far[warp] = sums.far;
        __syncthreads();
    }
    if (threadIdx.x < 32) {
        Pair a = threadIdx.x < kThreads / 32 ? pairs[threadIdx.x] : Pair{0.f, 0.f};
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) join(a, m);
        if (threadIdx.x == 0) {
            double d = static_cast<double>(a.hi) + a.lo;
            for (int w = 0; any_far && w < kThreads / 32; ++w) d += far[w];
            partial[blockIdx.x] = add_to ? partial[blockIdx.x] + d : d;
        }
    }
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
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) scale_kernel(const __grid_constant__ List<kCap> l, const double *partial,
                                                         int n_partial, double max_norm, double eps, float *norm) {
    __shared__ struct {
        int clips;
        float pre, s;
    } shared;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (threadIdx.x < 32) {
        const double sum = total_of(partial, n_partial);
        if (threadIdx.x == 0) {       // one thread: a root and a quotient in f64 by all took 20 us
            const double total = sqrt(sum);
            if (blockIdx.x == 0 && norm) *norm = static_cast<float>(total);
            // An infinite or NaN sum clips nothing: the gradients are left (or copied) as they are.  A sum of
            // finite ones is finite in f64, past f32's range too.
            const bool clips = total < __longlong_as_double(0x7FF0000000000000ll) && max_norm < total + eps;
            // A scale near or below f32's smallest normal number (a norm past 2^100) would lose
            // bits: part of it is applied ahead, as a power of two.
            const double whole = clips ? max_norm / (total + eps) : 1.0;
            shared.clips = clips;
            shared.pre = whole < 0x1p-100 ? 0x1p-100f : 1.0f;
            shared.s = static_cast<float>(whole < 0x1p-100 ? whole * 0x1p100 : whole);
        }
    }
    __syncthreads();
    const bool clips = shared.clips;
    const float pre = shared.pre, s = shared.s;
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

__global__ void __launch_bounds__(32) finish_kernel(const double *partial, int n_partial, float *norm) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const double total = total_of(partial, n_partial);
    if (threadIdx.x == 0) *norm = static_cast<float>(sqrt(total));
}

// Elements a chunk: small enough to spread over the blocks, large enough to stream.  And no more
// blocks than chunks: each leaves a sum that every block of the second kernel reads.
int chunk_size(const GradList &g, int *blocks) {
    int64_t all = 0, chunks = 0;
    for (int i = 0; i < g.n; ++i) all += g.sizes[i];
    int chunk = kMinChunk;
    while (chunk < kMaxChunk && all / chunk > 4ll * *blocks) chunk *= 2;
    for (int i = 0; i < g.n && chunks < *blocks; ++i) chunks += (g.sizes[i] + chunk - 1) / chunk;
    if (chunks < *blocks) *blocks = static_cast<int>(chunks);
    return chunk;
}

// Calls body(list, first) for every launch's worth of tensors.
template <int kCap, class Body>
moe_status for_lists(const GradList &g, int chunk, const Body &body) {
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

// A launch that may start under the end of the one before.
template <class... Args>
moe_status launch_after(void (*kernel)(Args...), int blocks, int threads, bool chained, cudaStream_t stream, const Args &...args) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = chained ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <int kCap>
moe_status run(const GradList &g, cudaStream_t stream, int num_sms, int *launches) {
    int blocks = num_sms * kBlocksPerSm;
    const int chunk = chunk_size(g, &blocks);
    double *partial = static_cast<double *>(g.partial);
    moe_status st = for_lists<kCap>(g, chunk, [&](const List<kCap> &l, bool first) {
        ++*launches;
        return launch_after(norm_kernel<kCap>, blocks, kThreads, false, stream, l, partial, static_cast<int>(!first));
    });
    if (st != MOE_OK) return st;
    const double *sums = partial;
    if (!g.out) {
        ++*launches;
        return launch_after(finish_kernel, 1, 32, true, stream, sums, blocks, g.norm);
    }
    // The first scaling launch follows a norm launch and may start under its end; in place it
    // writes what that read, but only behind its wait.
    return for_lists<kCap>(g, chunk, [&](const List<kCap> &l, bool first) {
        ++*launches;
        return launch_after(scale_kernel<kCap>, blocks, kThreads, first, stream, l, sums, blocks, g.max_norm, g.eps,
                            first ? g.norm : static_cast<float *>(nullptr));
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
