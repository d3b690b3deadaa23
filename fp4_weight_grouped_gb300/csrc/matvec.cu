// Products of a few rows with weight matrices that each row chooses:
//
//   out[r, n] = sum_k x[r / div, k] * w[e_r, n, k]          (SwiGLU: rows n and I + n)
//
// w in 4 bits (MXFP4: e2m1 * 2^(s - 127) per 32 k; NVFP4: e2m1 * e4m3 per 16 k, times
// an f32 an expert) or bf16.  For one to a few dozen rows: no sort, no row bands.
//
//  * Rows of the same expert are taken together, up to 8 at a time (a chunk), so a
//    weight is read once for them.  Every CTA works the chunks out from the ids itself.
//  * A tile is 16 weight rows (SwiGLU: 8 gate and the 8 matching up rows, so that one
//    thread finds both).  The warps of a CTA share the tile's K, 128 k (bf16: 32) a
//    stage, and add up their sums in shared memory in a fixed order.
//  * mma.sync m16n8k16 with the weights as A and the chunk's rows as B columns: eight
//    rows cost what one costs, and a thread's four sums are f32.  Tensor memory has
//    nothing to offer here: no operand is used twice.
//  * 4-bit weights become f16 by cvt (exact), so x has to be f16 as well: each row is
//    scaled by a power of two that brings its largest magnitude to [2^14, 2^15).  A bf16
//    has 8 bits, f16 spans 2^-24 .. 2^15: elements down to 2^-28 of the row's largest are
//    exact, smaller ones are off by at most 2^-39 of it.
//  * MXFP4: the scale is the same for the 32 k of two MMAs, whose sums it multiplies in
//    f32.  It is kept 2^-31 low until the end, which keeps the sums of scaled rows (up to
//    2^15 * 6 * 32 a block, 1,024 blocks) below 2^127 for every scale that the format has;
//    scales below 2^-118 underflow to 0 for it.
//    NVFP4: e2m1 * e4m3 has 6 bits and fits f16, so the scale goes into the weight.
//  * Each warp fetches its own stages with cp.async, kDepth ahead, across tiles: no
//    barriers to wait for and nothing to hang on.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "device_common.cuh"
#include "launch.h"

namespace moe {
namespace mv {

enum Format { kMx, kNv, kBf16 };

constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kTok = 8;                       // rows a chunk at most (the MMA's n)
constexpr int kRowBytes = 64;                 // of a weight row in a stage
constexpr int kTileFloats = 16 * kTok;        // sums of a tile

template <int F>
struct Fmt {
    static constexpr int kUnit = F == kBf16 ? 32 : 128;             // k of a stage
    // A row in a stage: MXFP4 is read by words, the others by 16 bytes; both free of conflicts.
    static constexpr int kPitch = F == kMx ? 80 : 64;
    static constexpr int kScaleWords = F == kMx ? 2 : F == kNv ? 3 : 0;   // a row, any alignment
    static constexpr int kStage = 16 * kPitch + 64 * kScaleWords;
    static constexpr int kDepth = F == kBf16 ? 8 : 6;
};

struct Params {
    const uint16_t *x;
    int64_t x_stride;
    int div;
    const int32_t *row_expert;    // null: expert 0
    int rows, K, E, N;            // N output columns
    const uint8_t *w, *scales;
    const float *ws2;
    void *out;
    int out_bf16;
    int *status;
    int tok;                      // rows a chunk, 1..kTok
    int k_pad;                    // K up to a stage
    int x_vec;                    // x rows at 16-byte addresses
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool real) {
    const int n = real ? 16 : 0;
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

template <bool kHalf>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    if constexpr (kHalf)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight e2m1 codes to f16 pairs: (0, 1), (2, 3), (4, 5), (6, 7).
__device__ __forceinline__ void decode8(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// Two e4m3 bytes as f16, each twice.
__device__ __forceinline__ void e4m3_pairs(uint32_t b, uint32_t &first, uint32_t &second) {
    uint32_t h;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h) : "r"(b));
    first = prmt(h, h, 0x1010u);
    second = prmt(h, h, 0x3232u);
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// The chunks of a call, worked out by every CTA: `order` holds the slots (rows with a valid
// expert) sorted by expert, chunk c is order[first[c] .. first[c + 1]) with one expert.
struct Chunks {
    int *order, *first, *expert;      // [rows], [rows + 1], [rows]
    int *scratch;                     // [rows]: expert of every slot
    int *count;
};

__device__ __forceinline__ void build_chunks(const Params &p, const Chunks &c) {
    const int tid = threadIdx.x;
    if (!p.row_expert) {
        const int n = (p.rows + p.tok - 1) / p.tok;
        for (int s = tid; s < p.rows; s += kThreads) c.order[s] = s;
        for (int i = tid; i <= n; i += kThreads) {
            c.first[i] = min(i * p.tok, p.rows);
            if (i < n) c.expert[i] = 0;
        }
        if (tid == 0) *c.count = n;
        __syncthreads();
        return;
    }
    if (p.rows <= 32) {               // one warp: the slots' experts in its lanes
        if (tid < 32) {
            int e = INT32_MAX;
            if (tid < p.rows) {
                e = __ldg(p.row_expert + tid);
                if (static_cast<unsigned>(e) >= static_cast<unsigned>(p.E)) e = INT32_MAX;
                c.scratch[tid] = e;
            }
            int before = 0, same = 0;
            for (int q = 0; q < p.rows; ++q) {
                const int f = __shfl_sync(0xffffffffu, e, q);
                same += f == e && q < tid;
                before += f < e;
            }
            const bool real = e != INT32_MAX;
            const int at = before + same;                              // a permutation of the valid slots
            const bool head = real && same % p.tok == 0;
            int n = 0;                                                 // chunks that start ahead of this one
            for (int q = 0; q < p.rows; ++q) {
                const int qa = __shfl_sync(0xffffffffu, head ? at : INT32_MAX, q);
                n += qa < at;
            }
            if (real) c.order[at] = tid;
            if (head) {
                c.first[n] = at;
                c.expert[n] = e;
            }
            const int chunks = __popc(__ballot_sync(0xffffffffu, head));
            const int valid = __popc(__ballot_sync(0xffffffffu, real));
            if (tid == 0) {
                *c.count = chunks;
                c.first[chunks] = valid;
            }
        }
        __syncthreads();
        return;
    }
    if (tid == 0) *c.count = 0;
    for (int s = tid; s < p.rows; s += kThreads) {
        const int e = __ldg(p.row_expert + s);
        c.scratch[s] = static_cast<unsigned>(e) < static_cast<unsigned>(p.E) ? e : INT32_MAX;
    }
    __syncthreads();
    for (int s = tid; s < p.rows; s += kThreads) {
        const int e = c.scratch[s];
        if (e == INT32_MAX) continue;
        int before = 0, same = 0;     // slots ahead of this one, and those of its expert among them
        for (int q = 0; q < p.rows; ++q) {
            const int f = c.scratch[q];
            same += f == e && q < s;
            before += f < e;
        }
        c.order[before + same] = same % p.tok == 0 ? ~s : s;       // a chunk starts here
    }
    __syncthreads();
    int valid = 0;
    for (int q = 0; q < p.rows; ++q) valid += c.scratch[q] != INT32_MAX;
    for (int i = tid; i < valid; i += kThreads) {
        const int v = c.order[i];
        if (v >= 0) continue;
        int n = 0;
        for (int q = 0; q < i; ++q) n += c.order[q] < 0;
        c.first[n] = i;
        c.expert[n] = c.scratch[~v];
        atomicAdd(c.count, 1);
    }
    __syncthreads();
    for (int i = tid; i < valid; i += kThreads)
        if (c.order[i] < 0) c.order[i] = ~c.order[i];
    if (tid == 0) c.first[*c.count] = valid;
    __syncthreads();
}

// The chunk's rows of x into shared memory (f16, scaled by 2^-e; bf16 as they are), zeros up
// to k_pad.  exps[t] receives e.  Everyone is past its last use of x when this is called.
// NVFP4: within 128 k, 16 bytes q go to place 4 (q % 4) + q / 4, where the lanes that hold
// 32 k each find theirs side by side.
template <int F>
__device__ __forceinline__ void stage_x(const Params &p, const int *slots, int n, uint8_t *xs, int pitch, int *exps) {
    const int tid = threadIdx.x, vecs = p.k_pad / 8;
    const auto load = [&](const uint16_t *row, int v) {
        uint4 a = make_uint4(0, 0, 0, 0);
        if (8 * v < p.K) {            // K is a multiple of 8
            if (p.x_vec) {
                a = __ldg(reinterpret_cast<const uint4 *>(row) + v);
            } else {
                const uint16_t *q = row + 8 * v;
                a.x = __ldg(q) | static_cast<uint32_t>(__ldg(q + 1)) << 16;
                a.y = __ldg(q + 2) | static_cast<uint32_t>(__ldg(q + 3)) << 16;
                a.z = __ldg(q + 4) | static_cast<uint32_t>(__ldg(q + 5)) << 16;
                a.w = __ldg(q + 6) | static_cast<uint32_t>(__ldg(q + 7)) << 16;
            }
        }
        return a;
    };
    if constexpr (F == kBf16) {
        for (int t = 0; t < n; ++t) {
            const uint16_t *row = p.x + (slots[t] / p.div) * p.x_stride;
            for (int v = tid; v < vecs; v += kThreads)
                *reinterpret_cast<uint4 *>(xs + t * pitch + 16 * v) = load(row, v);
        }
        __syncthreads();
        return;
    } else {
        if (tid < kTok) exps[tid] = 0;
        __syncthreads();
        // Largest finite magnitude of every row, by its exponent field.
        for (int t = 0; t < n; ++t) {
            const uint16_t *row = p.x + (slots[t] / p.div) * p.x_stride;
            uint32_t top = 0;
            for (int v = tid; v < vecs; v += kThreads) {
                const uint4 a = load(row, v);
                const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t lo = w[i] & 0x7F80u, hi = w[i] >> 16 & 0x7F80u;
                    top = max(top, lo == 0x7F80u ? 0u : lo);
                    top = max(top, hi == 0x7F80u ? 0u : hi);
                }
            }
            top = __reduce_max_sync(0xffffffffu, top);
            if ((tid & 31) == 0) atomicMax(&exps[t], static_cast<int>(top >> 7));
        }
        __syncthreads();
        for (int t = 0; t < n; ++t) {
            const uint16_t *row = p.x + (slots[t] / p.div) * p.x_stride;
            const int e = max(exps[t] - 127 - 14, -126);
            const float f = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
            for (int v = tid; v < vecs; v += kThreads) {
                const uint4 a = load(row, v);
                const uint32_t w[4] = {a.x, a.y, a.z, a.w};
                uint32_t o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    asm("cvt.rn.f16x2.f32 %0, %1, %2;"
                        : "=r"(o[i])
                        : "f"(__uint_as_float(w[i] & 0xFFFF0000u) * f), "f"(__uint_as_float(w[i] << 16) * f));
                const int at = F == kNv ? (v & ~15) | (v & 3) << 2 | (v >> 2 & 3) : v;
                *reinterpret_cast<uint4 *>(xs + t * pitch + 16 * at) = make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
        __syncthreads();
        // Only now: every thread has read the field above.
        if (tid < n) exps[tid] = max(exps[tid] - 127 - 14, -126);
        __syncthreads();
    }
}

// How many warps share a tile's K: a tile's sums are joined across them behind a barrier, so
// few is better, but the CTAs' shares come in items of kWarps / kw tiles.  In units of a
// stage's time; an item's end costs about two.
__device__ __forceinline__ int choose_kw(uint32_t tiles, uint32_t units) {
    uint32_t best = 1, cost = UINT32_MAX;
    for (uint32_t kw = 1; kw <= kWarps; kw *= 2) {
        const uint32_t items = (tiles * kw + kWarps - 1) / kWarps;
        const uint32_t c = (items + gridDim.x - 1) / gridDim.x * ((units + kw - 1) / kw + 2);
        if (c < cost) {
            cost = c;
            best = kw;
        }
    }
    return best;
}

// One stage (128 k; bf16: 32) of 16 weight rows: acc += w x.
template <int F, bool kShift>
__device__ __forceinline__ void multiply(uint32_t at, uint32_t xa, bool has_x, int blocks, int g, int t4,
                                         const uint32_t (&off)[2], float (&acc)[4], uint32_t (&bad)[2]) {
    using C = Fmt<F>;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    if constexpr (F == kBf16) {
        const uint4 a = lds128(at + g * C::kPitch + t4 * 16), c = lds128(at + (g + 8) * C::kPitch + t4 * 16);
        const uint4 v = has_x ? lds128(xa) : zero;
        mma16816<false>(acc, a.x, c.x, a.y, c.y, v.x, v.y);
        mma16816<false>(acc, a.z, c.z, a.w, c.w, v.z, v.w);
    } else if constexpr (F == kNv) {
        // Lane t4 holds the 32 k of block t4, two scales a row.
        const uint4 ra = lds128(at + g * C::kPitch + 16 * t4), rc = lds128(at + (g + 8) * C::kPitch + 16 * t4);
        uint4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = has_x ? lds128(xa + 64 * j) : zero;
        uint32_t b[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const uint32_t sa = at + 16 * C::kPitch + (g + 8 * r) * 4 * C::kScaleWords + 2 * t4;
            b[r] = kShift ? lds8(sa + off[r]) | lds8(sa + off[r] + 1) << 8 : lds16(sa);
            if (t4 >= blocks) b[r] = 0;               // past the row's end
        }
        bad[0] |= (((b[0] | b[1] << 16) & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;     // NaN
        uint32_t s[2][2];
        e4m3_pairs(b[0], s[0][0], s[0][1]);
        e4m3_pairs(b[1], s[1][0], s[1][1]);
        const uint32_t wa[4] = {ra.x, ra.y, ra.z, ra.w}, wc[4] = {rc.x, rc.y, rc.z, rc.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t a[4], c[4];
            decode8(wa[j], a);
            decode8(wc[j], c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = hmul2(a[i], s[0][j >> 1]);
                c[i] = hmul2(c[i], s[1][j >> 1]);
            }
            mma16816<true>(acc, a[0], c[0], a[1], c[1], v[j].x, v[j].y);
            mma16816<true>(acc, a[2], c[2], a[3], c[3], v[j].z, v[j].w);
        }
    } else {
        uint32_t wa[4], wc[4], sw[2];
        uint4 v[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            wa[b] = lds32(at + g * C::kPitch + 16 * b + 4 * t4);
            wc[b] = lds32(at + (g + 8) * C::kPitch + 16 * b + 4 * t4);
            v[b] = has_x ? lds128(xa + 64 * b) : zero;
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const uint32_t sa = at + 16 * C::kPitch + (g + 8 * r) * 4 * C::kScaleWords;
            sw[r] = kShift ? __funnelshift_r(lds32(sa), lds32(sa + 4), 8 * off[r]) : lds32(sa);
            if (blocks < 4) sw[r] &= (1u << (8 * blocks)) - 1;                            // past the row's end
            bad[r] |= ((sw[r] & 0x7F7F7F7Fu) + 0x03030303u) & sw[r] & 0x80808080u;        // 253 and more
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            uint32_t a[4], c[4];
            decode8(wa[b], a);
            decode8(wc[b], c);
            float d[4] = {0.f, 0.f, 0.f, 0.f};
            mma16816<true>(d, a[0], c[0], a[1], c[1], v[b].x, v[b].y);
            mma16816<true>(d, a[2], c[2], a[3], c[3], v[b].z, v[b].w);
            const float s0 = __uint_as_float((sw[0] >> (8 * b) & 0xFFu) << 23) * 0x1p-31f;
            const float s1 = __uint_as_float((sw[1] >> (8 * b) & 0xFFu) << 23) * 0x1p-31f;
            acc[0] = fmaf(s0, d[0], acc[0]);
            acc[1] = fmaf(s0, d[1], acc[1]);
            acc[2] = fmaf(s1, d[2], acc[2]);
            acc[3] = fmaf(s1, d[3], acc[3]);
        }
    }
}

template <int F, bool kSwiglu, bool kShift>
__global__ void __launch_bounds__(kThreads, 1) matvec_kernel(const Params p) {
    using C = Fmt<F>;
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t4 = lane & 3;
    const int pitch = p.k_pad * 2 + 64;
    // ring | sums | x | chunk tables
    uint8_t *ring = smem + warp * C::kDepth * C::kStage;
    float *sums = reinterpret_cast<float *>(smem + kWarps * C::kDepth * C::kStage);
    uint8_t *xs = reinterpret_cast<uint8_t *>(sums + 2 * kWarps * kTileFloats);
    int *tab = reinterpret_cast<int *>(xs + p.tok * pitch);
    const Chunks ch = {tab + kTok + 1, tab + kTok + 1 + p.rows, tab + kTok + 2 + 2 * p.rows,
                       tab + kTok + 2 + 3 * p.rows, tab + kTok};
    int *exps = tab;
    build_chunks(p, ch);

    constexpr int kTileCols = kSwiglu ? 8 : 16;
    const int tiles = (p.N + kTileCols - 1) / kTileCols;
    const int units = (p.K + C::kUnit - 1) / C::kUnit;
    const int n_chunks = *ch.count;
    const int kw = choose_kw(n_chunks * tiles, units), group = kWarps / kw;
    const int groups = (tiles + group - 1) / group;          // items a chunk
    // The CTA's share of the items, one after another.  (rows * N < 2^31, so counts fit.)
    const int total = n_chunks * groups, grid = gridDim.x, blk = blockIdx.x;
    const int first = total / grid * blk + min(blk, total % grid);
    const int count = total / grid + (blk < total % grid);
    const int wk = warp % kw, wt = warp / kw;
    const int u0 = units * wk / kw, u1 = units * (wk + 1) / kw;
    const int64_t w_pitch = F == kBf16 ? 2ll * p.K : p.K / 2;
    const int64_t s_pitch = F == kMx ? p.K / 32 : p.K / 16;
    const int64_t w_rows = kSwiglu ? 2ll * p.N : p.N;
    const int row_bytes = static_cast<int>(w_pitch), scale_bytes = static_cast<int>(s_pitch);

    // Weight row r of this warp's tile; columns past the last read the last one's.
    const auto weight_row = [&](int chunk, int grp, int r) {
        const int tile = grp * group + wt;
        const int n = kSwiglu ? min(tile * 8 + (r & 7), p.N - 1) + (r >= 8 ? p.N : 0) : min(tile * 16 + r, p.N - 1);
        return ch.expert[chunk] * w_rows + n;
    };
    // A stage: lane copies 32 bytes of row lane / 2; lanes 0..15 the scale words of row lane.
    const uint32_t ring_a = smem_u32(ring);
    const uint32_t dst0 = ring_a + (lane >> 1) * C::kPitch + (lane & 1) * 32;
    const uint32_t sdst0 = ring_a + 16 * C::kPitch + (lane & 15) * 4 * C::kScaleWords;
    constexpr int kScaleBytes = F == kMx ? 4 : 8;
    const uint8_t *wp = nullptr, *sp = nullptr;
    int f_left = u0 < u1 ? count : 0, f_unit = u0, f_chunk = n_chunks ? first / groups : 0;
    int f_grp = n_chunks ? first % groups : 0;
    const auto fetch_next = [&](int slot) {
        if (f_left > 0) {
            if (f_unit == u0) {
                wp = p.w + weight_row(f_chunk, f_grp, lane >> 1) * w_pitch + (lane & 1) * 32;
                if constexpr (F != kBf16) sp = p.scales + weight_row(f_chunk, f_grp, lane & 15) * s_pitch;
            }
            const int at = f_unit * kRowBytes;
            const uint32_t d = dst0 + slot * C::kStage;
            // A piece past the row's end becomes zeros; its address is not read.
            const int have = row_bytes - at - (lane & 1) * 32;
            cp_async16(d, wp + (have > 0 ? at : 0), have > 0);
            cp_async16(d + 16, wp + (have > 16 ? at + 16 : 0), have > 16);
            if constexpr (F != kBf16) {
                if (lane < 16) {
                    const uint32_t sd = sdst0 + slot * C::kStage;
                    const uint8_t *src = sp + f_unit * kScaleBytes;
                    const int bytes = min(scale_bytes - f_unit * kScaleBytes, kScaleBytes);     // of the row here
                    const int off = kShift ? static_cast<int>(reinterpret_cast<uintptr_t>(src) & 3) : 0;
#pragma unroll
                    for (int i = 0; i < (kShift ? C::kScaleWords : C::kScaleWords - 1); ++i)
                        if (4 * i < off + bytes) cp_async4(sd + 4 * i, src - off + 4 * i);      // words that hold one
                }
            }
            if (++f_unit == u1) {
                f_unit = u0;
                --f_left;
                if (++f_grp == groups) {
                    f_grp = 0;
                    ++f_chunk;
                }
            }
        }
        cp_commit();
    };
#pragma unroll 1
    for (int i = 0; i < C::kDepth - 1; ++i) fetch_next(i);

    // Weights and ids do not depend on the launch before (a chain of products); x does, and
    // so do the outputs' readers.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x == 0 && p.row_expert) {        // rows without an expert: zeros
        for (int s = warp; s < p.rows; s += kWarps) {
            if (ch.scratch[s] != INT32_MAX) continue;
            if (lane == 0) set_status(p.status, MOE_ERR_DATA);
            for (int n = lane; n < p.N; n += 32) {
                if (p.out_bf16) static_cast<uint16_t *>(p.out)[static_cast<int64_t>(s) * p.N + n] = 0;
                else static_cast<float *>(p.out)[static_cast<int64_t>(s) * p.N + n] = 0.0f;
            }
        }
    }

    int slot = 0, slot_in = C::kDepth - 1, buf = 0, n_tok = 0, start = 0;
    int chunk = count > 0 ? first / groups : 0, grp = count > 0 ? first % groups : 0;
    bool fresh = true;
    uint32_t any_bad = 0;
    for (int left = count; left > 0; --left) {
        if (fresh) {
            fresh = false;
            start = ch.first[chunk];
            n_tok = ch.first[chunk + 1] - start;
            __syncthreads();                      // sums of the last item are read with the old exponents
            stage_x<F>(p, ch.order + start, n_tok, xs, pitch, exps);
        }
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t bad[2] = {0, 0}, off[2] = {0, 0};
        if constexpr (kShift) {
#pragma unroll
            for (int r = 0; r < 2; ++r)           // a stage's scale bytes are a multiple of 4
                off[r] = reinterpret_cast<uintptr_t>(p.scales + weight_row(chunk, grp, g + 8 * r) * s_pitch) & 3;
        }
        uint32_t xa = smem_u32(xs) + min(g, n_tok - 1) * pitch + t4 * 16 + u0 * (F == kBf16 ? 64 : 256);
#pragma unroll 1
        for (int unit = u0; unit < u1; ++unit) {
            cp_wait<C::kDepth - 2>();
            __syncwarp();                         // all lanes' copies; and the slot to fill is read
            fetch_next(slot_in);
            multiply<F, kShift>(ring_a + slot * C::kStage, xa, g < n_tok, F == kBf16 ? 1 : (p.K - unit * 128) >> 5, g, t4,
                                off, acc, bad);
            xa += F == kBf16 ? 64 : 256;
            slot = slot + 1 == C::kDepth ? 0 : slot + 1;
            slot_in = slot_in + 1 == C::kDepth ? 0 : slot_in + 1;
        }
        if constexpr (F == kMx) {
            const float nan = __uint_as_float(0x7FC00000u);
            if (bad[0]) acc[0] = acc[1] = nan;
            if (bad[1]) acc[2] = acc[3] = nan;
        }
        any_bad |= bad[0] | bad[1];
        float *mine = sums + (buf * kWarps + warp) * kTileFloats;
        *reinterpret_cast<float2 *>(mine + g * kTok + 2 * t4) = make_float2(acc[0], acc[1]);
        *reinterpret_cast<float2 *>(mine + (g + 8) * kTok + 2 * t4) = make_float2(acc[2], acc[3]);
        __syncthreads();
        // Everyone adds up its outputs over the warps that shared the tile, in order.
        constexpr int kOuts = kTileCols * kTok;
        for (int i = tid; i < group * kOuts; i += kThreads) {
            const int tile = i / kOuts, r = i % kOuts / kTok, t = i % kTok;
            const int n = (grp * group + tile) * kTileCols + r;
            if (t >= n_tok || n >= p.N) continue;
            const float *q = sums + (buf * kWarps + tile * kw) * kTileFloats + r * kTok + t;
            float v = 0.f, u = 0.f;
            for (int j = 0; j < kw; ++j) {
                v += q[j * kTileFloats];
                if (kSwiglu) u += q[j * kTileFloats + 8 * kTok];
            }
            if constexpr (F != kBf16) {
                const int e = exps[t] + (F == kMx ? 31 : 0);
                const float s2 = F == kNv ? __ldg(p.ws2 + ch.expert[chunk]) : 1.0f;
                const auto whole = [&](float a) {
                    return e > 0 ? ldexpf(a * s2, e) : ldexpf(a, e) * s2;
                };
                v = whole(v);
                if (kSwiglu) u = whole(u);
            }
            if (kSwiglu) v = silu_f32(v) * u;
            const int64_t o = static_cast<int64_t>(ch.order[start + t]) * p.N + n;
            if (kSwiglu || p.out_bf16) static_cast<__nv_bfloat16 *>(p.out)[o] = __float2bfloat16_rn(v);
            else static_cast<float *>(p.out)[o] = v;
        }
        buf ^= 1;
        if (++grp == groups) {
            grp = 0;
            ++chunk;
            fresh = true;
        }
    }
    cp_wait<0>();
    if constexpr (F != kBf16)
        if (__any_sync(0xffffffffu, any_bad != 0) && lane == 0) set_status(p.status, MOE_ERR_DATA);
}

// out[t, n] = sum_j w[t, j] * y[t k + j, n] over the slots with a valid expert, in ascending j.
template <typename T>
__global__ void weigh_kernel(const float *y, const int32_t *ids, const float *w, int k, int N, int E, T *out) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int n = blockIdx.x * blockDim.x + threadIdx.x, t = blockIdx.y;
    if (n >= N) return;
    float acc = 0.f;
    for (int j = 0; j < k; ++j) {
        const int s = t * k + j;
        if (static_cast<unsigned>(__ldg(ids + s)) >= static_cast<unsigned>(E)) continue;
        acc = fmaf(__ldg(w + s), __ldcg(y + static_cast<int64_t>(s) * N + n), acc);
    }
    if constexpr (sizeof(T) == 2) out[static_cast<int64_t>(t) * N + n] = __float2bfloat16_rn(acc);
    else out[static_cast<int64_t>(t) * N + n] = acc;
}

constexpr int kMaxSmem = 232448;

template <int F, bool kSwiglu, bool kShift>
moe_status launch(Params p, bool chained, cudaStream_t stream, int num_sms) {
    using C = Fmt<F>;
    p.k_pad = (p.K + C::kUnit - 1) / C::kUnit * C::kUnit;
    const size_t fixed = kWarps * C::kDepth * C::kStage + 2 * kWarps * kTileFloats * sizeof(float) +
                         (kTok + 2 + 4 * static_cast<size_t>(p.rows)) * sizeof(int);
    const size_t pitch = static_cast<size_t>(p.k_pad) * 2 + 64;
    p.tok = p.rows < kTok ? p.rows : kTok;
    while (p.tok > 1 && fixed + p.tok * pitch > kMaxSmem) p.tok = (p.tok + 1) / 2;
    const size_t bytes = fixed + p.tok * pitch;
    if (bytes > kMaxSmem) return MOE_ERR_CAPACITY;
    static std::atomic<uint64_t> mask{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
    const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
    const auto kernel = matvec_kernel<F, kSwiglu, kShift>;
    if (!bit || !(mask.load(std::memory_order_acquire) & bit)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem) != cudaSuccess)
            return MOE_ERR_CUDA;
        mask.fetch_or(bit, std::memory_order_release);
    }
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_sms);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = chained ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace mv

moe_status launch_matvec(const Matvec &m, cudaStream_t stream, int num_sms) {
    if (m.rows == 0) return MOE_OK;
    mv::Params p = {};
    p.x = m.x;
    p.x_stride = m.x_stride;
    p.div = m.index_div;
    p.row_expert = m.row_expert;
    p.rows = m.rows;
    p.K = m.K;
    p.E = m.E;
    p.N = m.N;
    p.w = static_cast<const uint8_t *>(m.weights);
    p.scales = m.scales;
    p.ws2 = m.weight_scale_2;
    p.out = m.out;
    p.out_bf16 = m.out_bf16;
    p.status = m.status;
    p.x_vec = reinterpret_cast<uintptr_t>(m.x) % 16 == 0 && (m.x_stride % 8 == 0 || m.rows <= m.index_div);
    if (m.format == Matvec::kBf16)
        return m.swiglu ? mv::launch<mv::kBf16, true, false>(p, m.chained, stream, num_sms)
                        : mv::launch<mv::kBf16, false, false>(p, m.chained, stream, num_sms);
    const bool nv = m.format == Matvec::kNv;
    // Scale rows at 4-byte addresses are copied as they are; others as the words around them.
    const bool shift = (m.K / (nv ? 16 : 32)) % 4 != 0 || reinterpret_cast<uintptr_t>(m.scales) % 4 != 0;
    if (shift)
        return nv ? m.swiglu ? mv::launch<mv::kNv, true, true>(p, m.chained, stream, num_sms)
                             : mv::launch<mv::kNv, false, true>(p, m.chained, stream, num_sms)
                  : m.swiglu ? mv::launch<mv::kMx, true, true>(p, m.chained, stream, num_sms)
                             : mv::launch<mv::kMx, false, true>(p, m.chained, stream, num_sms);
    return nv ? m.swiglu ? mv::launch<mv::kNv, true, false>(p, m.chained, stream, num_sms)
                         : mv::launch<mv::kNv, false, false>(p, m.chained, stream, num_sms)
              : m.swiglu ? mv::launch<mv::kMx, true, false>(p, m.chained, stream, num_sms)
                         : mv::launch<mv::kMx, false, false>(p, m.chained, stream, num_sms);
}

moe_status launch_weigh(const float *y, const int32_t *ids, const float *w, int T, int k, int N, int E, void *out,
                        int out_bf16, cudaStream_t stream) {
    if (T == 0 || N == 0) return MOE_OK;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((N + 127) / 128, T);        // T: up to MOE_MATVEC_MAX_ROWS
    cfg.blockDim = dim3(128);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e =
        out_bf16 ? cudaLaunchKernelEx(&cfg, mv::weigh_kernel<__nv_bfloat16>, y, ids, w, k, N, E, static_cast<__nv_bfloat16 *>(out))
                 : cudaLaunchKernelEx(&cfg, mv::weigh_kernel<float>, y, ids, w, k, N, E, static_cast<float *>(out));
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
