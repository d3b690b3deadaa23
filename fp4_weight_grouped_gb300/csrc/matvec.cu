// Products of a few rows with weight matrices that each row chooses:
//
//   out[r, n] = sum_k x[r / div, k] * w[e_r, n, k]          (SwiGLU: rows n and I + n)
//
// w in 4 bits (MXFP4: e2m1 * 2^(s - 127) per 32 k; NVFP4: e2m1 * e4m3 per 16 k, times
// an f32 an expert) or bf16.  For one to a few dozen rows: no sort, no row bands.
//
// Bound by HBM where there are weights enough: 6.6 TB/s for every further token's six experts
// in MXFP4 (hidden 4,096, inter 2,048, w13; 6.3 for w2), on top of 7 to 8 us that a launch
// takes before and behind them (5.5 for a tiny product).  One token: w13 16 us, w2 11; eight
// in NVFP4: 75 us (6.0 TB/s) and 43 (5.3), in MXFP4 73 and 41.
//
//  * Rows of the same expert are taken together, up to 8 or 4 at a time (a chunk), so a
//    weight is read once for them.  Every CTA works the chunks out from the ids itself.
//  * A tile is 32 weight rows (SwiGLU: 16 gate rows and the 16 matching up rows, so that one
//    thread finds both).  kw warps of a CTA share a tile's K, 256 k (bf16: 64) a stage, every
//    kw-th stage each (that neighbours along a row are read together: one token through six
//    experts 29.4 -> 27.3 us), and add up their sums in shared memory in a fixed order.
//  * mma.sync m16n8k16 with the weights as A and the chunk's rows as B columns: eight
//    rows cost what one costs, and a thread's four sums are f32.  Tensor memory has
//    nothing to offer here: no operand is used twice.
//  * 4-bit weights become f16 by cvt (exact), so x has to be f16 as well: each row is
//    scaled by a power of two that brings its largest magnitude to [2^14, 2^15).  A bf16
//    has 8 bits, f16 spans 2^-24 .. 2^15: elements down to 2^-28 of the row's largest are
//    exact, smaller ones are off by at most 2^-39 of it.
//  * h is rounded to bf16 between a decode step's products, as in the layer that sorts its rows,
//    so that either gives the same step: the output's error is 0.0023 of its norm, with h in f32
//    it would be the output's own rounding, 0.0016.
//  * MXFP4: the scale is the same for the 32 k of two MMAs, whose sums it multiplies in
//    f32, beside as much of the power of two that x was scaled by as f32 holds (row_bias):
//    every scale of the format counts, and sums have the range of the result.
//    NVFP4: e2m1 * e4m3 has 6 bits and fits f16, so the scale goes into the weight.
//    Experts with one or two rows: the columns that are left over keep the scale blocks apart
//    (multiply_few), for either format.
//  * Each warp fetches its own stages by TMA into its own ring, across tiles: 128 bytes of 32
//    rows a box (a box costs an SM at least 33 ns: boxes of 64 bytes by 16 rows, and scales
//    in boxes of their own beside them, held the kernel at 4.4 TB/s; by cp.async the copies'
//    writes took half of the shared-memory pipe).  HBM gives rows of 128 bytes 6.0 to 6.2
//    TB/s when they come alone, rows of 256 and more 6.8 to 7.0.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include <cuda.h>

#include "device_common.cuh"
#include "launch.h"
#include "tensor_map.h"

namespace moe {
namespace mv {

enum Format { kMx, kNv, kBf16 };

constexpr int kTok = 8;                       // rows a chunk at most (the MMA's n)
constexpr int kTileRows = 32;                 // weight rows a tile: two MMAs' share one load of x
constexpr int kMaxDepth = 4;
constexpr int kSumPitch = 36;                 // floats of a token's 32 sums, free of bank conflicts

template <int v>
struct Int {
    static constexpr int value = v;
};

// A CTA with an SM to itself, or (kFew, chunks of up to four rows) two CTAs an SM: one works
// while the other starts, ends an item or waits (one token 27.3 -> 26.5 us, eight in NVFP4
// 115.5 -> 111.0; four CTAs of 4 warps 28.5 and 116; bf16 within 6% either way, so it has none).
template <bool kFew>
struct Shape {
    static constexpr int kWarps = kFew ? 8 : 16, kThreads = 32 * kWarps;
    static constexpr int kTok = kFew ? 4 : 8;
    static constexpr int kVecs = kFew ? 2 : 1;     // loads of a row of x that a thread keeps in registers
    static constexpr int kCtas = kFew ? 2 : 1;
    static constexpr int kMaxSmem = kFew ? 115712 : 232448;
};

template <int F>
struct Fmt {
    static constexpr int kUnit = F == kBf16 ? 64 : 256;             // k of a stage: 128 bytes a row
    // Scales come 16 bytes a row: NVFP4's of a stage, MXFP4's of two.
    static constexpr int kScaleBytes = F == kMx ? 8 : F == kNv ? 16 : 0;
    static constexpr int kStage = kTileRows * 128 + (F == kBf16 ? 0 : 16 * kTileRows);
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
    int tok;                      // rows a chunk, 1..Shape::kTok
    int kw;                       // warps that share a tile, a power of two
    int depth;                    // stages of a warp's ring
    int k_pad;                    // K up to a stage
    int smem;                     // bytes a CTA
    int x_vec;                    // x rows at 16-byte addresses
    int chained;                  // x comes from the launch before
    uint64_t wait_limit_ns;
};

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

// a += s f d for the two columns of a lane's row, two numbers an instruction.
__device__ __forceinline__ void add_scaled(float &a0, float &a1, float s, const float (&f)[2], float d0, float d1) {
    asm("{\n\t.reg .b64 a, d, s, f;\n\t"
        "mov.b64 a, {%0, %1};\n\tmov.b64 d, {%5, %6};\n\tmov.b64 s, {%2, %2};\n\tmov.b64 f, {%3, %4};\n\t"
        "mul.rn.f32x2 d, d, f;\n\tfma.rn.f32x2 a, s, d, a;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "+f"(a0), "+f"(a1)
        : "f"(s), "f"(f[0]), "f"(f[1]), "f"(d0), "f"(d1));
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
__device__ __forceinline__ void e4m3_floats(uint32_t b, float &first, float &second) {
    asm("{\n\t.reg .b16 t, lo, hi;\n\t.reg .b32 h;\n\tcvt.u16.u32 t, %2;\n\tcvt.rn.f16x2.e4m3x2 h, t;\n\t"
        "mov.b32 {lo, hi}, h;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
        : "=f"(first), "=f"(second)
        : "r"(b));
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

template <int kThreads>
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

__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Power of two that a row of x is scaled by, from the exponent field of its largest magnitude.
__device__ __forceinline__ int row_exponent(int top) { return max(top - 127 - 14, -126); }

// MXFP4: what a row's sums are multiplied by at the end is 2^(row_exponent - row_bias).  For x of
// ordinary size (largest magnitude 2^-17 to 2^16) the bias is the exponent: the sums are in the
// result's own units, and overflow or lose bits where the result does.  For smaller x they stay
// 2^-31 low, which holds 1,024 blocks' sums of up to 2^15 * 6 * 32 below 2^127 for every scale; for
// larger x they are lower than the result, but a step of theirs (2^-149) is no more than what the
// smallest weight, 2^-128, makes of x's own rounding to 2^-38 of its row's largest.
__device__ __forceinline__ int row_bias(int exponent) { return min(max(exponent, -31), 2); }

// A block's sum (2^-25 to 2^23) times half of 2^row_bias is exact, and twice the scale of any byte,
// 2^(s + 1 - 127), a normal number: the only rounding is the sum's.
__device__ __forceinline__ float bias_factor(int top) {
    return power_of_two(min(max(top - 127 - 14, -31), 2) - 1);             // row_bias(row_exponent(top)) - 1
}
__device__ __forceinline__ float twice_e8m0(uint32_t s) { return __uint_as_float(s * 0x800000u + 0x800000u); }

// Eight elements of a row of x; zeros past its end.  Not through the read-only path: x may come
// from a launch that ended after this one began.
__device__ __forceinline__ uint4 load_x(const Params &p, int slot, int v) {
    uint4 a = make_uint4(0, 0, 0, 0);
    if (8 * v < p.K) {                // K is a multiple of 8
        const uint16_t *q = p.x + (slot / p.div) * p.x_stride + 8 * v;
        if (p.x_vec) {
            a = __ldcg(reinterpret_cast<const uint4 *>(q));
        } else {
            a.x = __ldcg(q) | static_cast<uint32_t>(__ldcg(q + 1)) << 16;
            a.y = __ldcg(q + 2) | static_cast<uint32_t>(__ldcg(q + 3)) << 16;
            a.z = __ldcg(q + 4) | static_cast<uint32_t>(__ldcg(q + 5)) << 16;
            a.w = __ldcg(q + 6) | static_cast<uint32_t>(__ldcg(q + 7)) << 16;
        }
    }
    return a;
}

// Largest exponent field among the finite ones of eight elements.
__device__ __forceinline__ uint32_t top_of(const uint4 &a) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = w[i] & 0x7F80u, hi = w[i] >> 16 & 0x7F80u;
        top = max(top, lo == 0x7F80u ? 0u : lo);
        top = max(top, hi == 0x7F80u ? 0u : hi);
    }
    return top >> 7;
}

template <int F>
__device__ __forceinline__ void store_x(uint8_t *row, int v, const uint4 &a, int top, bool by_blocks) {
    if constexpr (F == kBf16) {
        *reinterpret_cast<uint4 *>(row + 16 * v) = a;
    } else {
        const float f = __uint_as_float(static_cast<uint32_t>(127 - row_exponent(top)) << 23);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("cvt.rn.f16x2.f32 %0, %1, %2;"
                : "=r"(o[i])
                : "f"(__uint_as_float(w[i] & 0xFFFF0000u) * f), "f"(__uint_as_float(w[i] << 16) * f));
        const int at = F == kNv || by_blocks ? (v & ~15) | (v & 3) << 2 | (v >> 2 & 3) : v;
        *reinterpret_cast<uint4 *>(row + 16 * at) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// Rows of x in registers, where a thread has kVecs loads of each at most.
template <class S>
__device__ __forceinline__ void fetch_x(const Params &p, const int *slots, int n, uint4 (&a)[kTok]) {
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
        const int t = i / S::kVecs, v = threadIdx.x + i % S::kVecs * S::kThreads;
        if (t < n && v < p.k_pad / 8) a[i] = load_x(p, slots[t], v);
    }
}

// The chunk's rows of x into shared memory (4-bit weights: f16, scaled by 2^-row_exponent;
// bf16 as they are), zeros up to k_pad.  tops[t] (zero before) receives row t's largest
// exponent field.  Where a lane holds 32 k of its own (NVFP4, and MXFP4 for few rows), 16 bytes
// q of 128 k go to place 4 (q % 4) + q / 4: the lanes find theirs side by side.
template <int F, class S>
__device__ __forceinline__ void stage_x(const Params &p, const int *slots, int n, uint8_t *xs, int pitch, int *tops,
                                        bool fetched, bool by_blocks, uint4 (&a)[kTok]) {
    constexpr int kThreads = S::kThreads, kVecs = S::kVecs;
    const int tid = threadIdx.x, vecs = p.k_pad / 8;
    if (vecs <= kThreads * kVecs) {
        if (!fetched) fetch_x<S>(p, slots, n, a);
        if constexpr (F != kBf16) {
#pragma unroll
            for (int t = 0; t < S::kTok; ++t) {
                if (t >= n) break;
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < kVecs; ++i)
                    if (tid + i * kThreads < vecs) top = max(top, top_of(a[t * kVecs + i]));
                top = __reduce_max_sync(0xffffffffu, top);
                if ((tid & 31) == 0) atomicMax(&tops[t], static_cast<int>(top));
            }
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
            const int t = i / kVecs, v = tid + i % kVecs * kThreads;
            if (t < n && v < vecs) store_x<F>(xs + t * pitch, v, a[i], F == kBf16 ? 0 : tops[t], by_blocks);
        }
    } else {
        if constexpr (F != kBf16) {
            for (int t = 0; t < n; ++t) {
                uint32_t top = 0;
                for (int v = tid; v < vecs; v += kThreads) top = max(top, top_of(load_x(p, slots[t], v)));
                top = __reduce_max_sync(0xffffffffu, top);
                if ((tid & 31) == 0) atomicMax(&tops[t], static_cast<int>(top));
            }
            __syncthreads();
        }
        for (int t = 0; t < n; ++t)
            for (int v = tid; v < vecs; v += kThreads)
                store_x<F>(xs + t * pitch, v, load_x(p, slots[t], v), F == kBf16 ? 0 : tops[t], by_blocks);
    }
    __syncthreads();
}

// 16 bytes where `real`, else what v holds already.
__device__ __forceinline__ void lds128_if(uint4 &v, uint32_t a, bool real) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
                 "@p ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
                 : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
                 : "r"(a), "r"(static_cast<int>(real)));
}

// Scale bytes, half a stage's, of the four rows that a lane multiplies: MXFP4 a word a row, NVFP4
// the two bytes of the lane's 32 k, MXFP4 for few rows of x the one byte of its 32 k.
using Scales = uint32_t[2][2];

// Rows of scales that TMA does not take (not a multiple of 16 bytes, or elsewhere aligned):
// byte by byte from global memory, zeros past the row's end.
template <int n>
__device__ __forceinline__ void load_scales(const uint8_t *const (&rows)[2][2], int at, int row_bytes, Scales &v) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            v[s][r] = 0;
#pragma unroll
            for (int i = 0; i < n; ++i)
                if (at + i < row_bytes) v[s][r] |= static_cast<uint32_t>(__ldg(rows[s][r] + at + i)) << (8 * i);
        }
}

// Half a stage (128 k; bf16: 32) of 32 weight rows: acc += w x.  The rows' 16-byte pieces lie
// in the 128-byte swizzle (piece ^ row % 8): `at` is, with the swizzle in it, the lane's
// piece t4 of its first row, or for MXFP4 (read by words of eight rows) word t4 of piece 0.
// step: bytes from row g of an MMA to row g + 8, next: to the second MMA's.  x: this lane's
// share of the chunk's rows, zeros in lanes without one.  factor: MXFP4: bias_factor of the rows in
// the lane's two columns.
template <int F>
__device__ __forceinline__ void multiply(uint32_t at, int step, int next, uint32_t xa, bool has_x, const Scales &sw,
                                         const float (&factor)[2], uint4 (&x)[4], float (&acc)[2][4], Scales &bad) {
    if constexpr (F == kBf16) {
        lds128_if(x[0], xa, has_x);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const uint32_t row = at + s * next;
            const uint4 a = lds128(row), c = lds128(row + step);
            mma16816<false>(acc[s], a.x, c.x, a.y, c.y, x[0].x, x[0].y);
            mma16816<false>(acc[s], a.z, c.z, a.w, c.w, x[0].z, x[0].w);
        }
    } else if constexpr (F == kNv) {
        // Lane t4 holds the 32 k of block t4, two scales a row.
        uint4 ra[2], rc[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const uint32_t row = at + s * next;
            ra[s] = lds128(row);
            rc[s] = lds128(row + step);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) lds128_if(x[j], xa + 64 * j, has_x);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            bad[0][0] |= (((sw[s][0] | sw[s][1] << 16) & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;     // NaN
            uint32_t f[2][2];
            e4m3_pairs(sw[s][0], f[0][0], f[0][1]);
            e4m3_pairs(sw[s][1], f[1][0], f[1][1]);
            const uint32_t wa[4] = {ra[s].x, ra[s].y, ra[s].z, ra[s].w}, wc[4] = {rc[s].x, rc[s].y, rc[s].z, rc[s].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t a[4], c[4];
                decode8(wa[j], a);
                decode8(wc[j], c);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a[i] = hmul2(a[i], f[0][j >> 1]);
                    c[i] = hmul2(c[i], f[1][j >> 1]);
                }
                mma16816<true>(acc[s], a[0], c[0], a[1], c[1], x[j].x, x[j].y);
                mma16816<true>(acc[s], a[2], c[2], a[3], c[3], x[j].z, x[j].w);
            }
        }
    } else {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int r = 0; r < 2; ++r)
                bad[s][r] |= ((sw[s][r] & 0x7F7F7F7Fu) + 0x03030303u) & sw[s][r] & 0x80808080u;         // 253 and more
#pragma unroll
        for (int b = 0; b < 4; ++b) lds128_if(x[b], xa + 64 * b, has_x);
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const uint32_t row = (at ^ (16 * b)) + s * next;
                uint32_t a[4], c[4];
                decode8(lds32(row), a);
                decode8(lds32(row + step), c);
                float d[4] = {0.f, 0.f, 0.f, 0.f};
                mma16816<true>(d, a[0], c[0], a[1], c[1], x[b].x, x[b].y);
                mma16816<true>(d, a[2], c[2], a[3], c[3], x[b].z, x[b].w);
                const float s0 = twice_e8m0(sw[s][0] >> (8 * b) & 0xFFu), s1 = twice_e8m0(sw[s][1] >> (8 * b) & 0xFFu);
                add_scaled(acc[s][0], acc[s][1], s0, factor, d[0], d[1]);
                add_scaled(acc[s][2], acc[s][3], s1, factor, d[2], d[3]);
            }
    }
}

// The same for one or two rows of x.  A lane's 16 bytes are 32 k of their own, and a column of the
// MMAs holds a row of x where k is in one scale block and zeros elsewhere: the sums keep the
// blocks apart, and a block's scale multiplies once behind them (half of the instructions of the
// form above: one token's w13 20.0 -> 18.1 us, w2 13.5 -> 11.6).  Column j: row j % 2, block j / 2
// of four (MXFP4: a half's; NVFP4: those of two words after those of the other two), or for one
// row of NVFP4 (kRows 1) block j of eight; of one row of MXFP4 every second column is empty.  has:
// whether this lane's words 0 and 1, and 2 and 3, belong to its column; x stays zero where they do
// not.  factor: as above.  What acc holds is a quarter of a sum.
template <int F, int kRows>
__device__ __forceinline__ void multiply_few(uint32_t at, int step, int next, uint32_t xa, const bool (&has)[2],
                                             const Scales &sw, const float (&factor)[2], uint4 (&x)[4],
                                             float (&acc)[2][4], Scales &bad) {
    uint4 ra[2], rc[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const uint32_t row = at + s * next;
        ra[s] = lds128(row);
        rc[s] = lds128(row + step);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) lds128_if(x[j], xa + 64 * j, has[j >> 1]);
    float scale[2][2][2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        if constexpr (F == kNv)
            bad[0][0] |= (((sw[s][0] | sw[s][1] << 16) & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;         // NaN
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            if constexpr (F == kMx) {
                bad[s][r] |= (sw[s][r] + 3u) & 0x100u;                                                   // 253 and more
                scale[s][r][0] = twice_e8m0(sw[s][r]);
            } else {
                e4m3_floats(sw[s][r], scale[s][r][0], scale[s][r][1]);
            }
        }
    }
    constexpr int kWords = F == kNv && kRows == 2 ? 2 : 4;      // that one set of sums takes
#pragma unroll
    for (int b = 0; b < 4; b += kWords) {
        float d[2][4] = {};
#pragma unroll
        for (int j = b; j < b + kWords; ++j)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const uint32_t wa[4] = {ra[s].x, ra[s].y, ra[s].z, ra[s].w}, wc[4] = {rc[s].x, rc[s].y, rc[s].z, rc[s].w};
                uint32_t a[4], c[4];
                decode8(wa[j], a);
                decode8(wc[j], c);
                mma16816<true>(d[s], a[0], c[0], a[1], c[1], x[j].x, x[j].y);
                mma16816<true>(d[s], a[2], c[2], a[3], c[3], x[j].z, x[j].w);
            }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            if constexpr (F == kMx && kRows == 1) {        // the second column of a lane has no row
                acc[s][0] = fmaf(scale[s][0][0], d[s][0] * factor[0], acc[s][0]);
                acc[s][2] = fmaf(scale[s][1][0], d[s][2] * factor[0], acc[s][2]);
            } else if constexpr (F == kMx) {
                add_scaled(acc[s][0], acc[s][1], scale[s][0][0], factor, d[s][0], d[s][1]);
                add_scaled(acc[s][2], acc[s][3], scale[s][1][0], factor, d[s][2], d[s][3]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)   // either column the same block and its own row, or the same row
                    acc[s][kRows == 2 ? i : i & 2] = fmaf(scale[s][i >> 1][kRows == 2 ? b >> 1 : i & 1], d[s][i], acc[s][kRows == 2 ? i : i & 2]);
            }
        }
    }
}

template <int F, bool kSwiglu, bool kTmaScales, bool kFew>
__global__ void __launch_bounds__(Shape<kFew>::kThreads, Shape<kFew>::kCtas)
    matvec_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_s, const Params p) {
    using C = Fmt<F>;
    using S = Shape<kFew>;
    constexpr int kWarps = S::kWarps, kThreads = S::kThreads;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t4 = lane & 3;
    const int kw = p.kw, depth = p.depth;
    const int group = kWarps / kw, group_log2 = 31 - __clz(group);      // tiles an item, a power of two
    const int pitch = p.k_pad * 2 + 64, sum_floats = p.tok * kSumPitch;
    // ring: stages, all warps' scales behind them | x | sums | barriers | chunk tables
    uint8_t *xs = smem + kWarps * depth * C::kStage;
    float *sums = reinterpret_cast<float *>(xs + p.tok * pitch);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sums + kWarps * sum_floats) + warp * kMaxDepth;
    int *tab = reinterpret_cast<int *>(bars + (kWarps - warp) * kMaxDepth);
    int *tops = tab;                              // [2][kTok], in turn
    tab += 2 * kTok;
    const Chunks ch = {tab + 1, tab + 1 + p.rows, tab + 2 + 2 * p.rows, tab + 2 + 3 * p.rows, tab};
    if (lane == 0) {
        for (int i = 0; i < depth; ++i) mbar_init(&bars[i], 1);
        mbar_fence_init();
        if (warp == 0) {
            tma_prefetch_map(&tm_w);
            if (kTmaScales) tma_prefetch_map(&tm_s);
        }
    }
    if (tid < 2 * kTok) tops[tid] = 0;
    build_chunks<kThreads>(p, ch);

    constexpr int kTileCols = kSwiglu ? kTileRows / 2 : kTileRows;
    const int tiles = (p.N + kTileCols - 1) / kTileCols;
    const int groups = (tiles + group - 1) / group;          // items a chunk
    // The CTA's share of the items, one after another.  (rows * N < 2^31, so counts fit.)
    const int chunks = *ch.count;
    const bool unnamed = ch.first[chunks] < p.rows;
    const int total = chunks * groups, grid = gridDim.x, blk = blockIdx.x;
    const int first = total / grid * blk + min(blk, total % grid);
    const int count = total / grid + (blk < total % grid);
    const int chunk0 = count > 0 ? first / groups : 0, grp0 = count > 0 ? first % groups : 0;
    const int wk = warp & (kw - 1), wt = warp / kw;
    const int units = (p.K + C::kUnit - 1) / C::kUnit;

    // A stage: 32 rows (SwiGLU: 16 gate rows, the 16 up rows of the same columns) and their
    // scales.  What lies past an expert's rows or a row's end reads as zeros.
    const uint32_t ring = smem_u32(smem) + warp * depth * (kTileRows * 128);
    const uint32_t scale_ring = smem_u32(smem) + kWarps * depth * (kTileRows * 128) + warp * depth * (16 * kTileRows);
    int f_left = wk < units ? count : 0, f_unit = wk, f_slot = 0, f_chunk = chunk0, f_grp = grp0;
    const auto fetch_next = [&]() {
        if (f_left > 0) {
            if (lane == 0) {
                const int z = ch.expert[f_chunk] * (kSwiglu ? 2 : 1), n = (f_grp * group + wt) * kTileCols;
                uint64_t *bar = &bars[f_slot];
                mbar_arrive_expect_tx(bar, kTileRows * (kTmaScales ? 128 + 16 : 128));
                tma_load_3d(ring + f_slot * (kTileRows * 128), &tm_w, f_unit * 128, n, z, bar);
                if constexpr (kTmaScales)
                    tma_load_3d(scale_ring + f_slot * (16 * kTileRows), &tm_s, f_unit * C::kScaleBytes & ~15, n, z, bar);
            }
            f_slot = f_slot + 1 == depth ? 0 : f_slot + 1;
            f_unit += kw;
            if (f_unit >= units) {
                f_unit = wk;
                --f_left;
                if (++f_grp == groups) {
                    f_grp = 0;
                    ++f_chunk;
                }
            }
        }
    };
    // The first rows of x ahead of the weights, behind which they would queue, unless they
    // come from the launch before (a chain of products): weights and ids do not.
    uint4 xr[kTok];
    const bool ahead = !p.chained && count > 0 && p.k_pad / 8 <= kThreads * S::kVecs;
    if (ahead) fetch_x<S>(p, ch.order + ch.first[chunk0], ch.first[chunk0 + 1] - ch.first[chunk0], xr);
#pragma unroll 1
    for (int i = 0; i < depth; ++i) fetch_next();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (unnamed) {                                // rows without an expert: zeros, by all CTAs
        constexpr int kPiece = 1024;              // columns a warp
        if (blk == 0 && tid == 0) set_status(p.status, MOE_ERR_DATA);
        const int pieces = (p.N - 1) / kPiece + 1;
        for (int i = blk * kWarps + warp; i < p.rows * pieces; i += grid * kWarps) {
            const int s = i / pieces, from = i % pieces * kPiece;
            if (ch.scratch[s] != INT32_MAX) continue;
            const int end = p.N - from < kPiece ? p.N : from + kPiece;
            for (int n = from + lane; n < end; n += 32) {
                if (p.out_bf16) static_cast<uint16_t *>(p.out)[static_cast<int64_t>(s) * p.N + n] = 0;
                else static_cast<float *>(p.out)[static_cast<int64_t>(s) * p.N + n] = 0.0f;
            }
        }
    }

    // MMA rows g and g + 8 are stage rows q and q + 8 of 16 (SwiGLU: gate and up of eight
    // columns).  Neighbours in g are four rows apart: the eight lanes that read 16 bytes
    // together then meet eight different pieces of the swizzle.
    const int q = g >> 1 | (g & 1) << 2;
    constexpr int kStep = (kSwiglu ? 16 : 8), kNext = (kSwiglu ? 8 : 16);
    const uint32_t piece0 = ring + q * 128 + (t4 ^ q) * 16, row0 = F == kMx ? ring + q * 128 + q * 16 + 4 * t4 : piece0;
    const uint32_t scale0 = scale_ring + q * 16;
    constexpr int kUnitX = 2 * C::kUnit;
    uint32_t slot = 0, phase = 0, any_bad = 0;
    int n_tok = 0, start = 0, turn = 0, chunk = chunk0, grp = grp0;
    bool fresh = true, ok = true, few = false;
    uint4 x[4];
    float factor[2] = {};
    for (int left = count; left > 0; --left) {
        if (fresh) {                              // everyone is past the last x
            fresh = false;
            start = ch.first[chunk];
            n_tok = ch.first[chunk + 1] - start;
            if (left != count) __syncthreads();   // and past its exponents
            turn ^= kTok;
            // Only where it is the expert's only chunk: rows that share an expert take one way, so that
            // equal ones have equal results.
            few = kFew && n_tok <= 2 && (chunk == 0 || ch.expert[chunk - 1] != ch.expert[chunk]) &&
                  (chunk + 1 == *ch.count || ch.expert[chunk + 1] != ch.expert[chunk]);
            stage_x<F, S>(p, ch.order + start, n_tok, xs, pitch, tops + turn, ahead && left == count, few, xr);
            if (tid < kTok) tops[(turn ^ kTok) + tid] = 0;
            if constexpr (F == kMx) {             // of the rows in this lane's columns
#pragma unroll
                for (int i = 0; i < 2; ++i) factor[i] = bias_factor(tops[turn + (few ? i : (2 * t4 + i) % kTok)]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = make_uint4(0, 0, 0, 0);
        }
        float acc[2][4] = {};
        Scales bad = {};
        const uint8_t *srow[2][2] = {};
        if constexpr (F != kBf16 && !kTmaScales) {
            const int n = (grp * group + wt) * kTileCols;
            const int64_t at = static_cast<int64_t>(ch.expert[chunk]) * (kSwiglu ? 2 : 1) * p.N;
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int r = 0; r < 2; ++r) {     // columns past the last: the last one's
                    const int c = kSwiglu ? min(n + 8 * s + q, p.N - 1) + r * p.N : min(n + 16 * s + 8 * r + q, p.N - 1);
                    srow[s][r] = p.scales + (at + c) * (p.K / (F == kMx ? 32 : 16));
                }
        }
        uint32_t xa = smem_u32(xs) + min(few ? g & 1 : g, n_tok - 1) * pitch + t4 * 16 + wk * kUnitX;
        // The scale bytes that a lane wants: n of a row, from byte `at` of a row's stage on.
        const auto scales_of = [&](auto n, int unit, int at, Scales &sw) {
            if constexpr (!kTmaScales) {
                load_scales<n.value>(srow, unit * C::kScaleBytes + at, p.K / (F == kMx ? 32 : 16), sw);
            } else {
                const uint32_t sa = scale0 + slot * (16 * kTileRows) + (unit * C::kScaleBytes & 15) + at;
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const uint32_t a = sa + (s * kNext + r * kStep) * 16;
                        sw[s][r] = n.value == 4 ? lds32(a) : n.value == 2 ? lds16(a) : lds8(a);
                    }
            }
        };
        const auto stages = [&](auto few_rows) {
            constexpr int kScales = F == kNv ? 2 : few_rows.value ? 1 : 4;
            const uint32_t rows = (F == kMx && !few_rows.value ? row0 : piece0);
            bool has[2] = {g < n_tok};
            if (few_rows.value > 0) has[0] = has[1] = t4 == g >> 1 && (g & 1) < n_tok;
            if (F == kNv && few_rows.value == 1) {
                has[0] = t4 == g >> 1 && (g & 1) == 0;
                has[1] = t4 == g >> 1 && (g & 1) == 1;
            }
#pragma unroll 1
            for (int unit = wk; ok && unit < units; unit += kw) {
                ok = warp_wait_bounded(&bars[slot], phase, nullptr, p.status, p.wait_limit_ns);
                if (!ok) break;
                // One half after the other, not unrolled: in a short launch (one token's w2) waiting
                // for instructions is the first of all stalls.
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    Scales sw = {};
                    if constexpr (F != kBf16) scales_of(Int<kScales>{}, unit, h * (C::kScaleBytes / 2) + (kScales < 4 ? kScales * t4 : 0), sw);
                    const uint32_t at = (rows + slot * (kTileRows * 128)) ^ (64 * h), x_at = xa + h * (kUnitX / 2);
                    if constexpr (few_rows.value > 0)
                        multiply_few<F, few_rows.value>(at, kStep * 128, kNext * 128, x_at, has, sw, factor, x, acc, bad);
                    else
                        multiply<F>(at, kStep * 128, kNext * 128, x_at, has[0], sw, factor, x, acc, bad);
                }
                xa += kUnitX * kw;
                __syncwarp();                     // the slot is read by all
                fetch_next();
                slot = slot + 1 == static_cast<uint32_t>(depth) ? 0 : slot + 1;
                phase ^= slot == 0;
            }
        };
        if constexpr (kFew) {
            if (few && n_tok == 1) stages(Int<1>{});
            else if (few) stages(Int<2>{});
            else stages(Int<0>{});
        } else {
            stages(Int<0>{});
        }
        if constexpr (F == kMx) {
            const float nan = __uint_as_float(0x7FC00000u);
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (bad[s][0]) acc[s][0] = acc[s][1] = nan;
                if (bad[s][1]) acc[s][2] = acc[s][3] = nan;
            }
        }
        any_bad |= bad[0][0] | bad[0][1] | bad[1][0] | bad[1][1];
        if (few) {                                // the quarters of a sum lie in four lanes
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[s][i] += __shfl_xor_sync(0xffffffffu, acc[s][i], 1);
                    acc[s][i] += __shfl_xor_sync(0xffffffffu, acc[s][i], 2);
                }
        }
        __syncthreads();                          // the last item's sums are read
        float *mine = sums + warp * sum_floats;   // [token][stage row]
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 2 * t4 + (i & 1);
                if (t < n_tok) mine[t * kSumPitch + s * kNext + (i >> 1) * kStep + q] = acc[s][i];
            }
        __syncthreads();
        // Everyone adds up its outputs over the warps that shared the tile, in order.
        for (int i = tid; i < group * kTileCols * n_tok; i += kThreads) {
            const int c = i % kTileCols, tile = i / kTileCols & (group - 1), t = i / kTileCols >> group_log2;
            const int n = (grp * group + tile) * kTileCols + c;
            if (n >= p.N) continue;
            const float *from = sums + tile * kw * sum_floats + t * kSumPitch + c;
            float v = 0.f, u = 0.f;
            for (int j = 0; j < kw; ++j) {
                v += from[j * sum_floats];
                if (kSwiglu) u += from[j * sum_floats + 16];
            }
            if constexpr (F != kBf16) {
                const int exponent = row_exponent(tops[turn + t]), e = exponent - (F == kMx ? row_bias(exponent) : 0);
                const float s2 = F == kNv ? __ldg(p.ws2 + ch.expert[chunk]) : 1.0f;
                // 2^e by two factors, each of them a normal number.
                const float f = power_of_two(e / 2), f2 = power_of_two(e - e / 2);
                const auto whole = [&](float a) { return e > 0 ? a * s2 * f * f2 : a * f * f2 * s2; };
                v = whole(v);
                if (kSwiglu) u = whole(u);
            }
            if (kSwiglu) v = silu_f32(v) * u;
            const int64_t o = static_cast<int64_t>(ch.order[start + t]) * p.N + n;
            if (kSwiglu || p.out_bf16) static_cast<__nv_bfloat16 *>(p.out)[o] = __float2bfloat16_rn(v);
            else static_cast<float *>(p.out)[o] = v;
        }
        if (++grp == groups) {
            grp = 0;
            ++chunk;
            fresh = true;
        }
    }
    // After a wait that gave up: what was issued, from that stage on, lands before the CTA leaves.
    if (!ok) {
        do {
            if (!warp_wait_bounded(&bars[slot], phase, nullptr, p.status, p.wait_limit_ns)) break;
            slot = slot + 1 == static_cast<uint32_t>(depth) ? 0 : slot + 1;
            phase ^= slot == 0;
        } while (slot != static_cast<uint32_t>(f_slot));
    }
    if constexpr (F != kBf16)
        if (__any_sync(0xffffffffu, any_bad != 0) && lane == 0) set_status(p.status, MOE_ERR_DATA);
}

// out[t, n] = sum_j w[t, j] * y[t k + j, n] over the slots with a valid expert, in ascending j.
// ids and weights come ahead of the wait for y, and the loads of eight rows go out together.
template <typename T>
__global__ void weigh_kernel(const float *y, const int32_t *ids, const float *w, int k, int N, int E, T *out) {
    __shared__ float weight[MOE_MATVEC_MAX_ROWS];
    __shared__ bool real[MOE_MATVEC_MAX_ROWS];
    const int n = blockIdx.x * blockDim.x + threadIdx.x, t = blockIdx.y;
    for (int j = threadIdx.x; j < k; j += blockDim.x) {        // k: up to MOE_MATVEC_MAX_ROWS
        weight[j] = __ldg(w + t * k + j);
        real[j] = static_cast<unsigned>(__ldg(ids + t * k + j)) < static_cast<unsigned>(E);
    }
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (n >= N) return;
    const float *row = y + static_cast<int64_t>(t) * k * N + n;
    float acc = 0.f;
    for (int j = 0; j < k; j += 8) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = j + i < k && real[j + i] ? __ldcg(row + static_cast<int64_t>(j + i) * N) : 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (j + i < k && real[j + i]) acc = fmaf(weight[j + i], v[i], acc);
    }
    if constexpr (sizeof(T) == 2) out[static_cast<int64_t>(t) * N + n] = __float2bfloat16_rn(acc);
    else out[static_cast<int64_t>(t) * N + n] = acc;
}

// Rows [outer][rows][bytes] in boxes of box_bytes by 32 rows, or by 16 rows of two neighbours
// in `outer`; what lies past an end reads as zeros.
bool encode(CUtensorMap *map, const void *base, int64_t bytes, int64_t rows, int64_t outer, uint32_t box_bytes, bool two) {
    PFN_cuTensorMapEncodeTiled_v12000 fn = tensor_map_encode();
    if (!fn) return false;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(bytes), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(outer)};
    cuuint64_t strides[2] = {dims[0], dims[0] * dims[1]};
    cuuint32_t box[3] = {box_bytes, two ? 16u : 32u, two ? 2u : 1u};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows a chunk, stages of a ring and warps a tile; the time that they will take in fifths of a
// stage's (INT64_MAX: no room).
template <int F, class S>
int64_t plan(Params &p, bool swiglu, int num_sms) {
    using C = Fmt<F>;
    p.k_pad = (p.K + C::kUnit - 1) / C::kUnit * C::kUnit;
    // As many rows and stages as there is room for; two stages at least (three measured no
    // faster: 256 experts, 6 and 48 rows, K = 4,096).
    const size_t rest = S::kWarps * kMaxDepth * sizeof(uint64_t) + (2 * kTok + 2 + 4 * static_cast<size_t>(p.rows)) * sizeof(int);
    const size_t x_row = static_cast<size_t>(p.k_pad) * 2 + 64 + S::kWarps * kSumPitch * sizeof(float);
    const size_t ring = S::kWarps * C::kStage;
    p.tok = p.rows < S::kTok ? p.rows : S::kTok;
    while (p.tok > 1 && rest + p.tok * x_row + 2 * ring > S::kMaxSmem) p.tok = (p.tok + 1) / 2;
    const size_t fixed = rest + p.tok * x_row;
    if (fixed + 2 * ring > S::kMaxSmem) return INT64_MAX;
    const size_t stages = (S::kMaxSmem - fixed) / ring;
    p.depth = static_cast<int>(stages < kMaxDepth ? stages : kMaxDepth);
    p.smem = static_cast<int>(fixed + p.depth * ring);
    // Warps a tile: the fewest rounds of items, in fifths of a stage's time.  An item's end costs
    // about one of them, but a whole stage where a warp has one stage an item and waits for the
    // next one's (K = 4,096, w13 by 1, 2, 4, 8 and 16 warps a tile, us: 6 rows 26.0, 16.5, 17.7,
    // 17.0, 18.4; 48 rows 79.7, 78.9, 75.3, 74.5, 88.1; w2, K = 2,048: 6 rows 15.8, 11.2, 12.0,
    // 12.5, 13.6; 48 rows 45.7, 44.7, 43.6, 49.5, 65.1).
    const int cols = swiglu ? kTileRows / 2 : kTileRows, ctas = S::kCtas * num_sms;
    const int64_t chunks = p.row_expert ? (p.rows < p.E ? p.rows : p.E) : (p.rows + p.tok - 1) / p.tok;
    const int64_t tiles = (p.N + cols - 1) / cols, units = p.k_pad / C::kUnit;
    int64_t best = INT64_MAX;
    for (int kw = S::kWarps; kw >= 1; kw /= 2) {
        const int64_t items = chunks * ((tiles * kw + S::kWarps - 1) / S::kWarps);
        const int64_t stages = (units + kw - 1) / kw;
        const int64_t cost = (items + ctas - 1) / ctas * (stages > 1 ? 5 * stages + 1 : 10);
        if (cost >= best) continue;
        best = cost;
        p.kw = kw;
    }
    return best;
}

template <int F, bool kSwiglu, bool kTmaScales, bool kFew>
moe_status launch(Params p, cudaStream_t stream, int num_sms) {
    using C = Fmt<F>;
    using S = Shape<kFew>;
    if (plan<F, S>(p, kSwiglu, num_sms) == INT64_MAX) return MOE_ERR_CAPACITY;
    CUtensorMap tm_w, tm_s;
    const int64_t outer = static_cast<int64_t>(p.E) * (kSwiglu ? 2 : 1);
    if (!encode(&tm_w, p.w, F == kBf16 ? 2ll * p.K : p.K / 2, p.N, outer, 128, kSwiglu)) return MOE_ERR_CUDA;
    tm_s = tm_w;
    if (kTmaScales && !encode(&tm_s, p.scales, p.K / (F == kMx ? 32 : 16), p.N, outer, 16, kSwiglu)) return MOE_ERR_CUDA;
    static std::atomic<uint64_t> mask{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
    const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
    const auto kernel = matvec_kernel<F, kSwiglu, kTmaScales, kFew>;
    if (!bit || !(mask.load(std::memory_order_acquire) & bit)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kMaxSmem) != cudaSuccess)
            return MOE_ERR_CUDA;
        mask.fetch_or(bit, std::memory_order_release);
    }
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(S::kCtas * num_sms);
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = p.smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = p.chained ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, tm_w, tm_s, p) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <int F>
moe_status launch_format(const Params &p, bool swiglu, bool tma, bool few, cudaStream_t stream, int num_sms) {
    // Two CTAs an SM where chunks of two rows fit and there are items for them (one row of one
    // matrix, K = N = 4,096: 8.3 us by them, 7.0 by one).
    if (few) {
        Params q = p;
        const int64_t one = plan<F, Shape<false>>(q, swiglu, num_sms);
        few = plan<F, Shape<true>>(q, swiglu, num_sms) <= one && (q.tok > 1 || q.rows == 1);
    }
    if (few)
        return swiglu ? tma ? launch<F, true, true, true>(p, stream, num_sms) : launch<F, true, false, true>(p, stream, num_sms)
                      : tma ? launch<F, false, true, true>(p, stream, num_sms) : launch<F, false, false, true>(p, stream, num_sms);
    return swiglu ? tma ? launch<F, true, true, false>(p, stream, num_sms) : launch<F, true, false, false>(p, stream, num_sms)
                  : tma ? launch<F, false, true, false>(p, stream, num_sms) : launch<F, false, false, false>(p, stream, num_sms);
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
    p.wait_limit_ns = m.wait_limit_ns;
    p.chained = m.chained;
    p.x_vec = reinterpret_cast<uintptr_t>(m.x) % 16 == 0 && (m.x_stride % 8 == 0 || m.rows <= m.index_div);
    if (m.format == Matvec::kBf16)
        return m.swiglu ? mv::launch<mv::kBf16, true, false, false>(p, stream, num_sms)
                        : mv::launch<mv::kBf16, false, false, false>(p, stream, num_sms);
    const bool nv = m.format == Matvec::kNv;
    // Whether experts with one or two rows have their own form in the kernel (and chunks up to four
    // rows, so that two CTAs fit an SM): not where a call has so many rows that these are the
    // exception (256 experts, w13 + w2 with and without it, MXFP4 / NVFP4, us: 24 rows 64, 73 / 65,
    // 73; 48 rows 106, 123 / 110, 123; 96 rows 184, 197 / 191, 196; 192 rows 312, 328 / 326, 326;
    // 384 rows 567, 492 / 579, 492), nor where it has one matrix (4 rows: 8.7, 8.4).
    const bool few = m.row_expert && m.E > 1 ? m.rows <= m.E : m.rows <= 2;
    // Rows of scales that TMA takes: a multiple of 16 bytes, at 16-byte addresses.
    const bool tma = m.K / (nv ? 16 : 32) % 16 == 0 && reinterpret_cast<uintptr_t>(m.scales) % 16 == 0;
    return nv ? mv::launch_format<mv::kNv>(p, m.swiglu, tma, few, stream, num_sms)
              : mv::launch_format<mv::kMx>(p, m.swiglu, tma, few, stream, num_sms);
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
