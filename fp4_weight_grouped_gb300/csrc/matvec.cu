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
    static constexpr int kPitch = F == kBf16 ? 64 : 80;             // free of bank conflicts
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
    int kw;                       // warps that share a tile's K
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

// The e4m3 in the low byte of b as an f16 pair, twice.
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t b) {
    uint32_t h;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h) : "r"(b & 0xFFu));
    return prmt(h, h, 0x1010u);
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
                *reinterpret_cast<uint4 *>(xs + t * pitch + 16 * v) = make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
        __syncthreads();
        // Only now: every thread has read the field above.
        if (tid < n) exps[tid] = max(exps[tid] - 127 - 14, -126);
        __syncthreads();
    }
}

// Position in a warp's stream of stages: its range of units of every tile of the CTA's items.
struct Cursor {
    int item, unit;
};

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
    const int n_chunks = *ch.count;
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

    const int tile_cols = kSwiglu ? 8 : 16;
    const int tiles = (p.N + tile_cols - 1) / tile_cols;
    const int kw = p.kw, group = kWarps / kw;     // tiles an item
    const int groups = (tiles + group - 1) / group;
    const int64_t total = static_cast<int64_t>(n_chunks) * groups;
    const int first = static_cast<int>(total * blockIdx.x / gridDim.x);
    const int last = static_cast<int>(total * (blockIdx.x + 1) / gridDim.x);
    const int units = (p.K + C::kUnit - 1) / C::kUnit;
    const int wk = warp % kw, wt = warp / kw;
    const int u0 = units * wk / kw, u1 = units * (wk + 1) / kw;
    const int64_t w_pitch = F == kBf16 ? 2ll * p.K : p.K / 2;
    const int64_t s_pitch = F == kMx ? p.K / 32 : p.K / 16;
    const int64_t w_rows = kSwiglu ? 2ll * p.N : p.N;
    const int row_bytes = static_cast<int>(w_pitch);

    // Weight row of the tile's row r; columns past the last read the last one's.
    const auto weight_row = [&](int item, int r) {
        const int e = ch.expert[item / groups], tile = item % groups * group + wt;
        if (kSwiglu) {
            const int n = min(tile * 8 + (r & 7), p.N - 1);
            return e * w_rows + n + (r >= 8 ? p.N : 0);
        }
        return e * w_rows + min(tile * 16 + r, p.N - 1);
    };
    // A stage: lane copies 32 bytes of row lane / 2; lanes 0..15 the scale words of row lane.
    const uint8_t *wp = nullptr, *sp = nullptr;
    const auto open = [&](int item) {
        wp = p.w + weight_row(item, lane >> 1) * w_pitch;
        if constexpr (F != kBf16) sp = p.scales + weight_row(item, lane & 15) * s_pitch;
    };
    const uint32_t ring_a = smem_u32(ring);
    const auto issue = [&](int unit, int slot) {
        const uint32_t dst = ring_a + slot * C::kStage;
        const int at = unit * kRowBytes + (lane & 1) * 32;
        const uint32_t d = dst + (lane >> 1) * C::kPitch + (lane & 1) * 32;
        // A piece past the row's end becomes zeros; its address is not read.
        cp_async16(d, wp + (at < row_bytes ? at : 0), at < row_bytes);
        cp_async16(d + 16, wp + (at + 16 < row_bytes ? at + 16 : 0), at + 16 < row_bytes);
        if constexpr (F != kBf16) {
            if (lane < 16) {
                constexpr int kBytes = F == kMx ? 4 : 8;
                const uint32_t sd = dst + 16 * C::kPitch + lane * 4 * C::kScaleWords;
                const uint8_t *src = sp + unit * kBytes;
                const int have = min(static_cast<int>(s_pitch) - unit * kBytes, kBytes);     // bytes of the row here
                const int off = kShift ? static_cast<int>(reinterpret_cast<uintptr_t>(src) & 3) : 0;
#pragma unroll
                for (int i = 0; i < C::kScaleWords; ++i)     // words that hold a byte of the row
                    if (4 * i < off + have) cp_async4(sd + 4 * i, src - off + 4 * i);
            }
        }
    };
    Cursor fetch = {first, u0};
    const auto fetch_next = [&](int slot) {
        if (u0 < u1 && fetch.item < last) {
            if (fetch.unit == u0) open(fetch.item);
            issue(fetch.unit, slot);
            if (++fetch.unit == u1) {
                fetch.unit = u0;
                ++fetch.item;
            }
        }
        cp_commit();
    };
#pragma unroll 1
    for (int i = 0; i < C::kDepth - 1; ++i) fetch_next(i);

    int slot = 0, slot_in = C::kDepth - 1, buf = 0, chunk = -1, n_tok = 0;
    uint32_t any_bad = 0;
    for (int item = first; item < last; ++item) {
        if (item / groups != chunk) {
            chunk = item / groups;
            n_tok = ch.first[chunk + 1] - ch.first[chunk];
            __syncthreads();                      // sums of the last item are read with the old exponents
            stage_x<F>(p, ch.order + ch.first[chunk], n_tok, xs, pitch, exps);
        }
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t bad[2] = {0, 0};
        const uint32_t xa = smem_u32(xs) + min(g, n_tok - 1) * pitch + t4 * 16;
#pragma unroll 1
        for (int unit = u0; unit < u1; ++unit) {
            cp_wait<C::kDepth - 2>();
            __syncwarp();                         // all lanes' copies; and the slot to fill is read
            fetch_next(slot_in);
            const uint32_t at = ring_a + slot * C::kStage;
            if constexpr (F == kBf16) {
                const uint4 a = lds128(at + g * C::kPitch + t4 * 16), b = lds128(at + (g + 8) * C::kPitch + t4 * 16);
                const uint4 v = lds128(xa + unit * 64);
                mma16816<false>(acc, a.x, b.x, a.y, b.y, v.x, v.y);
                mma16816<false>(acc, a.z, b.z, a.w, b.w, v.z, v.w);
            } else {
                const int blocks = min((p.K - unit * 128) >> 5, 4);      // of 32 k in this stage
                // Scale bytes of rows g and g + 8, in order.
                uint32_t sw[2][F == kNv ? 2 : 1];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint32_t sa = at + 16 * C::kPitch + (g + 8 * r) * 4 * C::kScaleWords;
                    if constexpr (kShift) {
                        const int64_t row = weight_row(item, g + 8 * r);
                        const uint32_t off = 8 * (reinterpret_cast<uintptr_t>(p.scales + row * s_pitch + unit * (F == kMx ? 4 : 8)) & 3);
                        uint32_t q[C::kScaleWords];
#pragma unroll
                        for (int i = 0; i < C::kScaleWords; ++i) q[i] = lds32(sa + 4 * i);
#pragma unroll
                        for (int i = 0; i + 1 < C::kScaleWords; ++i) sw[r][i] = __funnelshift_r(q[i], q[i + 1], off);
                    } else {
#pragma unroll
                        for (int i = 0; i < (F == kNv ? 2 : 1); ++i) sw[r][i] = lds32(sa + 4 * i);
                    }
                    if (blocks < 4) {             // bytes past the row's end
                        if constexpr (F == kMx) {
                            sw[r][0] &= (1u << (8 * blocks)) - 1;
                        } else {
                            const int bytes = 2 * blocks;
                            sw[r][0] &= bytes >= 4 ? 0xFFFFFFFFu : (1u << (8 * bytes)) - 1;
                            sw[r][1] &= bytes <= 4 ? 0u : (1u << (8 * (bytes - 4))) - 1;
                        }
                    }
                    if constexpr (F == kMx)       // 253 and more
                        bad[r] |= ((sw[r][0] & 0x7F7F7F7Fu) + 0x03030303u) & sw[r][0] & 0x80808080u;
                    else                          // NaN
                        bad[r] |= (((sw[r][0] & 0x7F7F7F7Fu) + 0x01010101u) | ((sw[r][1] & 0x7F7F7F7Fu) + 0x01010101u)) & 0x80808080u;
                }
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    if (b >= blocks) break;
                    uint32_t a[4], c[4];
                    decode8(lds32(at + g * C::kPitch + 16 * b + 4 * t4), a);
                    decode8(lds32(at + (g + 8) * C::kPitch + 16 * b + 4 * t4), c);
                    const uint4 v = lds128(xa + unit * 256 + b * 64);
                    if constexpr (F == kMx) {
                        float d[4] = {0.f, 0.f, 0.f, 0.f};
                        mma16816<true>(d, a[0], c[0], a[1], c[1], v.x, v.y);
                        mma16816<true>(d, a[2], c[2], a[3], c[3], v.z, v.w);
                        const float s0 = __uint_as_float((sw[0][0] >> (8 * b) & 0xFFu) << 23) * 0x1p-31f;
                        const float s1 = __uint_as_float((sw[1][0] >> (8 * b) & 0xFFu) << 23) * 0x1p-31f;
                        acc[0] = fmaf(s0, d[0], acc[0]);
                        acc[1] = fmaf(s0, d[1], acc[1]);
                        acc[2] = fmaf(s1, d[2], acc[2]);
                        acc[3] = fmaf(s1, d[3], acc[3]);
                    } else {
                        const int sh = 16 * (b & 1) + 8 * (t4 >> 1);      // this lane's half of the block
                        const uint32_t s0 = e4m3_pair(sw[0][b >> 1] >> sh), s1 = e4m3_pair(sw[1][b >> 1] >> sh);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            a[i] = hmul2(a[i], s0);
                            c[i] = hmul2(c[i], s1);
                        }
                        mma16816<true>(acc, a[0], c[0], a[1], c[1], v.x, v.y);
                        mma16816<true>(acc, a[2], c[2], a[3], c[3], v.z, v.w);
                    }
                }
            }
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
        constexpr int kOuts = (kSwiglu ? 8 : 16) * kTok;
        for (int i = tid; i < group * kOuts; i += kThreads) {
            const int tile = i / kOuts, r = i % kOuts / kTok, t = i % kTok;
            const int n = (item % groups * group + tile) * tile_cols + r;
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
            const int64_t o = static_cast<int64_t>(ch.order[ch.first[chunk] + t]) * p.N + n;
            if (kSwiglu || p.out_bf16) static_cast<__nv_bfloat16 *>(p.out)[o] = __float2bfloat16_rn(v);
            else static_cast<float *>(p.out)[o] = v;
        }
        buf ^= 1;
    }
    cp_wait<0>();
    if constexpr (F != kBf16)
        if (__any_sync(0xffffffffu, any_bad != 0) && lane == 0) set_status(p.status, MOE_ERR_DATA);
}

// out[t, n] = sum_j w[t, j] * y[t k + j, n] over the slots with a valid expert, in ascending j.
template <typename T>
__global__ void weigh_kernel(const float *y, const int32_t *ids, const float *w, int T_, int k, int N, int E, T *out) {
    const int n = blockIdx.x * blockDim.x + threadIdx.x;
    for (int t = blockIdx.y; t < T_ && n < N; t += gridDim.y) {
        float acc = 0.f;
        for (int j = 0; j < k; ++j) {
            const int s = t * k + j;
            if (static_cast<unsigned>(__ldg(ids + s)) >= static_cast<unsigned>(E)) continue;
            acc = fmaf(__ldg(w + s), __ldg(y + static_cast<int64_t>(s) * N + n), acc);
        }
        if constexpr (sizeof(T) == 2) out[static_cast<int64_t>(t) * N + n] = __float2bfloat16_rn(acc);
        else out[static_cast<int64_t>(t) * N + n] = acc;
    }
}

constexpr int kMaxSmem = 232448;

template <int F, bool kSwiglu, bool kShift>
moe_status launch(Params p, cudaStream_t stream, int num_sms) {
    using C = Fmt<F>;
    p.k_pad = (p.K + C::kUnit - 1) / C::kUnit * C::kUnit;
    const int units = p.k_pad / C::kUnit;
    p.kw = 1;
    while (p.kw < kWarps && p.kw < units) p.kw *= 2;
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
    kernel<<<num_sms, kThreads, bytes, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
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
        return m.swiglu ? mv::launch<mv::kBf16, true, false>(p, stream, num_sms)
                        : mv::launch<mv::kBf16, false, false>(p, stream, num_sms);
    const bool nv = m.format == Matvec::kNv;
    // Scale rows at 4-byte addresses are copied as they are; others as the words around them.
    const bool shift = (m.K / (nv ? 16 : 32)) % 4 != 0 || reinterpret_cast<uintptr_t>(m.scales) % 4 != 0;
    if (shift)
        return nv ? m.swiglu ? mv::launch<mv::kNv, true, true>(p, stream, num_sms)
                             : mv::launch<mv::kNv, false, true>(p, stream, num_sms)
                  : m.swiglu ? mv::launch<mv::kMx, true, true>(p, stream, num_sms)
                             : mv::launch<mv::kMx, false, true>(p, stream, num_sms);
    return nv ? m.swiglu ? mv::launch<mv::kNv, true, false>(p, stream, num_sms)
                         : mv::launch<mv::kNv, false, false>(p, stream, num_sms)
              : m.swiglu ? mv::launch<mv::kMx, true, false>(p, stream, num_sms)
                         : mv::launch<mv::kMx, false, false>(p, stream, num_sms);
}

moe_status launch_weigh(const float *y, const int32_t *ids, const float *w, int T, int k, int N, int E, void *out,
                        int out_bf16, cudaStream_t stream) {
    if (T == 0 || N == 0) return MOE_OK;
    const dim3 grid((N + 127) / 128, T < 65535 ? T : 65535);
    if (out_bf16) mv::weigh_kernel<<<grid, 128, 0, stream>>>(y, ids, w, T, k, N, E, static_cast<__nv_bfloat16 *>(out));
    else mv::weigh_kernel<<<grid, 128, 0, stream>>>(y, ids, w, T, k, N, E, static_cast<float *>(out));
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
