// Grouped product of 4-bit activations with 4-bit expert weights (W4A4), sm_103a:
//
//   out[r, n] = sum_k a[r, k] * w_e[n, k]     for every row r of band e,
//
// both operands e2m1 codes under block scales: MXFP4 (E8M0 per 32) or NVFP4
// (E4M3 per 16, times an f32 scale a tensor).  The tensor core takes the codes
// and the scales as they are (tcgen05.mma kind::mxf4 / kind::mxf4nvf4 with
// block scaling, f32 accumulators), so there is no decode at all: the weights
// go from global memory to shared memory by TMA and no thread touches them.
//
//  * Weights are the MMA's A operand (128 weight rows), the band's token rows
//    its B operand (N = 16..192), as in the W4A16 product: a decode band of one
//    row wastes no weight traffic.
//  * One K stage is 256 k: 128 bytes a row, the 128-byte swizzle TMA writes and
//    the MMA reads; four MMAs of 64 k.
//  * Block scales have to sit in tensor memory as 32-lane atoms (word of row m
//    at lane m % 32, column m / 32; a word holds four consecutive scales).
//    Two loader warps fetch the scale bytes row by row with a register prefetch
//    of kPrefetch stages, write the atoms to shared memory (a 4 x 4 word
//    transpose per lane, one 16-byte store), and the issuer copies them with
//    tcgen05.cp in front of the stage's MMAs.  So scales keep the layout the
//    rest of the library uses, and tokens may start at any row.
//  * Accumulators are double-buffered (2 x 192 columns): the epilogue warps of
//    one item run under the next item's MMAs.  A band's rows are cut into equal
//    chunks of at most 192 (96 with SwiGLU) tokens, multiples of 16.
//  * SwiGLU: an item holds 128 gate rows and the 128 matching up rows as two
//    MMAs into two column ranges, so a thread has g and u of one output column
//    at the same token and no shuffle pairs them.  The 32 lanes of a warp hold
//    32 consecutive h columns, one MX block: h is quantised in registers (block
//    maximum by redux / half-warp redux, an 8 x 8 nibble transpose by three
//    shuffles) and leaves the SM as 4-bit codes, never as bf16 or f32.
//  * Persistent CTAs, one per SM, over a static list of (expert, chunk, tile).
//  * Every wait is bounded; see wait_bounded.
#include <atomic>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <stdint.h>

#include "device_common.cuh"
#include "fp4_common.cuh"
#include "launch.h"

namespace moe {
namespace fp4 {

constexpr int kProducerWarp = 0, kIssuerWarp = 1;
constexpr int kLoaders = 4;                    // scale-loader warps an operand, on stages in turn
constexpr int kWScaleWarp = 2, kAScaleWarp = kWScaleWarp + kLoaders;
constexpr int kEpilogueWarp = kAScaleWarp + kLoaders;
constexpr int kThreads = 32 * (kEpilogueWarp + 4);
constexpr int kMaxE = 1024;
constexpr int kTileN = 128;                    // weight rows a tile (MMA M)
constexpr int kStageBytesRow = 128;            // 256 k
constexpr int kStageK = 256;
constexpr int kMaxStages = 12;
constexpr int kPrefetch = 2;                   // stages of scale bytes a loader holds in registers
constexpr int kAccCols = 192;                  // columns of one accumulator buffer
constexpr int kSfCol0 = 2 * kAccCols;          // scale atoms, two sets of 64 columns
constexpr int kSfSetCols = 64;
constexpr int kTmemCols = 512;
constexpr int kAtomBytes = 512;

constexpr int kRingBytes = 208 * 1024;
constexpr int kOffRow = kRingBytes;
constexpr int kOffItem = kOffRow + (kMaxE + 1) * 4;
constexpr int kOffBars = (kOffItem + (kMaxE + 1) * 4 + 7) & ~7;
constexpr int kNumBars = 3 * kMaxStages + 4 + 1;
constexpr int kOffMisc = kOffBars + kNumBars * 8;
constexpr int kSmemBytes = kOffMisc + 64 + 1024;
static_assert(kSmemBytes <= 232448, "shared memory budget");
static_assert(kSfCol0 + 2 * kSfSetCols <= kTmemCols, "tensor memory budget");

struct Params {
    const uint8_t *w_scales, *a_scales;
    const float *w_scale_2, *a_scale_2, *h_scale_2;
    const int32_t *group_sizes;
    void *out;               // f32 or bf16 [rows, N]; SwiGLU: codes [rows, I / 2]
    uint8_t *out_scales;     // SwiGLU: [rows, I / block]
    int *status;
    int rows, K, N, E;       // N: weight rows an expert (2 I with SwiGLU)
    int I;
    int out_bf16;
    int n_tiles;
    int scale_row;           // scale bytes a row of K: K / 32 or K / 16
    int w_vec, a_vec;        // a stage's scale bytes of a row load as one aligned vector
    uint64_t wait_limit_ns;
};

template <bool kNv, bool kSwiglu>
struct Shape {
    static constexpr int MT = kSwiglu ? 2 : 1;             // weight tiles an item
    static constexpr int NT = kSwiglu ? 96 : 192;          // tokens an item, at most
    static constexpr int W = kNv ? 4 : 2;                  // scale words a row and stage
    static constexpr int NA = kSwiglu ? 1 : 2;             // token atoms of 128 rows
    static constexpr int AR = NT / 32;                     // token rows a lane of the scale loader
    static constexpr int kABytes = MT * kTileN * kStageBytesRow;
    static constexpr int kSfaBytes = MT * W * kAtomBytes;
    static constexpr int kSfBytes = kSfaBytes + NA * W * kAtomBytes;
    static constexpr int kAccStep = kSwiglu ? 96 : 0;      // columns from the gate to the up sums
    static_assert(kSfBytes / kAtomBytes * 4 <= kSfSetCols, "scale columns of one stage");
};

// ------------------------------------------------------- block-scaled MMA

// Instruction descriptor of the block-scaled 4-bit kinds: e2m1 A and B (format
// 1), both K-major, M = 128; scale type E8M0 (1) or E4M3 (0); the ids pick the
// scale byte pair inside a word (MXFP4: 0 or 2).
template <bool kNv>
__device__ __forceinline__ uint32_t idesc_fp4(uint32_t n, uint32_t sf_id) {
    return (sf_id << 4) | (1u << 7) | (1u << 10) | ((n >> 3) << 17) | ((kNv ? 0u : 1u) << 23) |
           ((128u >> 4) << 24) | (sf_id << 29);
}

template <bool kNv>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
    if constexpr (kNv)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, "
            "[%5], [%6], p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa),
            "r"(sfb)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, "
            "[%5], [%6], p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa),
            "r"(sfb)
            : "memory");
}

// One 512-byte scale atom (32 rows of 16 bytes, contiguous) from shared memory
// to 4 tensor-memory columns, the same 32 lanes for all four lane quarters.
__device__ __forceinline__ void copy_atom(uint32_t taddr, uint32_t saddr) {
    uint64_t d = (saddr & 0x3FFFFu) >> 4;
    d |= static_cast<uint64_t>(16u >> 4) << 16;
    d |= static_cast<uint64_t>(128u >> 4) << 32;   // 8-row groups 128 bytes apart, no swizzle
    d |= 1ull << 46;
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}

// ------------------------------------------------------------------ items

struct Item {
    int e, row0, nvalid, nt, n0;
};

// Tokens an item of a band of n rows: equal chunks of at most `most`, rounded up to
// 16 (never past `most`, a multiple of 16, so no chunk comes out empty).
__device__ __forceinline__ int chunk_rows(int n, int most) {
    const int nch = (n + most - 1) / most;
    return ((n + nch - 1) / nch + 15) & ~15;
}

template <int kMost>
__device__ __forceinline__ Item decode_item(int j, const int *roff, const int *ioff, int E, int n_tiles) {
    int lo = 0, hi = E - 1;   // last e with ioff[e] <= j (its band is non-empty)
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (ioff[mid] <= j) lo = mid; else hi = mid - 1;
    }
    Item it;
    it.e = lo;
    const int n = roff[lo + 1] - roff[lo];
    const int cr = chunk_rows(n, kMost);
    const int r = j - ioff[lo];
    const int ch = r / n_tiles;
    it.n0 = (r - ch * n_tiles) * kTileN;
    const int t0 = ch * cr;
    it.nvalid = min(cr, n - t0);
    it.nt = (it.nvalid + 15) & ~15;
    it.row0 = roff[lo] + t0;
    return it;
}

// Position in the stage ring.
struct Ring {
    uint32_t slot = 0, phase = 0;
    __device__ __forceinline__ void next(uint32_t n, uint32_t by = 1) {
        for (slot += by; slot >= n; slot -= n) phase ^= 1u;
    }
};

// Items of this CTA times stages, in order.
template <int kMost>
struct Cursor {
    int j, ks;
    Item it;
    __device__ __forceinline__ bool valid(int total) const { return j < total; }
    __device__ __forceinline__ void start(int total, const int *roff, const int *ioff, int E, int n_tiles) {
        j = blockIdx.x;
        ks = 0;
        if (j < total) it = decode_item<kMost>(j, roff, ioff, E, n_tiles);
    }
    __device__ __forceinline__ void next(int total, int k_stages, const int *roff, const int *ioff, int E,
                                         int n_tiles, int by = 1) {
        ks += by;
        if (ks < k_stages) return;
        for (; ks >= k_stages; ks -= k_stages) j += gridDim.x;
        if (j < total) it = decode_item<kMost>(j, roff, ioff, E, n_tiles);
    }
};

// ---------------------------------------------------------- scale loaders

// The W scale words of one row and stage: bytes [first, first + 4 W) of a row of
// `scale_row` bytes, zeros past its end (2^-127 or 0: finite, times zero codes).
template <int W>
__device__ __forceinline__ void load_words(const uint8_t *row, int first, int scale_row, int vec,
                                           uint32_t (&w)[W]) {
    if (vec) {
        if constexpr (W == 2) {
            const uint2 v = __ldg(reinterpret_cast<const uint2 *>(row + first));
            w[0] = v.x; w[1] = v.y;
        } else {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(row + first));
            w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < W; ++i) {
        w[i] = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int k = first + 4 * i + b;
            if (k < scale_row) w[i] |= static_cast<uint32_t>(__ldg(row + k)) << (8 * b);
        }
    }
}

// A byte the format does not allow: E8M0 255; E4M3 NaN or a set sign bit (the
// block-scaled MMA takes unsigned scales).
template <bool kNv>
__device__ __forceinline__ bool bad_word(uint32_t w) {
    if constexpr (kNv) return ((w & 0x80808080u) | __vcmpeq4(w, 0x7F7F7F7Fu)) != 0;
    else return __vcmpeq4(w, 0xFFFFFFFFu) != 0;
}

// Body of scale-loader warp `part` of `parts`, which takes every parts-th stage.
// parts <= n_stages: a loader that waits for the slot of stage s has seen stage s -
// parts - n_stages consumed, so the slot's barrier is at most one phase behind and
// its parity is unambiguous.  kWeights: the weight tiles' scales (4 MT rows
// a lane), else the tokens' (AR rows a lane).
template <bool kNv, bool kSwiglu, bool kWeights>
__device__ __forceinline__ void load_scales(const Params &p, uint8_t *sf_ring, uint32_t n_stages, int total,
                                            const int *roff, const int *ioff, uint64_t *sf_full,
                                            uint64_t *empty, volatile int *abort_flag, int part, int parts) {
    using S = Shape<kNv, kSwiglu>;
    constexpr int R = kWeights ? 4 * S::MT : S::AR;
    constexpr int W = S::W;
    const int lane = threadIdx.x & 31;
    const int k_stages = (p.K + kStageK - 1) / kStageK;
    const int vec = kWeights ? p.w_vec : p.a_vec;
    uint32_t buf[kPrefetch][R][W] = {};
    bool bad = false;
    Cursor<S::NT> ld, st;
    ld.start(total, roff, ioff, p.E, p.n_tiles);
    if (part) ld.next(total, k_stages, roff, ioff, p.E, p.n_tiles, part);
    st = ld;

    auto fetch = [&](uint32_t (&b)[R][W]) {
        const int first = ld.ks * 4 * W;
#pragma unroll
        for (int q = 0; q < R; ++q) {
            // Rows past the tile's or the chunk's end read its last row again
            // (their sums are never stored): nothing here waits for the load.
            int64_t row;
            if constexpr (kWeights) {
                const int cols = kSwiglu ? p.I : p.N;
                row = static_cast<int64_t>(ld.it.e) * p.N + (q >= 4 ? p.I : 0) +
                      min(ld.it.n0 + lane + 32 * (q & 3), cols - 1);
            } else {
                if (32 * q >= ld.it.nt) continue;
                row = ld.it.row0 + min(lane + 32 * q, ld.it.nvalid - 1);
            }
            load_words<W>((kWeights ? p.w_scales : p.a_scales) + row * p.scale_row, first, p.scale_row, vec,
                          b[q]);
        }
        ld.next(total, k_stages, roff, ioff, p.E, p.n_tiles, parts);
    };

#pragma unroll
    for (int d = 0; d < kPrefetch; ++d)
        if (ld.valid(total)) fetch(buf[d]);

    Ring r;
    if (part) r.next(n_stages, part);
    bool ok = true;
    while (ok && st.valid(total)) {
#pragma unroll
        for (int d = 0; d < kPrefetch; ++d) {
            if (!ok || !st.valid(total)) break;
            ok = warp_wait_bounded(&empty[r.slot], r.phase ^ 1u, abort_flag, p.status, p.wait_limit_ns);
            if (!ok) break;
            uint8_t *dst = sf_ring + r.slot * S::kSfBytes + (kWeights ? 0 : S::kSfaBytes) + lane * 16;
#pragma unroll
            for (int q = 0; q < R; ++q) {
                if (!kWeights && 32 * q >= st.it.nt) continue;
#pragma unroll
                for (int i = 0; i < W; ++i) bad |= bad_word<kNv>(buf[d][q][i]);
            }
            constexpr int ATOMS = (R + 3) / 4;
#pragma unroll
            for (int a = 0; a < ATOMS; ++a)
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    uint4 v;
                    v.x = buf[d][4 * a][i];
                    v.y = 4 * a + 1 < R ? buf[d][4 * a + 1 < R ? 4 * a + 1 : 0][i] : 0u;
                    v.z = 4 * a + 2 < R ? buf[d][4 * a + 2 < R ? 4 * a + 2 : 0][i] : 0u;
                    v.w = 4 * a + 3 < R ? buf[d][4 * a + 3 < R ? 4 * a + 3 : 0][i] : 0u;
                    // weights: atom (tile, word); tokens: atoms of one word adjacent
                    const int atom = kWeights ? a * W + i : i * S::NA + a;
                    *reinterpret_cast<uint4 *>(dst + atom * kAtomBytes) = v;
                }
            // The atoms are read by tcgen05.cp (the async proxy).
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&sf_full[r.slot]);
            r.next(n_stages, parts);
            st.next(total, k_stages, roff, ioff, p.E, p.n_tiles, parts);
            if (ld.valid(total)) fetch(buf[d]);
        }
    }
    if (bad) set_status(p.status, MOE_ERR_DATA);
}

// -------------------------------------------------------------- epilogues

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&v)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
                   "=r"(v[7])
                 : "r"(taddr));
}

// f32 / bf16 sums: lane = weight row, so a warp stores 32 consecutive columns
// of one token row at a time.
__device__ __forceinline__ void store_plain(const Params &p, const Item &it, uint32_t acc, int n, float scale,
                                            uint64_t *acc_empty) {
    const int lane = threadIdx.x & 31;
    for (int c = 0; c < it.nt; c += 16) {
        uint32_t v[16];
        __syncwarp();
        tmem_ld16(acc + c, v);
        tmem_ld_wait();
        if (c + 16 >= it.nt) {      // the sums are in registers: release the buffer
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acc_empty);
        }
        if (n < p.N) {
            const size_t off = static_cast<size_t>(it.row0 + c) * p.N + n;
            const int left = it.nvalid - c;
            if (p.out_bf16) {
                __nv_bfloat16 *o = reinterpret_cast<__nv_bfloat16 *>(p.out) + off;
#pragma unroll
                for (int t = 0; t < 16; ++t)
                    if (t < left) o[static_cast<size_t>(t) * p.N] = __float2bfloat16_rn(__uint_as_float(v[t]) * scale);
            } else {
                float *o = reinterpret_cast<float *>(p.out) + off;
#pragma unroll
                for (int t = 0; t < 16; ++t)
                    if (t < left) o[static_cast<size_t>(t) * p.N] = __uint_as_float(v[t]) * scale;
            }
        }
    }
}

// SwiGLU sums -> h = silu(g) * u in f32 -> 4-bit codes and block scales.  The
// warp's lanes are 32 consecutive h columns; n0w is the first of them.
template <bool kNv>
__device__ __forceinline__ void store_swiglu(const Params &p, const Item &it, uint32_t acc, int n0w,
                                             float scale, float h_scale, uint64_t *acc_empty) {
    const int lane = threadIdx.x & 31;
    const int t8 = lane & 7, q = lane >> 3;
    const float g6 = 6.0f * h_scale;
    for (int c = 0; c < it.nt; c += 8) {
        uint32_t g[8], u[8];
        __syncwarp();
        tmem_ld8(acc + c, g);
        tmem_ld8(acc + Shape<kNv, true>::kAccStep + c, u);
        tmem_ld_wait();
        if (c + 8 >= it.nt) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acc_empty);
        }
        if (n0w >= p.I) continue;          // warp-uniform: I is a multiple of 32
        float h[8];
        uint32_t my_byte = 0;
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            h[t] = silu_f32(__uint_as_float(g[t]) * scale) * (__uint_as_float(u[t]) * scale);
            const uint32_t mag = __float_as_uint(h[t]) & 0x7FFFFFFFu;
            uint32_t byte;
            float inv;
            if constexpr (kNv) {
                uint32_t m = mag;
#pragma unroll
                for (int d = 8; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
                byte = nv_scale_byte(m, g6);
                inv = nv_inverse(byte, h_scale);
                h[t] = byte == 0x7Fu ? 0.0f : h[t] * inv;
            } else {
                byte = mx_scale_byte(__reduce_max_sync(0xffffffffu, mag));
                h[t] = byte == 255u ? 0.0f : h[t] * mx_inverse(byte);
            }
            if (t == t8) my_byte = byte;
        }
        // Nibble t of w: this lane's column at token c + t.  Transposed over the
        // eight lanes of a group: nibble i becomes column 8 q + i at token c + t8.
        uint32_t w = e2m1x8(h);
#pragma unroll
        for (int m = 4; m > 0; m >>= 1) {
            const uint32_t low = m == 4 ? 0x0000FFFFu : m == 2 ? 0x00FF00FFu : 0x0F0F0F0Fu;
            const uint32_t o = __shfl_xor_sync(0xffffffffu, w, m);
            w = (lane & m) ? ((w & ~low) | ((o >> (4 * m)) & low)) : ((w & low) | ((o & low) << (4 * m)));
        }
        if (c + t8 < it.nvalid) {
            const size_t row = static_cast<size_t>(it.row0 + c + t8);
            uint8_t *codes = static_cast<uint8_t *>(p.out) + row * (p.I / 2) + n0w / 2;
            *reinterpret_cast<uint32_t *>(codes + 4 * q) = w;
            if constexpr (kNv) {
                // lanes 0..15 have the first block's byte, 16..31 the second's
                if ((q & 1) == 0) p.out_scales[row * (p.I / 16) + n0w / 16 + (q >> 1)] = my_byte;
            } else {
                if (q == 0) p.out_scales[row * (p.I / 32) + n0w / 32] = my_byte;
            }
        }
    }
}

// ------------------------------------------------------------------ kernel

template <bool kNv, bool kSwiglu>
__global__ void __launch_bounds__(kThreads, 1)
    fp4_gemm_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_a64,
                    const __grid_constant__ CUtensorMap tm_a16, const Params p) {
    using S = Shape<kNv, kSwiglu>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    int *roff = reinterpret_cast<int *>(smem + kOffRow);
    int *ioff = reinterpret_cast<int *>(smem + kOffItem);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kOffBars);   // TMA -> issuer
    uint64_t *sf_full = full + kMaxStages;                            // scale loaders -> issuer
    uint64_t *empty = sf_full + kMaxStages;                           // MMA commit -> loaders
    uint64_t *acc_full = empty + kMaxStages;                          // MMA commit -> epilogue
    uint64_t *acc_empty = acc_full + 2;                               // epilogue -> issuer
    uint64_t *final_bar = acc_empty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + kOffMisc + 8);
    int *bad_flag = reinterpret_cast<int *>(smem + kOffMisc + 16);
    int *nt_slot = reinterpret_cast<int *>(smem + kOffMisc + 24);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int E = p.E;

    // Row and item offsets from the group sizes (64-bit sums: sizes that wrap 32
    // bits are caught).
    for (int e = tid; e < E; e += kThreads) roff[e] = __ldg(p.group_sizes + e);
    if (tid == 0) *abort_flag = 0;
    __syncthreads();
    if (warp == 0) {
        long long rsum = 0, isum = 0;
        int most = 0;
        bool neg = false;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            const int n = e < E ? roff[e] : 0;
            neg |= n < 0;
            long long rows = n > 0 ? n : 0, items = 0;
            if (rows > 0) {
                const int cr = chunk_rows(static_cast<int>(min(rows, static_cast<long long>(p.rows))), S::NT);
                most = max(most, min(cr, S::NT));
                items = ((rows + S::NT - 1) / S::NT) * p.n_tiles;
            }
            long long r = rows, i = items;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const long long ro = __shfl_up_sync(0xffffffffu, r, d), io = __shfl_up_sync(0xffffffffu, i, d);
                if (lane >= d) { r += ro; i += io; }
            }
            if (e < E) {
                // Stored as ints; used only when the totals check out below.
                roff[e] = static_cast<int>(rsum + r - rows);
                ioff[e] = static_cast<int>(isum + i - items);
            }
            rsum += __shfl_sync(0xffffffffu, r, 31);
            isum += __shfl_sync(0xffffffffu, i, 31);
        }
        most = __reduce_max_sync(0xffffffffu, most);
        const bool bad = __any_sync(0xffffffffu, neg) || rsum != p.rows || isum > INT32_MAX;
        if (lane == 0) {
            roff[E] = static_cast<int>(rsum);
            ioff[E] = static_cast<int>(isum);
            *bad_flag = bad;
            *nt_slot = most;
            if (bad) set_status(p.status, MOE_ERR_DATA);
        }
    }
    __syncthreads();
    if (*bad_flag) return;
    const int total = ioff[E];
    if (static_cast<int>(blockIdx.x) >= total) return;

    // Stage layout: as many stages as fit with the widest chunk of this call.
    const int nt_max = *nt_slot;
    const uint32_t b_rows = nt_max <= 32 ? nt_max : (nt_max + 63) & ~63;
    const uint32_t b_bytes = b_rows * kStageBytesRow;
    const uint32_t n_stages = min(static_cast<uint32_t>(kMaxStages), kRingBytes / (S::kABytes + b_bytes + S::kSfBytes));
    uint8_t *b_ring = smem + n_stages * S::kABytes;
    uint8_t *sf_ring = b_ring + n_stages * b_bytes;
    const int k_stages = (p.K + kStageK - 1) / kStageK;

    if (warp == kProducerWarp) tmem_alloc(tmem_slot, kTmemCols);
    if (tid == 0) {
        for (uint32_t s = 0; s < n_stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&sf_full[s], 2);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 4);
        }
        mbar_init(final_bar, 1);
        mbar_fence_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint64_t lim = p.wait_limit_ns;

    if (warp == kProducerWarp) {
        const bool leader = elect_one();
        if (leader) {
            tma_prefetch_map(&tm_w);
            tma_prefetch_map(&tm_a64);
            tma_prefetch_map(&tm_a16);
        }
        const uint32_t a_base = smem_u32(smem), b_base = smem_u32(b_ring);
        Ring r;
        uint32_t issued = 0;
        bool ok = true;
        for (int j = blockIdx.x; ok && j < total; j += gridDim.x) {
            const Item it = decode_item<S::NT>(j, roff, ioff, E, p.n_tiles);
            // Token rows in 64-row boxes; a last part of at most 32 rows in 16-row
            // boxes (rows past the chunk belong to the next one; their columns are
            // not stored).
            const int part = it.nt & 63;
            const int n64 = (it.nt >> 6) + (part > 32), n16 = part > 32 ? 0 : part >> 4;
            const uint32_t bytes = S::kABytes + (n64 * 64 + n16 * 16) * kStageBytesRow;
            const int wrow = it.e * p.N + it.n0;
            for (int ks = 0; ks < k_stages; ++ks) {
                ok = warp_wait_bounded(&empty[r.slot], r.phase ^ 1u, abort_flag, p.status, lim);
                if (!ok) break;
                uint64_t *bar = &full[r.slot];
                const uint32_t a_dst = a_base + r.slot * S::kABytes, b_dst = b_base + r.slot * b_bytes;
                const int x = ks * kStageBytesRow;
                if (leader) {
                    mbar_arrive_expect_tx(bar, bytes);
                    tma_load_2d(a_dst, &tm_w, x, wrow, bar);
                    if constexpr (kSwiglu) tma_load_2d(a_dst + kTileN * kStageBytesRow, &tm_w, x, wrow + p.I, bar);
                    for (int i = 0; i < n64; ++i)
                        tma_load_2d(b_dst + i * 64 * kStageBytesRow, &tm_a64, x, it.row0 + i * 64, bar);
                    for (int i = 0; i < n16; ++i)
                        tma_load_2d(b_dst + (n64 * 64 + i * 16) * kStageBytesRow, &tm_a16, x,
                                    it.row0 + n64 * 64 + i * 16, bar);
                }
                __syncwarp();
                ++issued;
                r.next(n_stages);
            }
        }
        if (!ok && lane == 0) {   // drain: every issued copy must land before the CTA exits
            for (uint32_t i = issued > n_stages ? issued - n_stages : 0; i < issued; ++i)
                wait_bounded(&full[i % n_stages], (i / n_stages) & 1u, nullptr, p.status, lim);
        }
    } else if (warp == kIssuerWarp) {
        // The whole warp runs the loop, so that addresses and descriptors stay in
        // the warp-uniform registers the tcgen05 instructions take; one elected
        // lane (always the same) issues.  A single-lane loop issued a stage in
        // 1,600 cycles, four times what its MMAs take.
        const bool leader = elect_one();
        const uint32_t a_base = smem_u32(smem), b_base = smem_u32(b_ring), sf_base = smem_u32(sf_ring);
        const int last_steps = (p.K - (k_stages - 1) * kStageK + 63) >> 6;
        Ring r;
        uint32_t buf = 0, acc_phase = 1, set = 0;
        bool ok = true;
        for (int j = blockIdx.x; ok && j < total; j += gridDim.x) {
            const Item it = decode_item<S::NT>(j, roff, ioff, E, p.n_tiles);
            const uint32_t id0 = idesc_fp4<kNv>(it.nt, 0), id2 = idesc_fp4<kNv>(it.nt, kNv ? 0 : 2);
            const bool two = S::NA == 2 && it.nt > 128;
            const uint32_t d = tmem + buf * kAccCols;
            ok = warp_wait_bounded(&acc_empty[buf], acc_phase, abort_flag, p.status, lim);
            for (int ks = 0; ok && ks < k_stages; ++ks) {
                ok = warp_wait_bounded(&full[r.slot], r.phase, abort_flag, p.status, lim) &&
                     warp_wait_bounded(&sf_full[r.slot], r.phase, abort_flag, p.status, lim);
                if (!ok) break;
                tc_fence_after();
                const uint32_t sf_s = sf_base + r.slot * S::kSfBytes;
                const uint32_t sfa = tmem + kSfCol0 + set * kSfSetCols;
                const uint32_t sfb = sfa + S::MT * S::W * 4;
                const uint64_t a_desc = smem_desc_sw128(a_base + r.slot * S::kABytes);
                const uint64_t b_desc = smem_desc_sw128(b_base + r.slot * b_bytes);
                const int steps = ks == k_stages - 1 ? last_steps : 4;
                if (leader) {
#pragma unroll
                    for (int i = 0; i < S::MT * S::W; ++i) copy_atom(sfa + 4 * i, sf_s + i * kAtomBytes);
#pragma unroll
                    for (int i = 0; i < S::W * S::NA; ++i)
                        if (i % S::NA == 0 || two)
                            copy_atom(sfb + 4 * i, sf_s + S::kSfaBytes + i * kAtomBytes);
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        if (t >= steps) break;
                        const int word = kNv ? t : t >> 1;
                        // 64 k are 32 bytes of the swizzled row: 2 in descriptor units
#pragma unroll
                        for (int m = 0; m < S::MT; ++m)
                            mma_fp4<kNv>(d + m * S::kAccStep, a_desc + 2 * t + m * (kTileN * kStageBytesRow >> 4),
                                         b_desc + 2 * t, t & 1 ? id2 : id0, sfa + 4 * (m * S::W + word),
                                         sfb + 4 * word * S::NA, (ks | t) != 0);
                    }
                    mma_commit(&empty[r.slot]);
                    if (ks == k_stages - 1) mma_commit(&acc_full[buf]);
                }
                __syncwarp();
                set ^= 1u;
                r.next(n_stages);
            }
            buf ^= 1u;
            if (buf == 0) acc_phase ^= 1u;
        }
        // Every MMA and commit of the warp done before the CTA leaves.
        if (leader) mma_commit(final_bar);
        __syncwarp();
        warp_wait_bounded(final_bar, 0, nullptr, p.status, lim);
    } else if (warp < kAScaleWarp) {
        const int parts = min(kLoaders, static_cast<int>(n_stages)), part = warp - kWScaleWarp;
        if (part < parts)
            load_scales<kNv, kSwiglu, true>(p, sf_ring, n_stages, total, roff, ioff, sf_full, empty, abort_flag, part,
                                            parts);
    } else if (warp < kEpilogueWarp) {
        const int parts = min(kLoaders, static_cast<int>(n_stages)), part = warp - kAScaleWarp;
        if (part < parts)
            load_scales<kNv, kSwiglu, false>(p, sf_ring, n_stages, total, roff, ioff, sf_full, empty, abort_flag, part,
                                             parts);
    } else {
        const int quarter = warp & 3;
        const float a2 = kNv ? __ldg(p.a_scale_2) : 1.0f;
        const float h2 = kNv && kSwiglu ? __ldg(p.h_scale_2) : 1.0f;
        if (!(h2 > 0.0f && h2 < __uint_as_float(kF32Inf)) && tid == kThreads - 1) set_status(p.status, MOE_ERR_DATA);
        uint32_t buf = 0, phase = 0;
        for (int j = blockIdx.x; j < total; j += gridDim.x) {
            const Item it = decode_item<S::NT>(j, roff, ioff, E, p.n_tiles);
            if (!warp_wait_bounded(&acc_full[buf], phase, abort_flag, p.status, lim)) break;
            tc_fence_after();
            const uint32_t acc = tmem + buf * kAccCols + (static_cast<uint32_t>(quarter * 32) << 16);
            const float scale = kNv ? __ldg(p.w_scale_2 + it.e) * a2 : 1.0f;
            if constexpr (kSwiglu)
                store_swiglu<kNv>(p, it, acc, it.n0 + 32 * quarter, scale, h2, &acc_empty[buf]);
            else
                store_plain(p, it, acc, it.n0 + 32 * quarter + lane, scale, &acc_empty[buf]);
            buf ^= 1u;
            if (buf == 0) phase ^= 1u;
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kProducerWarp) tmem_dealloc(tmem, kTmemCols);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    }();
    return fn;
}

// Codes [rows, K / 2] in boxes of 128 bytes (256 k) by `box_rows` rows; bytes
// past a row's end and rows past the last read as zero codes.
bool encode_codes(CUtensorMap *map, const void *base, int64_t rows, int K, uint32_t box_rows) {
    PFN_cuTensorMapEncodeTiled_v12000 encode = encode_fn();
    if (!encode) return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(K / 2), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(K / 2)};
    cuuint32_t box[2] = {kStageBytesRow, box_rows};
    cuuint32_t estr[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kNv, bool kSwiglu>
moe_status launch(const Fp4Gemm &g, cudaStream_t stream, int num_sms) {
    CUtensorMap tm_w, tm_a64, tm_a16;
    if (!encode_codes(&tm_w, g.w_codes, static_cast<int64_t>(g.E) * g.N, g.K, kTileN) ||
        !encode_codes(&tm_a64, g.a_codes, g.rows, g.K, 64) || !encode_codes(&tm_a16, g.a_codes, g.rows, g.K, 16))
        return MOE_ERR_CUDA;
    static std::atomic<uint64_t> attr_dev_mask{0};   // devices whose attribute is set
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
    const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
    if (!(attr_dev_mask.load(std::memory_order_acquire) & bit) || !bit) {
        if (cudaFuncSetAttribute(fp4_gemm_kernel<kNv, kSwiglu>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kSmemBytes) != cudaSuccess)
            return MOE_ERR_CUDA;
        attr_dev_mask.fetch_or(bit, std::memory_order_release);
    }
    Params p;
    p.w_scales = g.w_scales;
    p.a_scales = g.a_scales;
    p.w_scale_2 = g.w_scale_2;
    p.a_scale_2 = g.a_scale_2;
    p.h_scale_2 = g.h_scale_2;
    p.group_sizes = g.group_sizes;
    p.out = g.out;
    p.out_scales = g.out_scales;
    p.status = g.status;
    p.rows = g.rows;
    p.K = g.K;
    p.N = g.N;
    p.E = g.E;
    p.I = kSwiglu ? g.N / 2 : 0;
    p.out_bf16 = g.out_bf16;
    p.n_tiles = ((kSwiglu ? g.N / 2 : g.N) + kTileN - 1) / kTileN;
    p.scale_row = g.K / (kNv ? 16 : 32);
    const int vec_bytes = kNv ? 16 : 8;
    const bool whole = g.K % kStageK == 0;
    p.w_vec = whole && reinterpret_cast<uintptr_t>(g.w_scales) % vec_bytes == 0;
    p.a_vec = whole && reinterpret_cast<uintptr_t>(g.a_scales) % vec_bytes == 0;
    p.wait_limit_ns = g.wait_limit_ns;
    fp4_gemm_kernel<kNv, kSwiglu><<<num_sms, kThreads, kSmemBytes, stream>>>(tm_w, tm_a64, tm_a16, p);
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace fp4

moe_status launch_fp4_gemm(const Fp4Gemm &g, bool nv, bool swiglu, cudaStream_t stream, int num_sms) {
    if (g.rows == 0) return MOE_OK;
    if (nv) return swiglu ? fp4::launch<true, true>(g, stream, num_sms) : fp4::launch<true, false>(g, stream, num_sms);
    return swiglu ? fp4::launch<false, true>(g, stream, num_sms) : fp4::launch<false, false>(g, stream, num_sms);
}

}  // namespace moe
