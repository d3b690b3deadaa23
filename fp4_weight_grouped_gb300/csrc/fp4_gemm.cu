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
//  * Short bands (fp4_gemm_kernel): weights are the MMA's A operand (128 weight
//    rows), the band's token rows its B operand (N = 16..192), as in the W4A16
//    product: a decode band of one row wastes no weight traffic.  Long bands
//    (fp4_gemm_pair_kernel) run in CTA pairs with tokens as A; see there, and
//    launch() for which call takes which.
//  * One K stage is 256 k: 128 bytes a row, the 128-byte swizzle TMA writes and
//    the MMA reads; four MMAs of 64 k.
//  * Block scales have to sit in tensor memory (word of row m at lane m % 32 of
//    all four lane quarters, column m / 32; a word holds four consecutive
//    scales).  TMA brings the scale bytes of four stages at a time into a staging
//    area, and converter warps, one a lane quarter, read them back and write
//    them with tcgen05.st.  So scales keep the
//    layout the rest of the library uses, and tokens may start at any row.  The
//    other way, atoms in shared memory and tcgen05.cp, cost the tensor pipe about
//    66 cycles a copy: 600 (MXFP4) to 1,000 (NVFP4) cycles a stage, for 384 of MMA.
//    Two sets of four converter warps take the stages in turn; an arrival on the
//    stage's own barrier, which the issuer waits for anyway, hands the scales over.
//  * Accumulators are double-buffered (2 x 192 columns): the epilogue warps of
//    one item run under the next item's MMAs.  A band's rows are cut into equal
//    chunks of at most 192 (96 with SwiGLU) tokens, multiples of 16.
//  * SwiGLU: an item holds 128 gate rows and the 128 matching up rows as two
//    MMAs into two column ranges, so a thread has g and u of one output column
//    at the same token and no shuffle pairs them.  The 32 lanes of a warp hold
//    32 consecutive h columns, one MX block: h is quantised in registers (block
//    maximum by redux, for NVFP4 by shuffles that halve the tokens, an 8 x 8 nibble
//    transpose by three shuffles) and leaves the SM as 4-bit codes, never as bf16 or
//    f32.  Sums, silu and the product are f32; the only rounding is that to 4 bits.
//  * Persistent CTAs, one per SM, over a static list of (expert, chunk, tile).
//  * Every wait is bounded; see wait_bounded.
//
// Bound: HBM for short bands, what TMA brings into an SM for long ones.  Measured
// (perf/routed_bands.py), 256 experts, top-6, w13 K = 4,096, I = 2,048 and w2 K = 2,048,
// N = 4,096, of the bytes each has to move at the measured copy rate: 64 tokens (199 experts)
// w13 with SwiGLU MXFP4 262 us (100%), NVFP4 280 (99%), w2 f32 141 (93%) and 147 (94%);
// 8,192 tokens (bands of 192 rows) w13 436 us (82%) and 472 (81%), w2 307 (96%) and 313
// (97%); six bands of 8,192 rows, both products 447 us, 5,535 TFLOP/s.
#include <atomic>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <stdint.h>

#include "device_common.cuh"
#include "fp4_common.cuh"
#include "launch.h"
#include "ring_drain.h"
#include "vec_io.cuh"

namespace moe {
namespace fp4 {

constexpr int kProducerWarp = 0, kIssuerWarp = 1;
constexpr int kCopyWarp = 2;                           // scale bytes (by threads: 2 weights, 3 tokens)
constexpr int kSets = 2;                               // converter sets, on stages in turn
constexpr int kConvertWarp = 4, kEpilogueWarp = kConvertWarp + 4 * kSets;   // four warps a set: one a lane quarter
constexpr int kHalves = 2;                             // epilogue warps a lane quarter
constexpr int kThreads = 32 * (kEpilogueWarp + 4 * kHalves);
constexpr int kMaxE = 1024;
constexpr int kTileN = 128;                    // weight rows a tile (MMA M)
constexpr int kStageBytesRow = 128;            // 256 k
constexpr int kStageK = 256;
constexpr int kMaxStages = 5;                  // MXFP4 keeps as many stages of scales in tensor memory
constexpr int kGroup = 4;                      // stages of a group of staged scale bytes
constexpr int kDepth = 2;                      // groups in the staging area
constexpr int kAccCols = 192;                  // columns of one accumulator buffer
constexpr int kSfCol0 = 2 * kAccCols;          // scale columns after the accumulators
constexpr int kTmemCols = 512;

constexpr int kRingBytes = 172 * 1024;
constexpr int kOffStaging = kRingBytes;        // scale bytes on their way to tensor memory
constexpr int kOffRow = kOffStaging + kDepth * kGroup * 11 * 512;
constexpr int kOffItem = kOffRow + (kMaxE + 1) * 4;
constexpr int kOffBars = (kOffItem + (kMaxE + 1) * 4 + 7) & ~7;
constexpr int kNumBars = 2 * kMaxStages + 4 + 1 + 2 * kDepth + 2 * kSets;
constexpr int kOffMisc = kOffBars + kNumBars * 8;
constexpr int kMiscBytes = 64;                 // see Misc
constexpr int kSmemBytes = kOffMisc + kMiscBytes + 1024;
static_assert(kSmemBytes <= 232448, "shared memory budget");

// Scale columns of a stage, and the stages they are kept for: every shape here has 12
// columns a scale word (384 rows, 32 a column, over both operands).
template <bool kNv>
struct ScaleCols {
    static constexpr int W = kNv ? 4 : 2;                  // scale words a row and stage
    static constexpr int kCols = 12 * W;
    static constexpr int kSlots = (kTmemCols - kSfCol0) / kCols;
    static_assert(kSlots == (kNv ? 2 : kMaxStages), "see convert_scales");
};

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
    int windows;             // scale tensors at 16-byte addresses (see copy_scales_shift)
    int band_lo, band_hi;    // this launch's bands: those of band_lo to band_hi rows
    uint64_t wait_limit_ns;
};

template <bool kNv, bool kSwiglu>
struct Shape {
    static constexpr int MT = kSwiglu ? 2 : 1;             // weight tiles an item
    static constexpr int NT = kSwiglu ? 96 : 192;          // tokens an item, at most
    static constexpr int W = kNv ? 4 : 2;                  // scale words a row and stage
    static constexpr int NA = kSwiglu ? 1 : 2;             // token atoms of 128 rows
    static constexpr int AR = NT / 32;                     // token rows a lane of the scale copier
    static constexpr int kABytes = MT * kTileN * kStageBytesRow;
    static constexpr int kAccStep = kSwiglu ? 96 : 0;      // columns from the gate to the up sums
    static_assert(4 * MT + AR <= 11, "scale staging");
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

// ------------------------------------------------------------------ waits

// The roles' loops share the SM's instruction caches: with every wait, item decode
// and alignment case inlined, a third of all stalls were instruction fetches.  So
// what a loop does not run every time is out of line.

__device__ __noinline__ bool wait_slow(uint64_t *bar, uint32_t parity, volatile int *abort_flag, int *status,
                                       uint64_t lim) {
    return warp_wait_bounded(bar, parity, abort_flag, status, lim);
}

// warp_wait_bounded with its slow path out of line.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag, int *status,
                                     uint64_t lim) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return wait_slow(bar, parity, abort_flag, status, lim);
}

// A word of shared memory of a CTA of the cluster (address from cluster_addr).
__device__ __forceinline__ uint32_t load_cluster(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// A CTA's words that are no barriers.
struct Misc {
    uint32_t tmem;                 // tensor-memory address
    int nt;                        // widest chunk of the call
    int abort;                     // a wait of the CTA gave up
    int bad;                       // a converter saw a scale that the format does not allow
    uint32_t stages;               // of the ring,
    uint32_t issued;               // and how many the producer issued
    uint32_t relay;                // ring positions (slot + stages * phase) where the relay
    uint32_t stops[kStopWarps];    // and the converter warps stopped
};
static_assert(sizeof(Misc) <= kMiscBytes && kStopWarps == 4 * kSets, "misc area");

// The end of a CTA, by one thread once all warps (of a pair: of both CTAs) have stopped.
//
// Where a wait gave up, every copy that the producer issued has to land before the CTA
// leaves.  The stages' barriers count the converters and the relay too, so their missing
// arrivals are made up for; a stage that the producer issued has the phase before it
// complete (it waited for that stage's MMAs), so they fall into the right one.  Bounded by
// one limit: the first wait that gives up ends it.
//
// It takes nothing from the roles' registers but constants: with the barriers' address, the
// flag and the bad scales' report passed on to the end, the NVFP4 pair kernel of shifted
// scales spilled in its loops (K = 2,880, six bands of 4,096 rows 237 -> 251 us).
__device__ __noinline__ void finish(uint32_t off_bars, uint32_t off_misc, int k_stages, bool pair, int *status,
                                    uint64_t lim) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + off_bars);
    const Misc &misc = *reinterpret_cast<const Misc *>(smem + off_misc);
    if (misc.bad) set_status(status, MOE_ERR_DATA);
    if (!misc.abort) return;
    const uint32_t relay = pair ? load_cluster(cluster_addr(&misc.relay, 1)) : 0;
    const uint32_t *relayed = pair && cluster_rank() == 0 ? &relay : nullptr;
    const uint32_t issued = misc.issued, n_stages = misc.stages;
    uint32_t from = issued > n_stages ? issued - n_stages : 0;
    while (from < issued && mbar_try_wait(&full[from % n_stages], (from / n_stages) & 1u)) ++from;
    for (uint32_t i = from; i < issued; ++i) {
        uint64_t *bar = &full[i % n_stages];
        for (uint32_t n = missing_arrivals(i, from, n_stages, k_stages, misc.stops, relayed); n > 0; --n)
            mbar_arrive(bar);
        if (!wait_bounded(bar, (i / n_stages) & 1u, nullptr, status, lim)) return;
    }
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

template <int kMost, int kTile>
__device__ __noinline__ Item decode_item(int j, const int *roff, const int *ioff, int E, int n_tiles) {
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
    it.n0 = (r - ch * n_tiles) * kTile;
    const int t0 = ch * cr;
    it.nvalid = min(cr, n - t0);
    it.nt = (it.nvalid + 15) & ~15;
    it.row0 = roff[lo] + t0;
    return it;
}

// Position in a ring of n slots; by <= n.
struct Ring {
    uint32_t slot = 0, phase = 0;
    __device__ __forceinline__ void next(uint32_t n, uint32_t by = 1) {
        slot += by;
        if (slot >= n) {
            slot -= n;
            phase ^= 1u;
        }
    }
};

// ---------------------------------------------------------- scale loaders

// Staged bytes of a row that threads copy: the three 16-byte windows of two pieces (see
// copy_scales_shift); of 32 rows (one q).  An odd number of 16-byte units keeps the copies
// free of bank conflicts.
constexpr int kShiftRow = 48, kShiftStep = 32 * kShiftRow, kShiftPieces = 2;

// Scale bytes [at, at + 16) of R rows at any address into shared memory, zeros past a
// row's end: the aligned words that hold the bytes, up to six rows' in flight
// together, shifted into place.  A word that reaches outside the tensor
// [lo, hi) is put together from its bytes inside.
template <int R>
__device__ __forceinline__ void copy_unaligned(uint8_t *dst, const uint8_t *const (&src)[R], int at, int scale_row,
                                               const uint8_t *lo, const uint8_t *hi) {
    constexpr int kBatch = R <= 6 ? R : 4;
    const int n = min(16, scale_row - at);
#pragma unroll
    for (int q0 = 0; q0 < R; q0 += kBatch) {
        uint32_t w[kBatch][5];
#pragma unroll
        for (int q = q0; q < q0 + kBatch && q < R; ++q) {
            const uint8_t *from = src[q] + at;
            const int off = static_cast<int>(reinterpret_cast<uintptr_t>(from) & 3);
            from -= off;
#pragma unroll
            for (int i = 0; i < 5; ++i) {
                const uint8_t *a = from + 4 * i;
                uint32_t x = 0;
                if (4 * i < n + off) {
                    if (a >= lo && a + 4 <= hi) {
                        x = __ldg(reinterpret_cast<const uint32_t *>(a));
                    } else {
#pragma unroll 1
                        for (int b = 0; b < 4; ++b)
                            if (a + b >= lo && a + b < hi) x |= static_cast<uint32_t>(__ldg(a + b)) << (8 * b);
                    }
                }
                w[q - q0][i] = x;
            }
        }
#pragma unroll
        for (int q = q0; q < q0 + kBatch && q < R; ++q) {
            const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(src[q] + at) & 3) * 8;
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int left = n - 4 * i;        // bytes of this word inside the row
                o[i] = __funnelshift_r(w[q - q0][i], w[q - q0][i + 1], shift);
                if (left < 4) o[i] = left <= 0 ? 0u : o[i] & ((1u << (8 * left)) - 1u);
            }
            *reinterpret_cast<uint4 *>(dst + q * kShiftStep) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

// Bits 7 of the result's bytes: whether some byte of w is one the format does not
// allow.  E8M0: 255, the only byte with bit 7 set that loses it by adding 1 (a carry
// comes from a 255 alone).  E4M3: NaN (0x7F) or a set sign bit, as the block-scaled
// MMA takes unsigned scales: bit 7 before or after adding 1.
template <bool kNv>
__device__ __forceinline__ uint32_t bad_bits(uint32_t w) {
    const uint32_t plus = w + 0x01010101u;
    return kNv ? w | plus : w & ~plus;
}

// Staging of both operands' scale bytes: kDepth groups, the weights' rows first; R rows
// a lane and operand (row lane + 32 q of the tile).
//
// Rows of whole 16-byte pieces come by TMA, kGroup stages a group: 32 (MXFP4) or 64
// (NVFP4) bytes a row in the swizzle of that width, which keeps the converters' reads
// (a row a lane) free of bank conflicts, two-way at most for MXFP4.  (Copies by
// threads, cp.async a row a lane, cost 32 shared-memory cycles each: the converters'
// own reads then took 1,000 to 1,500 cycles a stage.)  Other rows: copy_scales_shift.
struct Staging {
    uint8_t *bytes;
    uint32_t group_bytes;
    uint64_t *full, *empty;           // one a group: copiers -> converters -> copiers
    uint64_t *sets;                   // two a converter set: its shifted words are there, were read
};

// Staged bytes of a row and group, and of 32 rows (one q).
template <bool kNv>
struct GroupRow {
    static constexpr int kBytes = kNv ? 64 : 32, kStep = 32 * kBytes;
};

// What the scale warps need of their kernel.
struct ScaleEnv {
    const Params *p;
    const int *roff, *ioff;
    volatile int *abort_flag;
    int first, step, total;           // the items: first, first + step, ... < total
};

// Copier warp by TMA.  issue(item, group, dst, bar), by one lane, starts the copies of
// a group; bytes(item): what they bring.
template <int kMost, int kTile, class Issue, class Bytes>
__device__ __forceinline__ void copy_scales(const ScaleEnv &v, const Staging &g, Issue issue, Bytes bytes) {
    const Params &p = *v.p;
    const bool leader = elect_one();
    const int groups = (p.K + kGroup * kStageK - 1) / (kGroup * kStageK);
    const uint32_t base = smem_u32(g.bytes);
    Ring r;
    uint32_t issued = 0;
    bool ok = true;
    for (int j = v.first; ok && j < v.total; j += v.step) {
        const Item it = decode_item<kMost, kTile>(j, v.roff, v.ioff, p.E, p.n_tiles);
        const uint32_t n = bytes(it);
        for (int i = 0; i < groups; ++i) {
            ok = wait(&g.empty[r.slot], r.phase ^ 1u, v.abort_flag, p.status, p.wait_limit_ns);
            if (!ok) break;
            if (leader) {
                mbar_arrive_expect_tx(&g.full[r.slot], n);
                issue(it, i, base + r.slot * g.group_bytes, &g.full[r.slot]);
            }
            __syncwarp();
            ++issued;
            r.next(kDepth);
        }
    }
    // Every issued copy lands before the CTA leaves, whoever else may have given up: these
    // barriers count this warp alone.
    if ((threadIdx.x & 31) == 0)
        for (uint32_t i = issued > kDepth ? issued - kDepth : 0; i < issued; ++i)
            if (!wait_bounded(&g.full[i % kDepth], (i / kDepth) & 1u, nullptr, p.status, p.wait_limit_ns)) break;
}

// Copier warp for rows that are not whole 16-byte pieces (one an operand), two pieces a
// group.  Tensors at 16-byte addresses: the three aligned 16-byte windows that hold the
// pieces go into the staging area as they are, side by side, and the converters shift.
// Others are shifted here.  row(item, q): row of this lane, clamped to the tile's or the
// chunk's last row past its end (those sums are never stored, and every staged byte is one
// of the tensor).  used(item): how many q have rows at all.
//
// One warp copies for the whole CTA, so its instructions count: row addresses are made once
// an item, and only items whose windows reach past the tensor's end look at sizes.  (With
// two windows a piece and sizes for each: K = 2,880, six bands of 4,096 rows, N = 3,840,
// NVFP4 f32 384 us.  Loads shifted here, before their store, waited for memory once a piece:
// 8 us of a 16 us call at K = 1,056.)
template <int R, int kMost, int kTile, class RowFn, class UsedFn>
__device__ __forceinline__ void copy_scales_shift(const ScaleEnv &v, const Staging &g, int first_row,
                                                  const uint8_t *base, int64_t rows, bool windows, RowFn row,
                                                  UsedFn used) {
    constexpr int P = kShiftPieces;
    const Params &p = *v.p;
    const int lane = threadIdx.x & 31;
    const int pieces = (p.scale_row + 15) / 16, groups = (pieces + P - 1) / P;
    const int64_t bytes = rows * p.scale_row;
    uint8_t *mine = g.bytes + first_row * kShiftStep + lane * kShiftRow;
    Ring r;
    bool ok = true;
    for (int j = v.first; ok && j < v.total; j += v.step) {
        const Item it = decode_item<kMost, kTile>(j, v.roff, v.ioff, p.E, p.n_tiles);
        const uint8_t *src[R];
        const int n_used = used(it);
        bool inside = true;
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const int64_t at = row(it, q) * p.scale_row, first = windows ? at & ~int64_t(15) : at;
            src[q] = base + first;
            inside = inside && first + 16 * (P * groups + 1) <= bytes;
        }
        inside = __all_sync(0xffffffffu, inside);
        for (int i = 0; i < groups; ++i) {
            ok = wait(&g.empty[r.slot], r.phase ^ 1u, v.abort_flag, p.status, p.wait_limit_ns);
            if (!ok) break;
            uint8_t *to = mine + r.slot * g.group_bytes;
            if (!windows) {
#pragma unroll 1
                for (int k = 0; k < P && i * P + k < pieces; ++k)
                    copy_unaligned<R>(to + k * 16, src, (i * P + k) * 16, p.scale_row, base, base + bytes);
                mbar_arrive(&g.full[r.slot]);
            } else {
                const uint32_t dst = smem_u32(to);
                if (inside) {
#pragma unroll
                    for (int q = 0; q < R; ++q) {
                        if (q >= n_used) break;
#pragma unroll
                        for (int k = 0; k <= P; ++k)
                            asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(
                                             dst + q * kShiftStep + k * 16),
                                         "l"(src[q] + k * 16)
                                         : "memory");
                        src[q] += 16 * P;
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < R; ++q) {
                        if (q >= n_used) break;
#pragma unroll 1
                        for (int k = 0; k <= P; ++k) {
                            const int64_t left = bytes - (src[q] + k * 16 - base);     // zeros past the tensor
                            asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(
                                             dst + q * kShiftStep + k * 16),
                                         "l"(left > 0 ? src[q] + k * 16 : base),
                                         "r"(static_cast<int>(max(min(left, int64_t(16)), int64_t(0))))
                                         : "memory");
                        }
                        src[q] += 16 * P;
                    }
                }
                asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_u32(&g.full[r.slot]))
                             : "memory");
            }
            __syncwarp();
            r.next(kDepth);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");   // none in flight when the CTA leaves
}

// Scale words of one row staged by copy_scales_shift, `bits` bits after the staged word
// `from`; `n` bytes of them are the row's, the rest reads as zeros.
template <int W>
__device__ __forceinline__ void read_shifted(const uint8_t *from, uint32_t bits, int n, uint32_t (&w)[W]) {
    uint32_t raw[W + 1];
#pragma unroll
    for (int i = 0; i <= W; ++i) raw[i] = reinterpret_cast<const uint32_t *>(from)[i];
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = __funnelshift_r(raw[i], raw[i + 1], bits);
    if (n < 4 * W) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const int left = n - 4 * i;
            w[i] &= left >= 4 ? 0xFFFFFFFFu : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
        }
    }
}

// 8, 16 or 32 consecutive columns of each lane's own tensor-memory lane.
template <int C>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&v)[C]) {
    static_assert(C == 8 || C == 16 || C == 32, "a width without a store would store nothing");
    if constexpr (C == 32) {
        tmem_st32(taddr, v);
    } else if constexpr (C == 16) {
        tmem_st16(taddr, v);
    } else {
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]),
                     "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    }
}

// W scale words of every row of one staged group, kStep bytes from one q to the next.
template <int kStep, int R, int W>
__device__ __forceinline__ void read_words(const uint8_t *at, uint32_t (&w)[R][W]) {
#pragma unroll
    for (int q = 0; q < R; ++q) {
        if constexpr (W == 2) {
            const uint2 x = *reinterpret_cast<const uint2 *>(at + q * kStep);
            w[q][0] = x.x; w[q][1] = x.y;
        } else {
            const uint4 x = *reinterpret_cast<const uint4 *>(at + q * kStep);
            w[q][0] = x.x; w[q][1] = x.y; w[q][2] = x.z; w[q][3] = x.w;
        }
    }
}

template <int W>
__device__ __forceinline__ void put_words(uint8_t *at, const uint32_t (&w)[W]) {
    if constexpr (W == 2) *reinterpret_cast<uint2 *>(at) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint4 *>(at) = make_uint4(w[0], w[1], w[2], w[3]);
}

// bad_bits of words kQuarter, kQuarter + 4, ... of both operands'.
template <bool kNv, int kQuarter, int RA, int RB, int W>
__device__ __forceinline__ uint32_t bad_quarter(const uint32_t (&a)[RA][W], const uint32_t (&b)[RB][W]) {
    uint32_t bad = 0;
#pragma unroll
    for (int i = kQuarter; i < (RA + RB) * W; i += 4)
        bad |= bad_bits<kNv>(i < RA * W ? a[i < RA * W ? i / W : 0][i % W] : b[i < RA * W ? 0 : i / W - RA][i % W]);
    return bad;
}

// A stage's columns of one operand.  kByTile: (tile of 128 rows, word, column), else
// (word, tile, column).
template <int R, int W, bool kByTile>
__device__ __forceinline__ void store_words(uint32_t taddr, const uint32_t (&w)[R][W]) {
    constexpr int T = (R + 3) / 4;
    uint32_t v[4 * T * W];
#pragma unroll
    for (int i = 0; i < W; ++i)
#pragma unroll
        for (int q = 0; q < 4 * T; ++q)
            v[(kByTile ? (q / 4) * W + i : i * T + q / 4) * 4 + (q & 3)] = q < R ? w[q < R ? q : 0][i] : 0u;
    tmem_st<4 * T * W>(taddr, v);
}

__device__ __forceinline__ void init_scale_bars(uint64_t *raw_bars, uint32_t copiers) {
    for (int d = 0; d < kDepth; ++d) {
        mbar_init(&raw_bars[d], copiers);             // by TMA: 1; by threads: the two warps' lanes
        mbar_init(&raw_bars[kDepth + d], 4 * kSets);  // the converter warps
    }
    for (int i = 0; i < 2 * kSets; ++i) mbar_init(&raw_bars[2 * kDepth + i], 4);   // a set's warps
}

// Converter warp: staged bytes of both operands -> scale columns in tensor memory, of
// stages set, set + 2, ... of each item.  The four warps of a set (one a lane quarter)
// arrive on the stage's `full` barrier, the TMA's.  MXFP4 has as many scale slots as
// stages, so a slot is free when its stage is; NVFP4 has two, so the slot of stage s
// is free once the MMAs of stage s - 2 are done.
//
// What counts here is instructions: a warp takes 7 to 10 cycles for each, so a set
// that handled whole groups with three rings to keep (280 instructions) needed 2,800
// cycles for two stages and bound the kernel.
//
// A: the MMA's A operand (kByTile), B: its B operand; their first rows in the group.
template <bool kNv, bool kShift, int RA, int RB, int kMost, int kTile, class RowA, class RowB, class UsedA, class UsedB>
__device__ __forceinline__ void convert_scales(const ScaleEnv &v, const Staging &g, int first_a, int first_b,
                                               uint32_t sf_tmem, uint64_t *full, uint64_t *empty, uint32_t n_stages,
                                               Misc *misc, bool windows, RowA row_a, RowB row_b, UsedA used_a,
                                               UsedB used_b) {
    using C = ScaleCols<kNv>;
    constexpr int W = C::W, kACols = 4 * ((RA + 3) / 4) * W;
    constexpr int kStages = kShift && kNv ? 2 : kGroup;       // of a group
    constexpr int kStep = GroupRow<kNv>::kStep;
    static_assert(kACols + 4 * ((RB + 3) / 4) * W == C::kCols, "scale columns of a stage");
    static_assert(kSets == 2 && kGroup % 2 == 0, "sets take stages in turn");
    const Params &p = *v.p;
    const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3;
    const int k_stages = (p.K + kStageK - 1) / kStageK;
    const int set = ((threadIdx.x >> 5) - kConvertWarp) >> 2;
    uint32_t bad = 0;
    bool ok = true;
    // By TMA: this lane's rows, whose 16-byte chunk c lies at c ^ swizzle.  Shifted: a
    // group is two pieces, of two MXFP4 stages or one of NVFP4 each.  The warps of a set
    // then shift a quarter of the rows each into `words` (all four shifting all rows spent
    // twice the shared-memory cycles: K = 2,880, NVFP4, 24 bands of 16 rows 70 us).
    const uint8_t *mine = g.bytes + lane * (kShift ? kShiftRow : GroupRow<kNv>::kBytes);
    const int swizzle = kNv ? lane >> 1 & 3 : lane >> 2 & 1;
    constexpr int RT = RA + RB, kShare = (RT + 3) / 4, kWordStep = 32 * 4 * W;
    uint8_t *words = g.bytes + kDepth * g.group_bytes + set * RT * kWordStep + lane * 4 * W;
    uint64_t *ready = g.sets + 2 * set, *taken = ready + 1;
    uint32_t turn = 0;
    Ring raw, r;                  // staged group, this set's next stage
    uint32_t sf = set;            // NVFP4: scale slot
    if (set) r.next(n_stages);
    for (int j = v.first; ok && j < v.total; j += v.step) {
        uint32_t from[kShare], bits[kShare];   // this warp's rows quarter, quarter + 4, ...
        bool has[kShare];
        if constexpr (kShift) {
            const Item it = decode_item<kMost, kTile>(j, v.roff, v.ioff, p.E, p.n_tiles);
#pragma unroll
            for (int t = 0; t < kShare; ++t) {
                const int q = min(quarter + 4 * t, RT - 1);
                const int64_t row = q < RA ? row_a(it, q) : row_b(it, q - RA);
                const uint32_t b = windows ? static_cast<uint32_t>(row * p.scale_row) & 15u : 0u;
                from[t] = (q < RA ? first_a + q : first_b + q - RA) * kShiftStep + (b & ~3u);
                bits[t] = 8 * (b & 3u);
                has[t] = quarter + 4 * t < RT && (q < RA ? q < used_a(it) : q - RA < used_b(it));
            }
        }
        for (int k0 = 0; ok && k0 < k_stages; k0 += kStages) {
            ok = wait(&g.full[raw.slot], raw.phase, v.abort_flag, p.status, p.wait_limit_ns);
            const uint8_t *group = mine + raw.slot * g.group_bytes;
            const int end = min(k0 + kStages, k_stages);
#pragma unroll 1
            for (int ks = k0; ok && ks < end; ks += 2) {
                const int by = ks + 2 <= k_stages ? 2 : 1;
                if (ks + set < k_stages) {     // an odd last stage is the first set's
                    uint32_t wa[RA][W], wb[RB][W];
                    const int i = (ks - k0) >> 1;
                    if constexpr (kShift) {
                        const uint8_t *at = group + (2 * i + set) * 4 * W;
                        const int n = p.scale_row - (ks + set) * 4 * W;
                        ok = wait(taken, (turn & 1u) ^ 1u, v.abort_flag, p.status, p.wait_limit_ns);
                        if (!ok) break;
#pragma unroll
                        for (int t = 0; t < kShare; ++t) {
                            if (!has[t]) continue;
                            uint32_t w[W];
                            read_shifted(at + from[t], bits[t], n, w);
#pragma unroll
                            for (int i = 0; i < W; ++i) bad |= bad_bits<kNv>(w[i]);
                            put_words(words + (quarter + 4 * t) * kWordStep, w);
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(ready);
                        ok = wait(ready, turn & 1u, v.abort_flag, p.status, p.wait_limit_ns);
                        if (!ok) break;
                        read_words<kWordStep>(words, wa);
                        read_words<kWordStep>(words + RA * kWordStep, wb);
                        __syncwarp();
                        if (lane == 0) mbar_arrive(taken);
                        ++turn;
                    } else {
                        const uint8_t *at = group + (((kNv ? 2 * i + set : i) ^ swizzle) << 4) + (kNv ? 0 : set * 8);
                        read_words<kStep>(at + first_a * kStep, wa);
                        read_words<kStep>(at + first_b * kStep, wb);
                    }
                    // The four warps hold the same words; each checks a quarter (shifted: did).
                    if constexpr (kShift) {
                    } else if (quarter == 0) bad |= bad_quarter<kNv, 0>(wa, wb);
                    else if (quarter == 1) bad |= bad_quarter<kNv, 1>(wa, wb);
                    else if (quarter == 2) bad |= bad_quarter<kNv, 2>(wa, wb);
                    else bad |= bad_quarter<kNv, 3>(wa, wb);
                    const bool back = r.slot < 2;
                    if constexpr (kNv)
                        ok = wait(&empty[back ? r.slot + n_stages - 2 : r.slot - 2], r.phase ^ back, v.abort_flag,
                                  p.status, p.wait_limit_ns);
                    else
                        ok = wait(&empty[r.slot], r.phase ^ 1u, v.abort_flag, p.status, p.wait_limit_ns);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t at = sf_tmem + (kNv ? sf : r.slot) * C::kCols;
                    store_words<RA, W, true>(at, wa);
                    store_words<RB, W, false>(at + kACols, wb);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&full[r.slot]);
                }
                sf ^= by & 1;
                r.next(n_stages, by);
            }
            // The group was read by loads; its next contents may come by TMA.
            if constexpr (!kShift) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&g.empty[raw.slot]);
            raw.next(kDepth);
        }
    }
    if (bad & 0x80808080u) misc->bad = 1;
    if (lane == 0) misc->stops[(threadIdx.x >> 5) - kConvertWarp] = r.phase * n_stages + r.slot;
}

// -------------------------------------------------------------- epilogues

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&v)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
                   "=r"(v[7])
                 : "r"(taddr));
}

// Two f32 in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// h = silu(g) u of two scaled pairs, silu(g) = g / (1 + 2^(-g log2 e)) with the hardware's
// base-2 exponential and reciprocal.  The exponent is rounded to f32 once, so the relative
// error grows with |g| where g < 0: about (1.25 |g| + 10) 2^-24, a few ulps near 0 and 7e-6
// at g = -88.  (h is rounded to 4 bits next.)  Below g = -88.7 the exponential is infinite
// and silu is -0, as f32 has it for this formula.
template <bool kNv>
__device__ __forceinline__ float2 gated2(uint32_t g0, uint32_t g1, uint32_t u0, uint32_t u1, float scale) {
    float2 g = make_float2(__uint_as_float(g0), __uint_as_float(g1));
    float2 u = make_float2(__uint_as_float(u0), __uint_as_float(u1));
    if constexpr (kNv) {
        g = mul2(g, make_float2(scale, scale));
        u = mul2(u, make_float2(scale, scale));
    }
    const float2 x = mul2(g, make_float2(-1.4426950408889634f, -1.4426950408889634f));
    float2 t, r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(t.x) : "f"(x.x));
    asm("ex2.approx.f32 %0, %1;" : "=f"(t.y) : "f"(x.y));
    t = add2(t, make_float2(1.0f, 1.0f));
    asm("rcp.approx.f32 %0, %1;" : "=f"(r.x) : "f"(t.x));
    asm("rcp.approx.f32 %0, %1;" : "=f"(r.y) : "f"(t.y));
    return mul2(mul2(g, r), u);
}

// max(m, |a|, |b|), NaN if one is.
__device__ __forceinline__ float max_abs(float m, float a, float b) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(m), "f"(a), "f"(b));
    return d;
}

// The sums of a buffer are in registers: release it.
__device__ __forceinline__ void release_acc(uint64_t *acc_empty) {
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(acc_empty);
}

// f32 / bf16 sums: lane = weight row, so a warp stores 32 consecutive columns of one
// token row at a time; the two warps of a lane quarter take 16 tokens in turn.
__device__ __forceinline__ void store_plain(const Params &p, const Item &it, uint32_t acc, int n, int half,
                                            float scale, uint64_t *acc_empty) {
    if (half * 16 >= it.nvalid) release_acc(acc_empty);
    for (int c = half * 16; c < it.nvalid; c += 16 * kHalves) {
        uint32_t v[16];
        __syncwarp();
        tmem_ld16(acc + c, v);
        tmem_ld_wait();
        if (c + 16 * kHalves >= it.nvalid) release_acc(acc_empty);
        if (n < p.N) {
            const size_t off = static_cast<size_t>(it.row0 + c) * p.N + n;
            const int left = it.nvalid - c;
            if (p.out_bf16) {
                __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.out) + off;
#pragma unroll
                for (int t = 0; t < 16; ++t)
                    if (t < left) o[static_cast<size_t>(t) * p.N] = __float2bfloat16_rn(__uint_as_float(v[t]) * scale);
            } else {
                float *o = static_cast<float *>(p.out) + off;
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
__device__ __forceinline__ void store_swiglu(const Params &p, const Item &it, uint32_t acc, int n0w, int half,
                                             float scale, float h_scale, uint64_t *acc_empty) {
    const int lane = threadIdx.x & 31;
    const int t8 = lane & 7, q = lane >> 3;
    const float g6 = 6.0f * h_scale;
    if (half * 8 >= it.nvalid) release_acc(acc_empty);
    for (int c = half * 8; c < it.nvalid; c += 8 * kHalves) {
        uint32_t g[8], u[8];
        __syncwarp();
        tmem_ld8(acc + c, g);
        tmem_ld8(acc + Shape<kNv, true>::kAccStep + c, u);
        tmem_ld_wait();
        if (c + 8 * kHalves >= it.nvalid) release_acc(acc_empty);
        if (n0w >= p.I) continue;          // warp-uniform: I is a multiple of 32
        float h[8];
        uint32_t m[8];
#pragma unroll
        for (int t = 0; t < 8; t += 2) {
            const float2 two = gated2<kNv>(g[t], g[t + 1], u[t], u[t + 1], scale);
            h[t] = two.x;
            h[t + 1] = two.y;
            m[t] = __float_as_uint(h[t]) & 0x7FFFFFFFu;
            m[t + 1] = __float_as_uint(h[t + 1]) & 0x7FFFFFFFu;
        }
        uint8_t *out_scale = p.out_scales + static_cast<size_t>(it.row0 + c) * (p.I / (kNv ? 16 : 32));
        if constexpr (kNv) {
            // Maxima of 8 tokens over the 16 lanes of a block by halving: each step
            // sends half of the tokens a lane still has to its partner.  Lane l ends
            // with the token of bits 3, 2, 1 of l, so the two divisions are done once,
            // not once a token; the factors come back by a shuffle each.
            uint32_t a[4], b[2], top;
            const bool h8 = lane & 8, h4 = lane & 4, h2 = lane & 2;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                a[i] = max(h8 ? m[4 + i] : m[i], __shfl_xor_sync(0xffffffffu, h8 ? m[i] : m[4 + i], 8));
#pragma unroll
            for (int i = 0; i < 2; ++i)
                b[i] = max(h4 ? a[2 + i] : a[i], __shfl_xor_sync(0xffffffffu, h4 ? a[i] : a[2 + i], 4));
            top = max(h2 ? b[1] : b[0], __shfl_xor_sync(0xffffffffu, h2 ? b[0] : b[1], 2));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            const uint32_t byte = nv_scale_byte(top, g6);
            const float inv = nv_inverse(byte, h_scale);
            const int token = (lane >> 1) & 7, t = (token >> 2 & 1) << 2 | (token >> 1 & 1) << 1 | (token & 1);
            if (!(lane & 1) && c + t < it.nvalid)
                out_scale[static_cast<size_t>(t) * (p.I / 16) + n0w / 16 + (lane >> 4)] = static_cast<uint8_t>(byte);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float f = __shfl_sync(0xffffffffu, inv, (lane & 16) | k << 1);
                h[k] = f == 0.0f ? 0.0f : h[k] * f;       // 0: zeros, or an infinity or NaN in the block
            }
        } else {
            uint32_t my_byte = 0;
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const uint32_t byte = mx_scale_byte(__reduce_max_sync(0xffffffffu, m[t]));
                h[t] = byte == 255u ? 0.0f : h[t] * mx_inverse(byte);
                if (t == t8) my_byte = byte;
            }
            if (q == 0 && c + t8 < it.nvalid)
                out_scale[static_cast<size_t>(t8) * (p.I / 32) + n0w / 32] = static_cast<uint8_t>(my_byte);
        }
        // Nibble t of w: this lane's column at token c + t.  Transposed over the
        // eight lanes of a group: nibble i becomes column 8 q + i at token c + t8.
        uint32_t w = e2m1x8(h);
#pragma unroll
        for (int k = 4; k > 0; k >>= 1) {
            const uint32_t low = k == 4 ? 0x0000FFFFu : k == 2 ? 0x00FF00FFu : 0x0F0F0F0Fu;
            const uint32_t o = __shfl_xor_sync(0xffffffffu, w, k);
            w = (lane & k) ? ((w & ~low) | ((o >> (4 * k)) & low)) : ((w & low) | ((o & low) << (4 * k)));
        }
        if (c + t8 < it.nvalid)
            *reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(p.out) +
                                          static_cast<size_t>(it.row0 + c + t8) * (p.I / 2) + n0w / 2 + 4 * q) = w;
    }
}

// Zeros in the staging area: the converters look at all of a group's bytes for ones
// the format does not allow, also where the item has fewer token rows (later they
// find an earlier item's).  Before the barrier that lets the copies start.
__device__ __forceinline__ void clear_staging(uint8_t *staging, int bytes) {
    for (int i = threadIdx.x * 16; i < bytes; i += kThreads * 16)
        *reinterpret_cast<uint4 *>(staging + i) = make_uint4(0, 0, 0, 0);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Row and item offsets from the group sizes (64-bit sums: sizes that wrap 32 bits
// are caught), and the widest chunk.  Rows count every band, items those of this
// launch.  The experts go 32 to a warp, first for their totals, then for the offsets
// on top of the totals before them (one warp over all of them took 2 us at 256
// experts and 6 at 1,024).  False: no items, or (recorded) the sizes do not add up.
// `scratch`: 1 KB.
struct Totals {
    long long rows, items;
    int most, bad;
};

template <int kMost>
__device__ __forceinline__ bool build_items(const Params &p, int *roff, int *ioff, void *scratch, int *nt_slot) {
    constexpr uint32_t kAll = 0xffffffffu;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = p.E, chunks = (E + 31) / 32;
    Totals *totals = static_cast<Totals *>(scratch);
    const auto rows_of = [&](int e, int *most) -> long long {    // items of expert e, its chunk's rows in *most
        const int n = e < E ? __ldg(p.group_sizes + e) : 0;
        *most = 0;
        if (n <= 0 || n < p.band_lo || n > p.band_hi) return 0;
        *most = chunk_rows(min(n, p.rows), kMost);
        return (static_cast<long long>(n) + kMost - 1) / kMost * p.n_tiles;
    };
    for (int c = warp; c < chunks; c += kThreads / 32) {
        const int e = c * 32 + lane, n = e < E ? __ldg(p.group_sizes + e) : 0;
        int most;
        long long items = rows_of(e, &most), rows = max(n, 0);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            rows += __shfl_xor_sync(kAll, rows, d);
            items += __shfl_xor_sync(kAll, items, d);
        }
        most = __reduce_max_sync(kAll, most);
        const int bad = __any_sync(kAll, n < 0);
        if (lane == 0) totals[c] = {rows, items, most, bad};
    }
    __syncthreads();
    // Lane l holds the totals of chunk l; sums up to and of all chunks.
    const Totals mine = lane < chunks ? totals[lane] : Totals{0, 0, 0, 0};
    long long rsum = mine.rows, isum = mine.items;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long ro = __shfl_up_sync(kAll, rsum, d), io = __shfl_up_sync(kAll, isum, d);
        if (lane >= d) { rsum += ro; isum += io; }
    }
    const long long all_rows = __shfl_sync(kAll, rsum, 31), all_items = __shfl_sync(kAll, isum, 31);
    const bool bad = __any_sync(kAll, mine.bad) || all_rows != p.rows || all_items > INT32_MAX;
    const int most = __reduce_max_sync(kAll, mine.most);
    if (bad) {
        if (threadIdx.x == 0) set_status(p.status, MOE_ERR_DATA);
        return false;
    }
    if (all_items == 0) return false;
    for (int c = warp; c < chunks; c += kThreads / 32) {
        const int e = c * 32 + lane, n = e < E ? __ldg(p.group_sizes + e) : 0;
        int unused;
        // The sums are below 2^31 here.
        const int items = static_cast<int>(rows_of(e, &unused));
        int r = n, i = items;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int ro = __shfl_up_sync(kAll, r, d), io = __shfl_up_sync(kAll, i, d);
            if (lane >= d) { r += ro; i += io; }
        }
        const int r0 = static_cast<int>(__shfl_sync(kAll, rsum - mine.rows, c));
        const int i0 = static_cast<int>(__shfl_sync(kAll, isum - mine.items, c));
        if (e < E) {
            roff[e] = r0 + r - n;
            ioff[e] = i0 + i - items;
        }
    }
    if (threadIdx.x == 0) {
        roff[E] = static_cast<int>(all_rows);
        ioff[E] = static_cast<int>(all_items);
        *nt_slot = most;
    }
    __syncthreads();
    return true;
}

// ------------------------------------------------------------------ kernel

// The end of every CTA of a launch that may run beside the long bands' (see launch):
// whoever waits for this launch then has waited for that one too.
__device__ __forceinline__ void after_pairs() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// kShift: scale rows that are not whole 16-byte pieces (see copy_scales_shift); an
// instantiation of its own, so that the others' registers do not pay for it.
template <bool kNv, bool kSwiglu, bool kShift>
__global__ void __launch_bounds__(kThreads, 1)
    fp4_gemm_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_a64,
                    const __grid_constant__ CUtensorMap tm_a16, const __grid_constant__ CUtensorMap tm_ws,
                    const __grid_constant__ CUtensorMap tm_as, const Params p) {
    using S = Shape<kNv, kSwiglu>;
    using C = ScaleCols<kNv>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    int *roff = reinterpret_cast<int *>(smem + kOffRow);
    int *ioff = reinterpret_cast<int *>(smem + kOffItem);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kOffBars);   // TMA, scale converters -> issuer
    uint64_t *empty = full + kMaxStages;                              // MMA commit -> TMA, scale converters
    uint64_t *acc_full = empty + kMaxStages;                          // MMA commit -> epilogue
    uint64_t *acc_empty = acc_full + 2;                               // epilogue -> issuer
    uint64_t *final_bar = acc_empty + 2;
    uint64_t *raw_bars = final_bar + 1;                               // scale copiers <-> converters
    Misc *misc = reinterpret_cast<Misc *>(smem + kOffMisc);
    volatile int *abort_flag = &misc->abort;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int E = p.E;

    if (tid == 0) misc->abort = misc->bad = 0;
    const bool any = build_items<S::NT>(p, roff, ioff, smem + kOffStaging, &misc->nt);
    // redux: the compiler then knows the loops' bounds as warp-uniform
    const int total = any ? __reduce_max_sync(0xffffffffu, ioff[E]) : 0;
    if (static_cast<int>(blockIdx.x) >= total) {
        after_pairs();
        return;
    }

    if constexpr (!kShift) clear_staging(smem + kOffStaging, kOffRow - kOffStaging);
    // Stage layout: as many stages as fit with the widest chunk of this call.
    const int nt_max = misc->nt;
    const uint32_t b_rows = nt_max <= 32 ? nt_max : (nt_max + 63) & ~63;
    const uint32_t b_bytes = b_rows * kStageBytesRow;
    const uint32_t n_stages = min(static_cast<uint32_t>(kMaxStages), kRingBytes / (S::kABytes + b_bytes));
    static_assert(kRingBytes / (S::kABytes + ((S::NT + 63) & ~63) * kStageBytesRow) >= kMinDrainStages, "see finish");
    uint8_t *b_ring = smem + n_stages * S::kABytes;
    const int k_stages = (p.K + kStageK - 1) / kStageK;

    if (warp == kProducerWarp) tmem_alloc(&misc->tmem, kTmemCols);
    if (tid == 0) {
        for (uint32_t s = 0; s < n_stages; ++s) {
            mbar_init(&full[s], 1 + 4);
            mbar_init(&empty[s], 1);
        }
        init_scale_bars(raw_bars, kShift ? 64 : 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 4 * kHalves);
        }
        mbar_init(final_bar, 1);
        mbar_fence_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc->tmem;
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
            const Item it = decode_item<S::NT, kTileN>(j, roff, ioff, E, p.n_tiles);
            // Token rows in 64-row boxes; a last part of at most 32 rows in 16-row
            // boxes (rows past the chunk belong to the next one; their columns are
            // not stored).
            const int part = it.nt & 63;
            const int n64 = (it.nt >> 6) + (part > 32), n16 = part > 32 ? 0 : part >> 4;
            const uint32_t bytes = S::kABytes + (n64 * 64 + n16 * 16) * kStageBytesRow;
            const int wrow = it.e * p.N + it.n0;
            for (int ks = 0; ks < k_stages; ++ks) {
                ok = wait(&empty[r.slot], r.phase ^ 1u, abort_flag, p.status, lim);
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
        if (lane == 0) {
            misc->stages = n_stages;
            misc->issued = issued;
        }
    } else if (warp == kIssuerWarp) {
        // The whole warp runs the loop, so that addresses and descriptors stay in
        // the warp-uniform registers the tcgen05 instructions take; one elected
        // lane (always the same) issues.  A single-lane loop issued a stage in
        // 1,600 cycles, four times what its MMAs take.
        const bool leader = elect_one();
        const uint32_t a_base = smem_u32(smem), b_base = smem_u32(b_ring);
        const int last_steps = (p.K - (k_stages - 1) * kStageK + 63) >> 6;
        Ring r;
        uint32_t sf = 0, buf = 0, acc_phase = 1;
        bool ok = true;
        for (int j = blockIdx.x; ok && j < total; j += gridDim.x) {
            const Item it = decode_item<S::NT, kTileN>(j, roff, ioff, E, p.n_tiles);
            const uint32_t id0 = idesc_fp4<kNv>(it.nt, 0), id2 = idesc_fp4<kNv>(it.nt, kNv ? 0 : 2);
            const uint32_t d = tmem + buf * kAccCols;
            ok = wait(&acc_empty[buf], acc_phase, abort_flag, p.status, lim);
            for (int ks = 0; ok && ks < k_stages; ++ks) {
                ok = wait(&full[r.slot], r.phase, abort_flag, p.status, lim);
                if (!ok) break;
                tc_fence_after();
                const uint32_t sfa = tmem + kSfCol0 + (kNv ? sf : r.slot) * C::kCols;
                const uint32_t sfb = sfa + S::MT * S::W * 4;
                const uint64_t a_desc = smem_desc_sw128(a_base + r.slot * S::kABytes);
                const uint64_t b_desc = smem_desc_sw128(b_base + r.slot * b_bytes);
                const int steps = ks == k_stages - 1 ? last_steps : 4;
                if (leader) {
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        if (t >= steps) break;
                        const int word = kNv ? t : t >> 1;
                        // 64 k are 32 bytes of the swizzled row: 2 in descriptor units
#pragma unroll
                        for (int m = 0; m < S::MT; ++m)
                            mma_fp4<kNv>(d + m * S::kAccStep, a_desc + 2 * t + m * (kTileN * kStageBytesRow >> 4),
                                         b_desc + 2 * t, t & 1 ? id2 : id0, sfa + 4 * (m * S::W + word),
                                         sfb + 4 * word * S::NA, t > 0 || ks > 0);
                    }
                    mma_commit(&empty[r.slot]);
                    if (ks == k_stages - 1) mma_commit(&acc_full[buf]);
                }
                __syncwarp();
                sf ^= 1u;
                r.next(n_stages);
            }
            buf ^= 1u;
            acc_phase ^= buf == 0;
        }
        // Every MMA and commit of the warp done before the CTA leaves.
        if (leader) mma_commit(final_bar);
        __syncwarp();
        wait(final_bar, 0, nullptr, p.status, lim);
    } else if (warp < kEpilogueWarp) {
        const ScaleEnv v = {&p,    roff, ioff, abort_flag, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x),
                            total};
        constexpr int RW = 4 * S::MT, RA = S::AR, kStep = GroupRow<kNv>::kStep;
        const Staging g = {smem + kOffStaging, (RW + RA) * (kShift ? uint32_t(kShiftStep) : kStep), raw_bars,
                           raw_bars + kDepth, raw_bars + 2 * kDepth};
        const int cols = kSwiglu ? p.I : p.N;
        const int64_t w_rows = static_cast<int64_t>(E) * p.N;
        const auto w_row = [&](const Item &it, int q) {
            return static_cast<int64_t>(it.e) * p.N + (q >= 4 ? p.I : 0) + min(it.n0 + lane + 32 * (q & 3), cols - 1);
        };
        const auto a_row = [&](const Item &it, int q) {
            return static_cast<int64_t>(it.row0 + min(lane + 32 * q, it.nvalid - 1));
        };
        const auto w_used = [](const Item &) { return RW; };
        const auto a_used = [](const Item &it) { return (it.nvalid + 31) / 32; };
        const uint32_t sf_tmem = tmem + kSfCol0 + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        if (warp >= kConvertWarp) {
            convert_scales<kNv, kShift, RW, RA, S::NT, kTileN>(v, g, 0, RW, sf_tmem, full, empty, n_stages,
                                                               misc, p.windows, w_row, a_row, w_used, a_used);
        } else if constexpr (kShift) {
            if (warp == kCopyWarp)
                copy_scales_shift<RW, S::NT, kTileN>(v, g, 0, p.w_scales, w_rows, p.windows, w_row, w_used);
            else
                copy_scales_shift<RA, S::NT, kTileN>(v, g, RW, p.a_scales, p.rows, p.windows, a_row, a_used);
        } else if (warp == kCopyWarp) {
            // 128-row boxes of weights, 32-row boxes of tokens.
            copy_scales<S::NT, kTileN>(
                v, g,
                [&](const Item &it, int i, uint32_t dst, uint64_t *bar) {
                    const int x = i * GroupRow<kNv>::kBytes;
#pragma unroll
                    for (int m = 0; m < S::MT; ++m)
                        tma_load_3d(dst + 4 * m * kStep, &tm_ws, x, it.n0, it.e * S::MT + m, bar);
                    for (int q = 0; 32 * q < it.nvalid; ++q)
                        tma_load_2d(dst + (RW + q) * kStep, &tm_as, x, it.row0 + 32 * q, bar);
                },
                [&](const Item &it) { return (RW + (it.nvalid + 31) / 32) * kStep; });
        }
    } else {
        const int quarter = warp & 3, half = (warp - kEpilogueWarp) >> 2;
        const float a2 = kNv ? __ldg(p.a_scale_2) : 1.0f;
        const float h2 = kNv && kSwiglu ? __ldg(p.h_scale_2) : 1.0f;
        if (!(h2 > 0.0f && h2 < __uint_as_float(kF32Inf)) && tid == kThreads - 1) set_status(p.status, MOE_ERR_DATA);
        uint32_t buf = 0, phase = 0;
        for (int j = blockIdx.x; j < total; j += gridDim.x) {
            const Item it = decode_item<S::NT, kTileN>(j, roff, ioff, E, p.n_tiles);
            if (!wait(&acc_full[buf], phase, abort_flag, p.status, lim)) break;
            tc_fence_after();
            const uint32_t acc = tmem + buf * kAccCols + (static_cast<uint32_t>(quarter * 32) << 16);
            const float scale = kNv ? __ldg(p.w_scale_2 + it.e) * a2 : 1.0f;
            if constexpr (kSwiglu)
                store_swiglu<kNv>(p, it, acc, it.n0 + 32 * quarter, half, scale, h2, &acc_empty[buf]);
            else
                store_plain(p, it, acc, it.n0 + 32 * quarter + lane, half, scale, &acc_empty[buf]);
            buf ^= 1u;
            if (buf == 0) phase ^= 1u;
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kProducerWarp) {
        if (lane == 0) finish(kOffBars, kOffMisc, (p.K + kStageK - 1) / kStageK, false, p.status, p.wait_limit_ns);
        __syncwarp();
        tmem_dealloc(tmem, kTmemCols);
    }
    after_pairs();
}

// ------------------------------------------------- long bands: CTA pairs
//
// Bands of many rows are bound by what TMA brings into an SM (about 53 bytes a
// cycle), not by the MMA.  So two CTAs of a cluster share an item (cta_group::2,
// M = 256): 256 token rows, 128 a CTA, are now the A operand, and 192 weight rows
// the B operand, of which each CTA loads half.  A 256-k stage is 28 KB a CTA, 541
// cycles of copies for 384 cycles of MMA; one CTA with a 128 x 192 tile would copy
// 40 KB for the same 384.
//
// With tokens as rows of D a thread holds one token's consecutive output columns:
// an MX or NV block of h lies in one thread (no shuffles, no transpose), with the
// gate sums in columns 0..95 and the up sums in 96..191 (CTA 0 loads the gate rows,
// CTA 1 the up rows).
//
// Measured (perf/routed_bands.py slope), six bands of 4,096 rows, N = 3,840, MXFP4, bf16
// out: K = 8,192 237 us (6,510 TFLOP/s), K = 2,048 82 us.  A stage more costs about 520
// cycles at 2,070 MHz (NVFP4 560), the copies' 541 within the clock's doubt.  What does not
// grow with K is 31 us with bf16 outputs, 52 with f32 ones and 28 with SwiGLU (NVFP4 30, 52
// and 38), several times the start-up.  With plain outputs that is about their write time at
// the copy rate (28 and 55 us); with SwiGLU's 26 MB it is not, and no cause has been shown:
// the epilogue's instructions are too few for it.  (Over whole calls at 590 cycles a stage,
// no epilogue left 550, no scale conversion 557, neither 509.)
//
// The even CTA issues.  Token scales sit in the CTA of their rows, weight scales in
// both (each SM scales its own half of D).  The odd CTA's issuer warp relays: once
// its CTA's copies and scale columns of a stage are there (it has waited for both on
// its own `full` barrier) it arrives on the even CTA's; commits are multicast to
// both.  Three agents then order a scale column before the MMA that reads it: the
// converter that stored it (tcgen05.wait::st, fence before its arrival), the relay (a
// fence after its wait and one before its arrival) and the issuer (a fence after its
// wait).  The relay's arrival itself is relaxed: a release at cluster scope waits for
// memory accesses that no MMA reads, and took 1,650 cycles a stage.

constexpr int kPairM = 256;                    // token rows of an item
constexpr int kPairN = 192;                    // weight rows of an item
constexpr int kPairStages = 5;
constexpr int kPairABytes = 128 * kStageBytesRow;
constexpr int kPairBBytes = kPairN / 2 * kStageBytesRow;
constexpr int kPairRing = kPairStages * (kPairABytes + kPairBBytes);
constexpr int kPairStaging = kDepth * kGroup * (6 + 4) * 512;  // scale bytes on their way to tensor memory
constexpr int kStoreBytes = 32 * 128;          // one epilogue warp's box of outputs: 32 rows of 128 bytes
constexpr int kPairOffStore = kPairRing;
constexpr int kPairOffStaging = kPairOffStore + 4 * kHalves * kStoreBytes;
constexpr int kPairOffRow = kPairOffStaging + kPairStaging;
constexpr int kPairOffItem = kPairOffRow + (kMaxE + 1) * 4;
constexpr int kPairOffBars = (kPairOffItem + (kMaxE + 1) * 4 + 7) & ~7;
constexpr int kPairOffMisc = kPairOffBars + (2 * kPairStages + 4 + 1 + 2 * kDepth + 2 * kSets) * 8;
constexpr int kPairSmem = kPairOffMisc + kMiscBytes + 1024;
static_assert(kPairSmem <= 232448, "shared memory budget (pairs)");

template <bool kNv>
__device__ __forceinline__ void mma_fp4_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                             uint32_t sfb, uint32_t accumulate) {
    if constexpr (kNv)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, "
            "[%5], [%6], p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa),
            "r"(sfb)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, "
            "[%5], [%6], p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa),
            "r"(sfb)
            : "memory");
}

// Token rows of CTA `rank` of an item: the chunk in two halves, the first a
// multiple of 16.
__device__ __forceinline__ void pair_rows(const Item &it, uint32_t rank, int *row0, int *valid) {
    const int half = ((it.nvalid + 1) / 2 + 15) & ~15;
    *row0 = it.row0 + (rank ? half : 0);
    *valid = rank ? max(it.nvalid - half, 0) : min(half, it.nvalid);
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr));
}

// 32 consecutive bytes, 32-byte aligned.
__device__ __forceinline__ void store_sector(void *p, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// 16 lanes x 32 columns: lane l holds columns 8 i + 2 (l % 4) + {0, 1} of rows l / 4
// (v[4 i], v[4 i + 1]) and l / 4 + 8 (v[4 i + 2], v[4 i + 3]).
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
}

__device__ __forceinline__ void release_acc_pair(uint32_t empty_bar) {
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive_cluster(empty_bar);
}

// Plain outputs of one warp: 32 token rows, 32 columns at a time, the two warps of a
// lane quarter in turn.  bf16 rows of whole sectors: lane = row, a lane stores its own
// two sectors.  f32 (and any row alignment): the 16-lane load shape gives four lanes
// eight consecutive columns of a row, one sector, so no transpose is needed.  (Through
// shared memory the same blocks took 1,700 cycles each, more than their MMAs; lanes
// that stored four f32 sectors of their own rows slowed the whole SM's loads.)
__device__ __forceinline__ void pair_store_plain(const Params &p, uint32_t acc, int row0, int valid, int n0, int half,
                                                 int cols, float scale, int vec, uint32_t empty_bar) {
    const int lane = threadIdx.x & 31;
    if (half * 32 >= cols) release_acc_pair(empty_bar);
    for (int c = half * 32; c < cols; c += 32 * kHalves) {
        const bool last = c + 32 * kHalves >= cols;
        const int left = p.N - n0 - c;
        if (p.out_bf16 && vec) {
            uint32_t v[32];
            __syncwarp();
            tmem_ld32(acc + c, v);
            tmem_ld_wait();
            if (last) release_acc_pair(empty_bar);
            __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.out) + static_cast<size_t>(row0 + lane) * p.N + n0 + c;
            if (lane < valid) {
#pragma unroll
                for (int i = 0; i < 32; i += 16) {
                    uint32_t w[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        w[k] = bf16_pair(__uint_as_float(v[i + 2 * k]) * scale,
                                         __uint_as_float(v[i + 2 * k + 1]) * scale);
                    if (i < left) store_sector(o + i, w);
                }
            }
            continue;
        }
        uint32_t v[2][16];
        __syncwarp();
        tmem_ld_16x32(acc + c, v[0]);
        tmem_ld_16x32(acc + c + (16u << 16), v[1]);
        tmem_ld_wait();
        if (last) release_acc_pair(empty_bar);
        const int k = 2 * (lane & 3);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int r = 8 * g + (lane >> 2);
            if (r >= valid) continue;
            const size_t at = static_cast<size_t>(row0 + r) * p.N + n0 + c + k;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = __uint_as_float(v[g >> 1][4 * i + 2 * (g & 1)]) * scale;
                const float y = __uint_as_float(v[g >> 1][4 * i + 2 * (g & 1) + 1]) * scale;
                if (!p.out_bf16 && vec) {
                    if (8 * i < left)
                        *reinterpret_cast<float2 *>(static_cast<float *>(p.out) + at + 8 * i) = make_float2(x, y);
                } else if (p.out_bf16) {
                    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.out) + at + 8 * i;
                    if (8 * i + k < left) o[0] = __float2bfloat16_rn(x);
                    if (8 * i + k + 1 < left) o[1] = __float2bfloat16_rn(y);
                } else {
                    float *o = static_cast<float *>(p.out) + at + 8 * i;
                    if (8 * i + k < left) o[0] = x;
                    if (8 * i + k + 1 < left) o[1] = y;
                }
            }
        }
    }
}

// The same of 32 rows that are all there, by TMA: boxes of 128 bytes a row through this
// warp's `box` (128-byte swizzle: a lane's 16-byte writes, a row a lane, are free of
// bank conflicts).  Whole lines leave the SM in one request each; sectors stored by
// lanes held up the loads (24,576 rows, N = 3,840, six bands, by lanes / by TMA, us:
// MXFP4 bf16 K = 512 63.9 / 52.2, K = 2,048 91.7 / 87.1, K = 4,096 138 / 139; NVFP4 66.3 /
// 53.8, 102 / 90, 158 / 146; MXFP4 f32 87.0 / 79.3, 110 / 107, 157 / 158).
template <bool kBf16>
__device__ __forceinline__ void pair_store_box(const CUtensorMap *map, uint32_t acc, int row0, int n0, int first,
                                               int cols, float scale, uint8_t *box, uint32_t empty_bar) {
    constexpr int kWidth = kBf16 ? 64 : 32;
    const int lane = threadIdx.x & 31;
    uint8_t *mine = box + lane * 128;
    if (first * kWidth >= cols) release_acc_pair(empty_bar);
    for (int c = first * kWidth; c < cols; c += kWidth * kHalves) {
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");   // the box was read
        __syncwarp();
#pragma unroll
        for (int h = 0; h < kWidth; h += 32) {
            uint32_t v[32];
            tmem_ld32(acc + c + h, v);
            tmem_ld_wait();
            if (h + 32 == kWidth && c + kWidth * kHalves >= cols) release_acc_pair(empty_bar);
            constexpr int kEach = kBf16 ? 8 : 4;                     // values of 16 bytes
#pragma unroll
            for (int i = 0; i < 32; i += kEach) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    w[k] = kBf16 ? bf16_pair(__uint_as_float(v[i + 2 * k]) * scale,
                                             __uint_as_float(v[i + 2 * k + 1]) * scale)
                                 : __float_as_uint(__uint_as_float(v[i + k]) * scale);
                const int chunk = (h + i) / kEach;
                *reinterpret_cast<uint4 *>(mine + ((chunk ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
            asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                             reinterpret_cast<uint64_t>(map)),
                         "r"(n0 + c), "r"(row0), "r"(smem_u32(box))
                         : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
    }
}

// SwiGLU of one warp: lane = token row; blocks of 32 h columns, from block `half` on.
template <bool kNv>
__device__ __forceinline__ void pair_store_swiglu(const Params &p, uint32_t acc, int row0, int valid, int n0,
                                                  int half, float scale, float h_scale, uint32_t empty_bar) {
    const int lane = threadIdx.x & 31;
    const float g6 = 6.0f * h_scale;
    for (int b = 32 * half; b < kPairN / 2; b += 32 * kHalves) {
        float h[32];
#pragma unroll
        for (int k = 0; k < 32; k += 16) {
            uint32_t g[16], u[16];
            __syncwarp();
            tmem_ld16(acc + b + k, g);
            tmem_ld16(acc + kPairN / 2 + b + k, u);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                const float2 two = gated2<kNv>(g[i], g[i + 1], u[i], u[i + 1], scale);
                h[k + i] = two.x;
                h[k + i + 1] = two.y;
            }
        }
        if (b + 32 * kHalves >= kPairN / 2) release_acc_pair(empty_bar);
        if (n0 + b >= p.I || lane >= valid) continue;      // I is a multiple of 32
        const size_t row = static_cast<size_t>(row0 + lane);
        uint32_t w[4];
        constexpr int kBlock = kNv ? 16 : 32;
#pragma unroll
        for (int k = 0; k < 32; k += kBlock) {
            float most = 0.0f;
#pragma unroll
            for (int i = 0; i < kBlock; i += 2) most = max_abs(most, h[k + i], h[k + i + 1]);
            const uint32_t m = __float_as_uint(most);
            uint32_t byte;
            float inv;
            bool nan;
            if constexpr (kNv) {
                byte = nv_scale_byte(m, g6);
                inv = nv_inverse(byte, h_scale);
                nan = byte == 0x7Fu;
            } else {
                byte = mx_scale_byte(m);
                inv = mx_inverse(byte);
                nan = byte == 255u;
            }
#pragma unroll
            for (int i = 0; i < kBlock; i += 8) {
                float q[8];
#pragma unroll
                for (int t = 0; t < 8; t += 2) {
                    const float2 two = mul2(make_float2(h[k + i + t], h[k + i + t + 1]), make_float2(inv, inv));
                    q[t] = two.x;
                    q[t + 1] = two.y;
                }
                w[(k + i) / 8] = nan ? 0u : e2m1x8(q);
            }
            p.out_scales[row * (p.I / kBlock) + (n0 + b + k) / kBlock] = static_cast<uint8_t>(byte);
        }
        *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.out) + row * (p.I / 2) + (n0 + b) / 2) =
            make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <bool kNv, bool kSwiglu, bool kShift>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    fp4_gemm_pair_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_a128,
                         const __grid_constant__ CUtensorMap tm_a64, const __grid_constant__ CUtensorMap tm_a32,
                         const __grid_constant__ CUtensorMap tm_ws, const __grid_constant__ CUtensorMap tm_as,
                         const __grid_constant__ CUtensorMap tm_out, const Params p, int out_vec, int out_tma) {
    using C = ScaleCols<kNv>;
    constexpr int kTile = kSwiglu ? kPairN / 2 : kPairN;            // output columns of an item
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    int *roff = reinterpret_cast<int *>(smem + kPairOffRow);
    int *ioff = reinterpret_cast<int *>(smem + kPairOffItem);
    // TMA, scale converters (and relay) -> issuer (relay)
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kPairOffBars);
    uint64_t *empty = full + kPairStages;                                 // pair commit -> TMA, converters of both
    uint64_t *acc_full = empty + kPairStages;                             // pair commit -> epilogues of both
    uint64_t *acc_empty = acc_full + 2;                                   // epilogues of both -> issuer
    uint64_t *final_bar = acc_empty + 2;
    uint64_t *raw_bars = final_bar + 1;                               // scale copiers <-> converters
    Misc *misc = reinterpret_cast<Misc *>(smem + kPairOffMisc);
    volatile int *abort_flag = &misc->abort;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int E = p.E;
    const uint32_t rank = cluster_rank();
    const int first = static_cast<int>(blockIdx.x >> 1), step = static_cast<int>(gridDim.x >> 1);

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid == 0) misc->abort = misc->bad = 0;
    // Both CTAs read the same sizes, so both return here or neither does.
    if (!build_items<kPairM>(p, roff, ioff, smem + kPairOffStaging, &misc->nt)) return;
    // redux: the compiler then knows the loops' bounds as warp-uniform
    const int total = __reduce_max_sync(0xffffffffu, ioff[E]);
    if (first >= total) return;
    if constexpr (!kShift) clear_staging(smem + kPairOffStaging, kPairStaging);
    constexpr uint32_t n_stages = kPairStages;
    static_assert(kPairStages == kMaxStages, "see convert_scales");
    const int k_stages = (p.K + kStageK - 1) / kStageK;
    uint8_t *b_ring = smem + n_stages * kPairABytes;

    if (warp == kProducerWarp) tmem_alloc_pair(&misc->tmem, kTmemCols);
    if (tid == 0) {
        for (uint32_t s = 0; s < n_stages; ++s) {
            mbar_init(&full[s], 1 + 4 + (rank == 0 ? 1 : 0));
            mbar_init(&empty[s], 1);
        }
        init_scale_bars(raw_bars, kShift ? 64 : 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 2 * 4 * kHalves);
        }
        mbar_init(final_bar, 1);
        mbar_fence_init();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();        // the peer's barriers exist before any remote arrival
    tc_fence_after();
    const uint32_t tmem = misc->tmem;
    const uint64_t lim = p.wait_limit_ns;

    if (warp == kProducerWarp) {
        const bool leader = elect_one();
        if (leader) {
            tma_prefetch_map(&tm_w);
            tma_prefetch_map(&tm_a128);
            tma_prefetch_map(&tm_a64);
            tma_prefetch_map(&tm_a32);
        }
        const uint32_t a_base = smem_u32(smem), b_base = smem_u32(b_ring);
        Ring r;
        uint32_t issued = 0;
        bool ok = true;
        for (int j = first; ok && j < total; j += step) {
            const Item it = decode_item<kPairM, kTile>(j, roff, ioff, E, p.n_tiles);
            int row0, valid;
            pair_rows(it, rank, &row0, &valid);
            // Token rows in one box of 128 or 64, or 64 + 32, or 32: a copy costs per
            // request as well as per byte.
            const int n64 = valid > 96 ? 2 : valid > 32 ? 1 : 0;
            const int n32 = valid > 64 && valid <= 96 ? 1 : valid > 0 && valid <= 32 ? 1 : 0;
            const uint32_t bytes = kPairBBytes + (n64 * 64 + n32 * 32) * kStageBytesRow;
            // This CTA's half of the weight rows: gate or up, or 96 of 192.
            const int wrow = it.e * p.N + it.n0 + (rank ? (kSwiglu ? p.I : kPairN / 2) : 0);
            for (int ks = 0; ks < k_stages; ++ks) {
                ok = wait(&empty[r.slot], r.phase ^ 1u, abort_flag, p.status, lim);
                if (!ok) break;
                uint64_t *bar = &full[r.slot];
                const uint32_t a_dst = a_base + r.slot * kPairABytes;
                const int x = ks * kStageBytesRow;
                if (leader) {
                    mbar_arrive_expect_tx(bar, bytes);
                    tma_load_2d(b_base + r.slot * kPairBBytes, &tm_w, x, wrow, bar);
                    if (n64 == 2) tma_load_2d(a_dst, &tm_a128, x, row0, bar);
                    if (n64 == 1) tma_load_2d(a_dst, &tm_a64, x, row0, bar);
                    if (n32) tma_load_2d(a_dst + n64 * 64 * kStageBytesRow, &tm_a32, x, row0 + n64 * 64, bar);
                }
                __syncwarp();
                ++issued;
                r.next(n_stages);
            }
        }
        if (lane == 0) {
            misc->stages = n_stages;
            misc->issued = issued;
        }
    } else if (warp == kIssuerWarp && rank == 1) {
        const uint32_t peer_full = cluster_addr(full, 0);
        Ring r;
        bool ok = true;
        for (int j = first; ok && j < total; j += step)
            for (int ks = 0; ok && ks < k_stages; ++ks) {
                ok = wait(&full[r.slot], r.phase, abort_flag, p.status, lim);
                tc_fence_after();           // this CTA's scale columns before the pair's MMAs
                tc_fence_before();
                if (!ok) break;
                if (lane == 0) mbar_arrive_cluster(peer_full + r.slot * 8);
                __syncwarp();
                r.next(n_stages);
            }
        if (lane == 0) misc->relay = r.phase * n_stages + r.slot;
    } else if (warp == kIssuerWarp) {
        const bool leader = elect_one();
        const uint32_t a_base = smem_u32(smem), b_base = smem_u32(b_ring);
        const int last_steps = (p.K - (k_stages - 1) * kStageK + 63) >> 6;
        // M = 256: the descriptor's M field (units of 16) is twice idesc_fp4's.
        const uint32_t m256 = (128u >> 4) << 24;
        const uint32_t id0 = idesc_fp4<kNv>(kPairN, 0) + m256, id2 = idesc_fp4<kNv>(kPairN, kNv ? 0 : 2) + m256;
        Ring r;
        uint32_t sf = 0, buf = 0, acc_phase = 1;
        bool ok = true;
        for (int j = first; ok && j < total; j += step) {
            const uint32_t d = tmem + buf * kAccCols;
            ok = wait(&acc_empty[buf], acc_phase, abort_flag, p.status, lim);
            for (int ks = 0; ok && ks < k_stages; ++ks) {
                ok = wait(&full[r.slot], r.phase, abort_flag, p.status, lim);
                if (!ok) break;
                tc_fence_after();
                const uint32_t sfa = tmem + kSfCol0 + (kNv ? sf : r.slot) * C::kCols;
                const uint32_t sfb = sfa + C::W * 4;
                const uint64_t a_desc = smem_desc_sw128(a_base + r.slot * kPairABytes);
                const uint64_t b_desc = smem_desc_sw128(b_base + r.slot * kPairBBytes);
                const int steps = ks == k_stages - 1 ? last_steps : 4;
                if (leader) {
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        if (t >= steps) break;
                        const int word = kNv ? t : t >> 1;
                        mma_fp4_pair<kNv>(d, a_desc + 2 * t, b_desc + 2 * t, t & 1 ? id2 : id0, sfa + 4 * word,
                                          sfb + 8 * word, t > 0 || ks > 0);
                    }
                    mma_commit_pair(&empty[r.slot], 3);
                    if (ks == k_stages - 1) mma_commit_pair(&acc_full[buf], 3);
                }
                __syncwarp();
                sf ^= 1u;
                r.next(n_stages);
            }
            buf ^= 1u;
            acc_phase ^= buf == 0;
        }
        if (leader) mma_commit_pair(final_bar, 1);
        __syncwarp();
        wait(final_bar, 0, nullptr, p.status, lim);
    } else if (warp < kEpilogueWarp) {
        const ScaleEnv v = {&p, roff, ioff, abort_flag, first, step, total};
        constexpr int RW = kPairN / 32, RA = 4, kStep = GroupRow<kNv>::kStep;
        const Staging g = {smem + kPairOffStaging, (RW + RA) * (kShift ? uint32_t(kShiftStep) : kStep), raw_bars,
                           raw_bars + kDepth, raw_bars + 2 * kDepth};
        const int cols = kSwiglu ? p.I : p.N;
        const int64_t w_rows = static_cast<int64_t>(E) * p.N;
        // All 192 weight rows, in the order of the MMA's columns.
        const auto w_row = [&](const Item &it, int q) {
            const int n = kSwiglu ? (q >= 3 ? q - 3 : q) * 32 + lane : q * 32 + lane;
            return static_cast<int64_t>(it.e) * p.N + (kSwiglu && q >= 3 ? p.I : 0) + min(it.n0 + n, cols - 1);
        };
        const auto a_row = [&](const Item &it, int q) {
            int row0, valid;
            pair_rows(it, rank, &row0, &valid);
            return static_cast<int64_t>(min(row0 + min(lane + 32 * q, max(valid - 1, 0)), p.rows - 1));
        };
        const auto w_used = [](const Item &) { return RW; };
        // Long bands nearly always use all; leaving some out cost 7% (NVFP4, 4,096 rows).
        const auto a_used = [](const Item &) { return RA; };
        const uint32_t sf_tmem = tmem + kSfCol0 + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        if (warp >= kConvertWarp) {
            convert_scales<kNv, kShift, RA, RW, kPairM, kTile>(v, g, RW, 0, sf_tmem, full, empty, n_stages,
                                                               misc, p.windows, a_row, w_row, a_used, w_used);
        } else if constexpr (kShift) {
            if (warp == kCopyWarp)
                copy_scales_shift<RW, kPairM, kTile>(v, g, 0, p.w_scales, w_rows, p.windows, w_row, w_used);
            else
                copy_scales_shift<RA, kPairM, kTile>(v, g, RW, p.a_scales, p.rows, p.windows, a_row, a_used);
        } else if (warp == kCopyWarp) {
            // Two 96-row boxes of weights (gate and up, or 192 rows), 64-row boxes of
            // this CTA's tokens.
            copy_scales<kPairM, kTile>(
                v, g,
                [&](const Item &it, int i, uint32_t dst, uint64_t *bar) {
                    const int x = i * GroupRow<kNv>::kBytes;
                    int row0, valid;
                    pair_rows(it, rank, &row0, &valid);
                    tma_load_3d(dst, &tm_ws, x, it.n0, kSwiglu ? 2 * it.e : it.e, bar);
                    tma_load_3d(dst + 3 * kStep, &tm_ws, x, kSwiglu ? it.n0 : it.n0 + kPairN / 2,
                                kSwiglu ? 2 * it.e + 1 : it.e, bar);
                    for (int q = 0; 32 * q < valid; q += 2)
                        tma_load_2d(dst + (RW + q) * kStep, &tm_as, x, row0 + 32 * q, bar);
                },
                [&](const Item &it) {
                    int row0, valid;
                    pair_rows(it, rank, &row0, &valid);
                    return (RW + (valid + 63) / 64 * 2) * kStep;
                });
        }
    } else {
        const int quarter = warp & 3, half = (warp - kEpilogueWarp) >> 2;
        const float a2 = kNv ? __ldg(p.a_scale_2) : 1.0f;
        const float h2 = kNv && kSwiglu ? __ldg(p.h_scale_2) : 1.0f;
        if (!(h2 > 0.0f && h2 < __uint_as_float(kF32Inf)) && tid == kThreads - 1) set_status(p.status, MOE_ERR_DATA);
        // The three blocks of an item go two to one warp of a lane quarter and one to the
        // other, the other way round for the next item.
        uint32_t buf = 0, phase = 0;
        int turn = 0;
        uint8_t *box = smem + kPairOffStore + (warp - kEpilogueWarp) * kStoreBytes;
        for (int j = first; j < total; j += step) {
            const Item it = decode_item<kPairM, kTile>(j, roff, ioff, E, p.n_tiles);
            int row0, valid;
            pair_rows(it, rank, &row0, &valid);
            if (!wait(&acc_full[buf], phase, abort_flag, p.status, lim)) break;
            tc_fence_after();
            const uint32_t acc = tmem + buf * kAccCols + (static_cast<uint32_t>(quarter * 32) << 16);
            const float scale = kNv ? __ldg(p.w_scale_2 + it.e) * a2 : 1.0f;
            const uint32_t bar = cluster_addr(&acc_empty[buf], 0);
            if constexpr (kSwiglu)
                pair_store_swiglu<kNv>(p, acc, row0 + quarter * 32, valid - quarter * 32, it.n0, half ^ turn, scale,
                                       h2, bar);
            else {
                const int row = row0 + quarter * 32, cols = min(kPairN, (p.N - it.n0 + 31) & ~31);
                if (!out_tma || valid < quarter * 32 + 32)
                    pair_store_plain(p, acc, row, valid - quarter * 32, it.n0, half, cols, scale, out_vec, bar);
                else if (p.out_bf16)
                    pair_store_box<true>(&tm_out, acc, row, it.n0, half ^ turn, cols, scale, box, bar);
                else
                    pair_store_box<false>(&tm_out, acc, row, it.n0, half, cols, scale, box, bar);
            }
            buf ^= 1u;
            turn ^= 1;
            if (buf == 0) phase ^= 1u;
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    // Neither CTA frees its tensor memory or leaves while the pair's MMAs, commits
    // or the peer's arrivals may still reach it.
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    if (warp == kProducerWarp) {
        if (lane == 0)
            finish(kPairOffBars, kPairOffMisc, (p.K + kStageK - 1) / kStageK, true, p.status, p.wait_limit_ns);
        __syncwarp();
        tmem_dealloc_pair(tmem, kTmemCols);
    }
    cluster_sync();
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

// Scale bytes [outer][rows][scale_row] in boxes of one group's bytes a row by `box_rows`
// rows; bytes past a row's end and rows past the last of an expert (half) read as zeros.
bool encode_scales(CUtensorMap *map, const void *base, int scale_row, int64_t rows, int64_t outer, uint32_t box_rows,
                   bool nv) {
    PFN_cuTensorMapEncodeTiled_v12000 encode = encode_fn();
    if (!encode) return false;
    const cuuint64_t pitch = static_cast<cuuint64_t>(scale_row);
    cuuint64_t dims[3] = {pitch, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(outer)};
    cuuint64_t strides[2] = {pitch, pitch * static_cast<cuuint64_t>(rows)};
    cuuint32_t box[3] = {nv ? 64u : 32u, box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, outer ? 3 : 2, const_cast<void *>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, nv ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Outputs [rows, N] in boxes of 128 bytes by 32 rows.
bool encode_out(CUtensorMap *map, void *base, int64_t rows, int N, bool bf16) {
    PFN_cuTensorMapEncodeTiled_v12000 encode = encode_fn();
    if (!encode) return false;
    const uint32_t size = bf16 ? 2 : 4;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(N) * size};
    cuuint32_t box[2] = {128 / size, 32};
    cuuint32_t estr[2] = {1, 1};
    return encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, base, dims,
                  strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Shared-memory attribute of a kernel, set once per device (the mask is the
// caller's, one per kernel).
bool set_smem(const void *kernel, int bytes, std::atomic<uint64_t> &mask) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
    if (bit && (mask.load(std::memory_order_acquire) & bit)) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
    mask.fetch_or(bit, std::memory_order_release);
    return true;
}

// Bands of at least this many rows run in CTA pairs.  Calls of 24 bands at K = 4,096 (w13
// with SwiGLU) and K = 2,048 (w2, f32), N = 4,096, one CTA / pair, us, the pairs' with 3 to 4
// us for the other class's empty launch:
//   rows a band           64         128         160         192         256         512        2,048
//   MXFP4 SwiGLU  44.1 / 52.9 55.6 / 53.9 59.9 / 54.5 61.8 / 54.7 73.3 / 55.5 126 / 85.3 412 / 278
//   MXFP4 plain   31.2 / 36.8 35.1 / 39.5 39.0 / 41.1 41.2 / 42.6 48.6 / 45.6 75.6 / 67.8 249 / 212
//   NVFP4 SwiGLU  46.9 / 55.6 57.5 / 56.7 61.5 / 57.7 63.9 / 58.8 75.7 / 60.9 128 / 97.0 417 / 323
//   NVFP4 plain   31.8 / 37.7 36.9 / 41.2 38.8 / 42.3 41.5 / 44.1 50.0 / 47.2 76.1 / 69.9 243 / 217
// (a chunk is 96 tokens with SwiGLU and 192 without, against 256 in a pair).
constexpr int kPairBandSwiglu = 112, kPairBand = 160;
// Calls of fewer multiplications are one launch, without pairs: what pairs gain there is less
// than the empty launch (MXFP4, bands x rows, one CTA / pair: SwiGLU 8 x 128 23.0 / 27.0, 8 x
// 192 26.9 / 27.0, 8 x 256 33.2 / 27.3, 4 x 512 31.2 / 26.9; plain 8 x 256 20.8 / 22.7, 8 x
// 512 33.1 / 32.9; 8 x 192 rows are 2.6e10 with SwiGLU and 1.3e10 without).  The rule does not
// see the bands: a large call of short ones alone pays an empty launch of pairs, most of it
// beside the other (2,048 tokens, top-6 of 256 experts, bands of up to 63 rows, pairs / none:
// w13 MXFP4 338 / 338, NVFP4 364 / 362, w2 204 / 202 and 211 / 209).
constexpr double kPairMacsSwiglu = 2.5e10, kPairMacs = 4.5e10;

std::atomic<int> g_pairing{MOE_PAIRING_AUTO};      // process-wide

template <bool kNv, bool kSwiglu, bool kShift>
moe_status launch(const Fp4Gemm &g, cudaStream_t stream, int num_sms, int *launches) {
    constexpr int band = kSwiglu ? kPairBandSwiglu : kPairBand;
    const double macs = static_cast<double>(g.rows) * g.N * g.K;
    const int mode = g_pairing.load(std::memory_order_relaxed);
    const bool pairs = mode != MOE_PAIRING_OFF && g.rows >= band &&
                       (mode == MOE_PAIRING_ON || g.E == 1 || macs >= (kSwiglu ? kPairMacsSwiglu : kPairMacs));
    const bool singles = !pairs || g.E > 1;
    // The pairs first, the short bands as a programmatic dependent launch: their CTAs take the
    // SMs that the pairs leave (one launch after the other: Zipf prefill w13 407 us for 400,
    // full layer w2 311 for 304).  The other way round, clusters start out of order as SMs
    // come free one by one (full layer w13 with SwiGLU 451 -> 490 us).
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
    p.scale_row = g.K / (kNv ? 16 : 32);
    p.windows = (reinterpret_cast<uintptr_t>(g.w_scales) | reinterpret_cast<uintptr_t>(g.a_scales)) % 16 == 0;
    p.wait_limit_ns = g.wait_limit_ns;
    const int64_t w_rows = static_cast<int64_t>(g.E) * g.N;
    const int columns = kSwiglu ? g.N / 2 : g.N;
    CUtensorMap tm_w, tm_a64, tm_a2, tm_a128, tm_ws, tm_as;
    if (!encode_codes(&tm_a64, g.a_codes, g.rows, g.K, 64)) return MOE_ERR_CUDA;
    tm_ws = tm_as = tm_a64;         // not used where threads copy the scales
    const auto scale_maps = [&](uint32_t w_box, uint32_t a_box) {
        return kShift || (encode_scales(&tm_ws, g.w_scales, p.scale_row, columns,
                                        static_cast<int64_t>(g.E) * (kSwiglu ? 2 : 1), w_box, kNv) &&
                          encode_scales(&tm_as, g.a_scales, p.scale_row, g.rows, 0, a_box, kNv));
    };
    *launches = 0;
    if (pairs) {
        static std::atomic<uint64_t> mask{0};
        const auto kernel = fp4_gemm_pair_kernel<kNv, kSwiglu, kShift>;
        if (!set_smem(reinterpret_cast<const void *>(kernel), kPairSmem, mask) ||
            !encode_codes(&tm_w, g.w_codes, w_rows, g.K, kPairN / 2) ||
            !encode_codes(&tm_a2, g.a_codes, g.rows, g.K, 32) || !encode_codes(&tm_a128, g.a_codes, g.rows, g.K, 128) ||
            !scale_maps(kPairN / 2, 64))
            return MOE_ERR_CUDA;
        constexpr int tile = kSwiglu ? kPairN / 2 : kPairN;
        p.n_tiles = (columns + tile - 1) / tile;
        p.band_lo = band;
        p.band_hi = INT32_MAX;
        const int out_vec = reinterpret_cast<uintptr_t>(g.out) % 32 == 0 && g.N % (g.out_bf16 ? 16 : 8) == 0;
        // TMA wants whole 16-byte pieces; smaller alignments store by threads.
        const int out_tma = !kSwiglu && reinterpret_cast<uintptr_t>(g.out) % 16 == 0 && g.N % (g.out_bf16 ? 8 : 4) == 0;
        CUtensorMap tm_out = tm_w;
        if (out_tma && !encode_out(&tm_out, g.out, g.rows, g.N, g.out_bf16)) return MOE_ERR_CUDA;
        kernel<<<num_sms & ~1, kThreads, kPairSmem, stream>>>(tm_w, tm_a128, tm_a64, tm_a2, tm_ws, tm_as, tm_out, p,
                                                              out_vec, out_tma);
        if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;
        ++*launches;
    }
    if (singles) {
        static std::atomic<uint64_t> mask{0};
        const auto kernel = fp4_gemm_kernel<kNv, kSwiglu, kShift>;
        if (!set_smem(reinterpret_cast<const void *>(kernel), kSmemBytes, mask) ||
            !encode_codes(&tm_w, g.w_codes, w_rows, g.K, kTileN) || !encode_codes(&tm_a2, g.a_codes, g.rows, g.K, 16) ||
            !scale_maps(kTileN, 32))
            return MOE_ERR_CUDA;
        p.n_tiles = (columns + kTileN - 1) / kTileN;
        p.band_lo = 1;
        p.band_hi = pairs ? band - 1 : INT32_MAX;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr.val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(num_sms);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kSmemBytes;
        cfg.stream = stream;
        cfg.attrs = &attr;
        cfg.numAttrs = pairs ? 1 : 0;
        if (cudaLaunchKernelEx(&cfg, kernel, tm_w, tm_a64, tm_a2, tm_ws, tm_as, p) != cudaSuccess) return MOE_ERR_CUDA;
        ++*launches;
    }
    return MOE_OK;
}

}  // namespace fp4

void set_fp4_pairing(int mode) { fp4::g_pairing.store(mode, std::memory_order_relaxed); }

moe_status launch_fp4_gemm(const Fp4Gemm &g, bool nv, bool swiglu, cudaStream_t stream, int num_sms, int *launches) {
    *launches = 0;
    if (g.rows == 0) return MOE_OK;
    const uintptr_t scales = reinterpret_cast<uintptr_t>(g.w_scales) | reinterpret_cast<uintptr_t>(g.a_scales);
    const bool shift = (g.K / (nv ? 16 : 32)) % 16 != 0 || scales % 16 != 0;
    if (shift)
        return nv ? swiglu ? fp4::launch<true, true, true>(g, stream, num_sms, launches)
                           : fp4::launch<true, false, true>(g, stream, num_sms, launches)
                  : swiglu ? fp4::launch<false, true, true>(g, stream, num_sms, launches)
                           : fp4::launch<false, false, true>(g, stream, num_sms, launches);
    return nv ? swiglu ? fp4::launch<true, true, false>(g, stream, num_sms, launches)
                       : fp4::launch<true, false, false>(g, stream, num_sms, launches)
              : swiglu ? fp4::launch<false, true, false>(g, stream, num_sms, launches)
                       : fp4::launch<false, false, false>(g, stream, num_sms, launches);
}

}  // namespace moe
