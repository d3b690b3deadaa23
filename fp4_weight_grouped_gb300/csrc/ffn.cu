// Dense gated feed-forward block in bf16, forward and backward:
//
//   [g | u] = x W13^T          h = silu(g) u         out = h W2^T
//   dh = dout W2               dg = dh u s (1 + g (1 - s))      du = dh g s,   s = 1 / (1 + e^-g)
//   dx = [dg | du] W13         dW13 = [dg | du]^T x             dW2 = dout^T h
//
// Every product is D[m, n] = sum_k A(m, k) B(n, k) with each operand stored along k (rows
// of k) or along m / n (rows of m or n, for the products whose k is an outer dimension):
// the tensor core reads either from shared memory as TMA leaves it, so nothing is
// transposed in memory.
//
// Bound by the tensor pipe for many tokens (hidden 4,096, inter 2,048: 8,192 tokens forward
// 212 us, 1,950 TFLOP/s, forward and backward 660, 1,870, in a short burst; one call after another
// the power cap makes the latter 770, 1,600), below some 512 by start-up, about
// 6 us a launch (64 tokens 20.7 us, of which the MMAs of 256 rows take 8; 250 tokens of hidden
// 1,032, inter 520, forward and backward 36.6 us in four launches).
//
//  * CTA pairs (tcgen05.mma cta_group::2): 256 rows by kN columns an item, the rows split
//    over the pair's tensor memory, either CTA fetching half of A and half of B.  64 k are
//    128-byte rows in the 128-byte swizzle, an atom; a stage is one of them or two.
//  * Accumulators are double-buffered: eight epilogue warps empty one while the other fills (four took
//    longer than the MMAs for the gradient's part: 64 tokens' backward 45 -> 39 us).
//  * SwiGLU: the even CTA fetches gate rows of W13 and the odd CTA the matching up rows, so
//    a thread finds g and u of one output in two column ranges of its own lane.
//  * The gradient's elementwise part is the epilogue of dh: dh is never stored.
//  * Sums are f32, as the tensor core has it: what does not fit is cut off, up to a step in eight
//    products (2^14 tokens of one sign: 8e-5 of the sum; 2^19, the most that is taken: 0.0034).
//  * h, dg and du are rounded to bf16 once, where they are stored for the next product, whose
//    operands are bf16 (f32 ones would be tf32, at half of the rate and twice the bytes).  g and u
//    are read back by the gradient's elementwise part alone and could be f32; bf16 halves the memory
//    that a training step holds for them between forward and backward, and saves their bytes (134 MB
//    for 8,192 tokens of inter 2,048: some 20 us).  dW13 and dx carry g and u's rounding, dg and du's
//    and their own: 0.0030 of the norm, against 0.0017 for their own alone.
//  * Persistent pairs over a list of jobs; a job is one product.
//  * Every wait is bounded (see wait_bounded and pair_drain.h).
#include <atomic>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <stdint.h>

#include "device_common.cuh"
#include "launch.h"
#include "pair_drain.h"
#include "pair_schedule.h"
#include "tensor_map.h"
#include "vec_io.cuh"

namespace moe {
namespace ffn {

constexpr int kProducerWarp = 0, kIssuerWarp = 1, kEpilogueWarp = 2;
constexpr int kEpilogueWarps = 8;                  // two a quarter of the tensor memory, half of the columns each
constexpr int kThreads = 32 * (kEpilogueWarp + kEpilogueWarps);
constexpr int kStageK = 64;
constexpr int kRows = 128;                         // of A a CTA
constexpr int kABytes = kRows * 128;
constexpr int kMaxJobs = 2;
constexpr int kFewRows = 8;                        // tokens up to which matvec.cu streams the weights

constexpr int kRingBytes = 230400;                 // of shared memory, for the stages
constexpr int kMaxStages = 16;
constexpr int kNumBars = 2 * kMaxStages + 5;
constexpr int kOffMisc = kRingBytes + kNumBars * 8;
constexpr int kSmem = kRingBytes + 1024 + 1024;
static_assert(kSmem <= 232448 && kOffMisc + 32 <= kRingBytes + 1024, "shared memory budget");

template <int kN>
struct Tile {
    static constexpr int kBRows = kN / 2;          // of B a CTA
    static constexpr int kBBytes = kBRows * 128;
    // Of 64 k a stage: the short stages of narrow items take two (64 tokens 26.8 us with one,
    // 23.4 with two, 26.3 with three, whose ring has three stages).
    static constexpr int kAtoms = kN == 64 ? 2 : 1;
    static constexpr int kCols = 2 * kN;           // of tensor memory
    // Narrow items, those of few tokens, have stages that hold no more rows of A than the jobs do.
    static constexpr bool kSized = kN == 64;
    static constexpr int kStageBytes = kAtoms * (kABytes + kBBytes);
    static constexpr int kStages = kRingBytes / kStageBytes;
    // Whether a launch in a chain fetches its first B ahead of the wait for A (a training step of
    // 250 tokens, hidden 1,032, inter 520: 38.8 -> 37.8 us).  Narrow items lose by it (64 tokens
    // 20.7 -> 21.4): their B is the weights, which the launch before still reads from memory too.
    static constexpr bool kAhead = kN > 64;
    static_assert(kStages <= kMaxStages);
};

enum Epilogue { kStore, kGate, kGateBack };

struct Job {
    int m, n, k;                 // n: columns of the output (gate: of h)
    int tiles_m, tiles_n, k_stages;
    int first, full;             // first item; items of all kN columns, the others have half
    int a_mn, b_mn;              // operand stored along m (n) instead of k
    int a_rows, odd_a;           // rows of A in a box (along k), whether the odd CTA has any
    int tile_cols, b_step;       // output columns an item; gate: the odd CTA's first row of B
    int epilogue;
    int out_f32;
    void *out;                   // [m, n]; gate: h; gate back: dgu [m, 2 n]
    uint16_t *gu;                // [m, 2 n]: gate: written if given; gate back: read
};

struct Args {
    CUtensorMap a[kMaxJobs], b[kMaxJobs], b_half[kMaxJobs];      // b_half: boxes of half the rows
    Job job[kMaxJobs];
    int jobs, items;
    PairSchedule schedule;
    int stages, stage_bytes, a_bytes;        // of the ring: atoms of A, then those of B
    int chained;                             // A comes from the launch before
    int *status;
    uint64_t wait_limit_ns;
};

struct Misc {
    uint32_t tmem;
    int abort;
    uint32_t issued;
    uint32_t odd_issued, odd_abort;     // the odd CTA's, left with the even one at the end
};

// One box into this CTA's shared memory, its bytes counted on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap *map, int32_t x, int32_t y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// Descriptors by halves: a stage moves their addresses, all in the lower one.
__device__ __forceinline__ void mma_pair(uint32_t d, uint32_t a, uint32_t a_hi, uint32_t b, uint32_t b_hi, uint32_t idesc,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "mov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %5, p;\n\t}" ::"r"(d),
        "r"(a), "r"(a_hi), "r"(b), "r"(b_hi), "r"(idesc), "r"(accumulate)
        : "memory");
}

// An operand in rows of m or n: boxes of 64 elements (128 bytes) by 64 k, one behind another.
// Eight k are 1,024 bytes apart, 64 elements a box.
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(8192u >> 4) << 16;          // next 64 elements
    d |= static_cast<uint64_t>(1024u >> 4) << 32;          // next 8 k
    d |= 1ull << 46;
    d |= 2ull << 61;
    return d;
}

__device__ __noinline__ bool wait_slow(uint64_t *bar, uint32_t parity, volatile int *abort_flag, int *status,
                                       uint64_t lim) {
    return wait_bounded(bar, parity, abort_flag, status, lim);
}

// By one thread.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag, int *status,
                                     uint64_t lim) {
    if (mbar_try_wait(bar, parity)) return true;
    return wait_slow(bar, parity, abort_flag, status, lim);
}

struct Item {
    int job, m0, n0;
    int half;                    // half as many columns
};

__device__ __forceinline__ Item item_of(const Args &p, int i) {
    int j = 0;
    while (j + 1 < p.jobs && i >= p.job[j + 1].first) ++j;
    const Job &w = p.job[j];
    const int at = i - w.first, over = at - w.full;
    const int tile = over < 0 ? at : w.full + (over >> 1);
    return {j, tile / w.tiles_n * 2 * kRows, tile % w.tiles_n * w.tile_cols + (over >= 0 && (over & 1) ? w.tile_cols / 2 : 0),
            over >= 0};
}

// What the odd CTA copies in stage i of a pair's stream.
template <int kN>
__device__ __noinline__ uint32_t odd_bytes(const Args &p, int pair, uint32_t i) {
    int item = pair;
    for (; p.schedule.next(pair, item) < p.items; item = p.schedule.next(pair, item)) {
        const uint32_t n = p.job[item_of(p, item).job].k_stages;
        if (i < n) break;
        i -= n;
    }
    const Item it = item_of(p, item);
    const Job &w = p.job[it.job];
    return Tile<kN>::kAtoms * (w.odd_a * w.a_rows * 128 + (Tile<kN>::kBBytes >> it.half));
}

// 16 consecutive outputs of a row at column n: n columns are a multiple of 8.
__device__ __forceinline__ void store16(void *row, int n, int cols, bool f32, bool sector, const float (&v)[16]) {
    if (f32) {
        float *o = static_cast<float *>(row) + n;
#pragma unroll
        for (int i = 0; i < 16; i += 4)
            if (n + i < cols) *reinterpret_cast<float4 *>(o + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        return;
    }
    uint16_t *o = static_cast<uint16_t *>(row) + n;
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
    if (sector && n + 16 <= cols) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(o), "r"(w[0]), "r"(w[1]),
                     "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
        return;
    }
    if (n < cols) *reinterpret_cast<uint4 *>(o) = make_uint4(w[0], w[1], w[2], w[3]);
    if (n + 8 < cols) *reinterpret_cast<uint4 *>(o + 8) = make_uint4(w[4], w[5], w[6], w[7]);
}

// 16 consecutive elements of a row at column n, as they are; zeros past the last column.
__device__ __forceinline__ void load16(const uint16_t *row, int n, int cols, uint4 (&v)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
        v[h] = n + 8 * h < cols ? __ldg(reinterpret_cast<const uint4 *>(row + n + 8 * h)) : make_uint4(0, 0, 0, 0);
}

__device__ __forceinline__ float bf16_of(const uint4 (&v)[2], int i) {
    const uint4 &q = v[i >> 3];
    const uint32_t w = (i & 7) < 2 ? q.x : (i & 7) < 4 ? q.y : (i & 7) < 6 ? q.z : q.w;
    return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
}

// dg and du of one element; s and 1 - s both without cancellation.
__device__ __forceinline__ void gate_back(float dh, float g, float u, float &dg, float &du) {
    float t, r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(t) : "f"(-1.4426950408889634f * fabsf(g)));
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.0f + t));
    const float s = g >= 0.0f ? r : t * r, c = g >= 0.0f ? t * r : r;
    dg = dh * u * (s * fmaf(g, c, 1.0f));
    du = dh * (g * s);
}

template <int kN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) ffn_kernel(const __grid_constant__ Args p) {
    using T = Tile<kN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kRingBytes);       // the even CTA's count
    uint64_t *empty = full + kMaxStages;
    uint64_t *acc_full = empty + kMaxStages, *acc_empty = acc_full + 2, *final_bar = acc_empty + 2;
    Misc *misc = reinterpret_cast<Misc *>(smem + kOffMisc);
    const uint32_t n_stages = T::kSized ? p.stages : T::kStages;
    const uint32_t stage_bytes = T::kSized ? p.stage_bytes : T::kStageBytes, a_bytes = T::kSized ? p.a_bytes : kABytes;
    volatile int *abort_flag = &misc->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1;
    const uint64_t lim = p.wait_limit_ns;

    if (threadIdx.x == 0) {
        misc->abort = 0;
        misc->issued = 0;
        for (uint32_t i = 0; i < n_stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 2 * kEpilogueWarps);
        }
        mbar_init(final_bar, 1);
        mbar_fence_init();
    }
    if (warp == kIssuerWarp) tmem_alloc_pair(&misc->tmem, T::kCols);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = misc->tmem;
    // A launch in a chain starts under the end of the one before, whose outputs are its A.
    if (warp != kProducerWarp) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    }

    // The two loops that feed the tensor core are one thread each, an instruction after the
    // other: no votes or reconvergence of a warp, and what they need of a job in registers
    // ahead of them (64 tokens: read from the parameters stage by stage 265 ns a stage whatever
    // its work, from registers 172).
    if (warp == kProducerWarp) {
        if (elect_one()) {
            const uint32_t base = smem_u32(smem), bar0 = cluster_addr(full, 0);
            uint32_t slot = 0, phase = 1, issued = 0, ahead = 0;
            bool ok = true;
            if (!T::kAhead) asm volatile("griddepcontrol.wait;" ::: "memory");
            for (int i = pair; ok && i < p.items; i = p.schedule.next(pair, i)) {
                const Item it = item_of(p, i);
                const Job &w = p.job[it.job];
                const CUtensorMap *ma = &p.a[it.job], *mb = it.half ? &p.b_half[it.job] : &p.b[it.job];
                const int b_rows = T::kBRows >> it.half;
                const int row_a = it.m0 + rank * kRows;
                const int row_b = it.n0 + rank * (w.epilogue == kGate ? w.b_step : b_rows);
                const uint32_t bytes = T::kAtoms * (w.a_rows * 128 * (1 + w.odd_a) + 2 * (T::kBBytes >> it.half));
                const bool a_mn = w.a_mn, b_mn = w.b_mn, has_a = rank == 0 || w.odd_a;
                const auto load_a = [&](uint32_t at, int k) {
                    const uint32_t bar = bar0 + at * 8;
#pragma unroll
                    for (int h = 0; h < T::kAtoms; ++h) {
                        const uint32_t a = base + at * stage_bytes + h * a_bytes;
                        if (a_mn) {
                            tma_load_pair(a, ma, row_a, k + h * kStageK, bar);
                            tma_load_pair(a + 8192, ma, row_a + 64, k + h * kStageK, bar);
                        } else if (has_a) {
                            tma_load_pair(a, ma, k + h * kStageK, row_a, bar);
                        }
                    }
                };
                const auto load_b = [&](uint32_t at, int k) {
                    const uint32_t bar = bar0 + at * 8;
                    if (rank == 0) mbar_arrive_expect_tx(&full[at], bytes);
#pragma unroll
                    for (int h = 0; h < T::kAtoms; ++h) {
                        const uint32_t b = base + at * stage_bytes + T::kAtoms * a_bytes + h * T::kBBytes;
                        if (b_mn) {
#pragma unroll
                            for (int q = 0; q < T::kBRows / 64 * 64; q += 64)
                                if (q < b_rows) tma_load_pair(b + q * 128, mb, row_b + q, k + h * kStageK, bar);
                        } else {
                            tma_load_pair(b, mb, k + h * kStageK, row_b, bar);
                        }
                    }
                };
                constexpr int kStep = T::kAtoms * kStageK;
                if (T::kAhead && p.chained && i == pair) {      // B, which the launch before does not write
                    ahead = min(min(n_stages, 4u), static_cast<uint32_t>(w.k_stages));
                    for (uint32_t q = 0; q < ahead; ++q) load_b(q, q * kStep);
                    asm volatile("griddepcontrol.wait;" ::: "memory");
                }
                const int k_end = w.k_stages * kStep;
                for (int k = 0; k < k_end; k += kStep) {
                    ok = wait(&empty[slot], phase, abort_flag, p.status, lim);
                    if (!ok) break;
                    if (!T::kAhead || issued >= ahead) load_b(slot, k);
                    load_a(slot, k);
                    ++issued;
                    slot = slot + 1 == n_stages ? 0 : slot + 1;
                    phase ^= slot == 0;
                }
            }
            misc->issued = issued;
        }
    } else if (warp == kIssuerWarp && rank == 0) {
        if (elect_one()) {
            const uint32_t base = smem_u32(smem);
            uint32_t slot = 0, phase = 0, buf = 0, acc_phase = 1;
            bool ok = true;
            for (int i = pair; ok && i < p.items; i = p.schedule.next(pair, i)) {
                const Item it = item_of(p, i);
                const Job &w = p.job[it.job];
                const uint32_t idesc = idesc_bf16_f32(2 * kRows, kN >> it.half) | (w.a_mn ? 1u << 15 : 0) | (w.b_mn ? 1u << 16 : 0);
                // 16 k further: 32 bytes along a row, or 16 rows of 128 bytes.
                const uint32_t a_step = w.a_mn ? 128 : 2, b_step = w.b_mn ? 128 : 2;
                const uint64_t da0 = w.a_mn ? smem_desc_mn(base) : smem_desc_sw128(base);
                const uint64_t db0 = w.b_mn ? smem_desc_mn(base + T::kAtoms * a_bytes) : smem_desc_sw128(base + T::kAtoms * a_bytes);
                const uint32_t d = tmem + buf * kN;
                const int k_stages = w.k_stages;
                ok = wait(&acc_empty[buf], acc_phase, abort_flag, p.status, lim);
                tc_fence_after();
                for (int ks = 0; ok && ks < k_stages; ++ks) {
                    ok = wait(&full[slot], phase, abort_flag, p.status, lim);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t at = slot * (stage_bytes >> 4), da = static_cast<uint32_t>(da0) + at,
                                   db = static_cast<uint32_t>(db0) + at;
#pragma unroll
                    for (int t = 0; t < T::kAtoms * kStageK / 16; ++t)
                        mma_pair(d, da + (t & 3) * a_step + (t >> 2) * (a_bytes >> 4), da0 >> 32,
                                 db + (t & 3) * b_step + (t >> 2) * (T::kBBytes >> 4), db0 >> 32, idesc, t > 0 || ks > 0);
                    mma_commit_pair(&empty[slot], 3);
                    if (ks == k_stages - 1) mma_commit_pair(&acc_full[buf], 3);
                    slot = slot + 1 == n_stages ? 0 : slot + 1;
                    phase ^= slot == 0;
                }
                buf ^= 1u;
                acc_phase ^= buf == 0;
            }
            mma_commit_pair(final_bar, 1);
            wait(final_bar, 0, nullptr, p.status, lim);
        }
    } else if (warp >= kEpilogueWarp) {
        const int quarter = warp & 3, side = (warp - kEpilogueWarp) >> 2;
        uint32_t buf = 0, phase = 0;
        for (int i = pair; i < p.items; i = p.schedule.next(pair, i)) {
            const Item it = item_of(p, i);
            const Job &w = p.job[it.job];
            if (!warp_wait_bounded(&acc_full[buf], phase, abort_flag, p.status, lim)) break;
            tc_fence_after();
            const uint32_t acc = tmem + buf * kN + (static_cast<uint32_t>(quarter * 32) << 16);
            const int64_t row = it.m0 + static_cast<int64_t>(rank) * kRows + quarter * 32 + lane;
            const bool real = row < w.m;
            const int cols = kN >> it.half;
            const int width = w.epilogue == kGateBack ? 2 * w.n : w.n;
            uint8_t *out = static_cast<uint8_t *>(w.out) + (real ? row : 0) * width * (w.out_f32 ? 4 : 2);
            const bool sector = (reinterpret_cast<uintptr_t>(w.out) & 31) == 0 && width % 16 == 0;
            if (w.epilogue == kGate) {
                uint16_t *gu = w.gu ? w.gu + (real ? row : 0) * 2 * w.n : nullptr;
                const bool gu_sector = (reinterpret_cast<uintptr_t>(w.gu) & 31) == 0 && w.n % 16 == 0;
#pragma unroll 1
                for (int c = side * cols / 4; c < (side + 1) * cols / 4; c += 16) {
                    const int n = it.n0 + c;
                    if (n >= w.n) break;
                    uint32_t rg[16], ru[16];
                    tmem_ld16(acc + c, rg);
                    tmem_ld16(acc + cols / 2 + c, ru);
                    tmem_ld_wait();
                    float g[16], u[16], h[16];
#pragma unroll
                    for (int q = 0; q < 16; ++q) {
                        g[q] = __uint_as_float(rg[q]);
                        u[q] = __uint_as_float(ru[q]);
                        h[q] = silu_f32(g[q]) * u[q];
                    }
                    if (real) {
                        store16(out, n, w.n, false, sector, h);
                        if (gu) {
                            store16(gu, n, w.n, false, gu_sector, g);
                            store16(gu + w.n, n, w.n, false, gu_sector, u);
                        }
                    }
                    __syncwarp();
                }
            } else {
                const uint16_t *gu = w.gu + (real ? row : 0) * 2 * w.n;
                uint16_t *up = reinterpret_cast<uint16_t *>(out) + w.n;
                // g and u of the next columns are asked for ahead of the work on these.
                uint4 g[2], u[2];
                if (w.epilogue == kGateBack) {
                    load16(gu, it.n0 + side * cols / 2, w.n, g);
                    load16(gu + w.n, it.n0 + side * cols / 2, w.n, u);
                }
#pragma unroll 1
                for (int c = side * cols / 2; c < (side + 1) * cols / 2; c += 16) {
                    const int n = it.n0 + c;
                    if (n >= w.n) break;
                    uint32_t r[16];
                    tmem_ld16(acc + c, r);
                    float v[16];
                    if (w.epilogue == kGateBack) {
                        float du[16];
                        uint4 next_g[2], next_u[2];
                        const int next = c + 16 < (side + 1) * cols / 2 ? n + 16 : w.n;
                        load16(gu, next, w.n, next_g);
                        load16(gu + w.n, next, w.n, next_u);
                        tmem_ld_wait();
#pragma unroll
                        for (int q = 0; q < 16; ++q) gate_back(__uint_as_float(r[q]), bf16_of(g, q), bf16_of(u, q), v[q], du[q]);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            g[h] = next_g[h];
                            u[h] = next_u[h];
                        }
                        if (real) store16(up, n, w.n, false, sector && w.n % 16 == 0, du);
                    } else {
                        tmem_ld_wait();
#pragma unroll
                        for (int q = 0; q < 16; ++q) v[q] = __uint_as_float(r[q]);
                    }
                    if (real) store16(out, n, w.n, w.out_f32, sector, v);
                    __syncwarp();
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(cluster_addr(&acc_empty[buf], 0));
            buf ^= 1u;
            phase ^= buf == 0;
        }
    }
    // Neither CTA frees its tensor memory or leaves while the pair's MMAs, copies, commits or
    // the peer's arrivals may still reach it.
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (rank == 1 && threadIdx.x == 0) {
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr(&misc->odd_issued, 0)), "r"(misc->issued) : "memory");
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr(&misc->odd_abort, 0)), "r"(misc->abort) : "memory");
    }
    cluster_sync();
    tc_fence_after();
    if (rank == 0 && threadIdx.x == 0) {
        if (misc->odd_abort || misc->abort) {       // every copy that was issued lands before the pair leaves
            const uint32_t n1 = misc->odd_issued;
            const uint32_t n0 = misc->issued, n = n0 > n1 ? n0 : n1;
            for (uint32_t i = pair_first(n0, n1, n_stages); i < n; ++i) {
                uint64_t *bar = &full[i % n_stages];
                const uint32_t parity = (i / n_stages) & 1u;
                if (mbar_try_wait(bar, parity)) continue;
                const PairFix f = pair_fix(i, n0, n1, odd_bytes<kN>(p, pair, i));
                if (f.arrive) mbar_arrive_expect_tx(bar, f.expect);
                if (f.complete)
                    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)),
                                 "r"(f.complete)
                                 : "memory");
                if (!wait_bounded(bar, parity, nullptr, p.status, lim)) break;
            }
        }
    }
    if (warp == kIssuerWarp) tmem_dealloc_pair(tmem, T::kCols);
    cluster_sync();
}

// A bf16 matrix [rows, cols] with rows `pitch` elements apart, in boxes of 64 columns by
// box_rows rows; what lies past its edges reads as zeros.
bool encode(CUtensorMap *map, const void *base, int64_t rows, int64_t cols, int64_t pitch, uint32_t box_rows) {
    PFN_cuTensorMapEncodeTiled_v12000 fn = tensor_map_encode();
    if (!fn) return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch) * 2};
    cuuint32_t box[2] = {64, box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// An operand (i, k): [rows of i, k], or with mn [rows of k, i].
struct Operand {
    const void *p;
    int64_t pitch;
    bool mn;
};

struct Product {
    Operand a, b;
    int64_t m, n, k;             // n: rows of B; gate: output columns
    int epilogue;
    void *out;
    int out_f32;
    uint16_t *gu;
};

int64_t count_items(const Product &w, int kN) {
    const int cols = w.epilogue == kGate ? kN / 2 : kN;
    return (w.m + 2 * kRows - 1) / (2 * kRows) * ((w.n + cols - 1) / cols);
}

// An item's time in stages of 64 k, or its epilogue's, which runs beside the next item's stages:
// about four, and where it reads g and u and works out their gradients (256 columns 14 us) 44.
int64_t item_stages(const Product &w, int kN) {
    const int64_t k = (w.k + kStageK - 1) / kStageK, end = w.epilogue == kGateBack ? kN * 11 / 64 : 4;
    return k > end ? k : end;
}

// How a launch's items are shared out: job `first` first, `ahead` rounds (0: none) of the other
// job's items by the pairs without one of its; the stages of the pair that takes longest.
struct Plan {
    int first, ahead;
    int64_t stages;
};

// Either one round after another in the order given, or, where a job's items are few and long (the
// gradients of weights over many tokens, of x over a wide block), those first, one a pair, and
// about as many of the others meanwhile on the other pairs as they take (8,179 tokens, hidden
// 2,360, inter 192, forward and backward 135 -> 113 us; 512 tokens, 4,096 by 2,048, 102 -> 78).  What is
// less than a tenth better by this count is not by the clock (6,000 tokens, 2,048 by 1,024).
Plan plan(const Product *w, int jobs, int kN, int64_t pairs) {
    const int64_t n = count_items(w[0], kN), a = item_stages(w[0], kN), rest = n % pairs;
    Plan best = {0, 0, (n + pairs - 1) / pairs * a};
    if (jobs == 1) return best;
    const int64_t more = count_items(w[1], kN), b = item_stages(w[1], kN), over = more % pairs, rounds = n / pairs * a + more / pairs * b;
    best.stages = rounds + (rest + over > pairs ? a + b : rest > 0 && (over == 0 || a > b) ? a : over > 0 ? b : 0);
    for (int j = 0; j < 2; ++j) {
        const int64_t few = count_items(w[j], kN), many = count_items(w[1 - j], kN);
        const int64_t long_k = item_stages(w[j], kN), short_k = item_stages(w[1 - j], kN), others = pairs - few;
        if (others <= 0 || long_k < 2 * short_k) continue;
        for (int64_t r = long_k / short_k; r <= long_k / short_k + 1; ++r) {
            const int64_t meanwhile = (many < r * others ? (many + others - 1) / others : r) * short_k;
            const int64_t left = many > r * others ? many - r * others : 0;
            const int64_t stages = (long_k > meanwhile ? long_k : meanwhile) + (left + pairs - 1) / pairs * short_k;
            if (stages * 10 < best.stages * 9) best = {j, static_cast<int>(r), stages};
        }
    }
    return best;
}

template <int kN>
moe_status launch(const Product *w, int jobs, bool chained, int *status, uint64_t limit, cudaStream_t stream, int num_sms) {
    using T = Tile<kN>;
    Args p = {};
    p.jobs = jobs;
    p.chained = chained;
    p.status = status;
    p.wait_limit_ns = limit;
    int64_t items = 0;
    const int pairs_most = num_sms / 2;
    const Plan how = plan(w, jobs, kN, pairs_most);
    const Product in_order[kMaxJobs] = {w[how.first], w[jobs - 1 - how.first]};
    w = in_order;
    for (int j = 0; j < jobs; ++j) {
        Job &o = p.job[j];
        const bool gate = w[j].epilogue == kGate;
        o.m = static_cast<int>(w[j].m);
        o.n = static_cast<int>(w[j].n);
        o.k = static_cast<int>(w[j].k);
        o.a_mn = w[j].a.mn;
        o.b_mn = w[j].b.mn;
        o.tile_cols = gate ? kN / 2 : kN;
        o.b_step = gate ? o.n : 0;
        o.tiles_m = (o.m + 2 * kRows - 1) / (2 * kRows);
        o.tiles_n = (o.n + o.tile_cols - 1) / o.tile_cols;
        o.k_stages = (o.k + T::kAtoms * kStageK - 1) / (T::kAtoms * kStageK);
        // Up to 128 rows, the box holds no more of them and the odd CTA copies none: its half of
        // the products, of what is left in its memory, goes nowhere (their boxes would cost what full ones do).
        const bool few = !w[j].a.mn && o.m <= kRows;
        o.a_rows = few ? (o.m + 7) & ~7 : kRows;
        o.odd_a = !few;
        o.first = static_cast<int>(items);
        o.epilogue = w[j].epilogue;
        o.out = w[j].out;
        o.out_f32 = w[j].out_f32;
        o.gu = w[j].gu;
        // Where a last round of items would give less than half of the pairs one, its items are
        // cut in two (4,096 tokens, 256 items on 76 pairs: 123 -> 116 us).
        const int64_t tiles = static_cast<int64_t>(o.tiles_m) * o.tiles_n;
        if (items + 2 * tiles > INT32_MAX / 2) return MOE_ERR_CAPACITY;
        const int64_t rest = (items + tiles) % pairs_most;
        const bool cut = kN == 256 && j == jobs - 1 && how.ahead == 0 && items + tiles > pairs_most && 2 * rest <= pairs_most && rest <= tiles;
        o.full = static_cast<int>(cut ? tiles - rest : tiles);
        items += tiles + (cut ? rest : 0);
        const int64_t n_rows = gate ? 2 * w[j].n : w[j].n;
        const Operand &a = w[j].a, &b = w[j].b;
        if (!(a.mn ? encode(&p.a[j], a.p, w[j].k, w[j].m, a.pitch, kStageK)
                   : encode(&p.a[j], a.p, w[j].m, w[j].k, a.pitch, o.a_rows)) ||
            !(b.mn ? encode(&p.b[j], b.p, w[j].k, n_rows, b.pitch, kStageK)
                   : encode(&p.b[j], b.p, n_rows, w[j].k, b.pitch, T::kBRows)))
            return MOE_ERR_CUDA;
        p.b_half[j] = p.b[j];
        if (o.full < tiles && !b.mn && !encode(&p.b_half[j], b.p, n_rows, w[j].k, b.pitch, T::kBRows / 2))
            return MOE_ERR_CUDA;
    }
    p.items = static_cast<int>(items);
    const int pairs = static_cast<int>(items < pairs_most ? items : pairs_most);
    p.schedule = PairSchedule(pairs, how.ahead > 0 ? p.job[1].first : 0, how.ahead);
    // With few rows of A more stages are on their way (64 tokens 23.4 -> 21.3 us).  The MMAs read
    // 128 rows all the same, what lies behind A among them, whose products nobody reads; the
    // last stage's lie within the ring.
    int a_rows = 0;
    for (int j = 0; j < jobs; ++j) a_rows = p.job[j].a_rows > a_rows ? p.job[j].a_rows : a_rows;
    p.a_bytes = a_rows * 128;              // a multiple of 1,024
    p.stage_bytes = T::kAtoms * (p.a_bytes + T::kBBytes);
    p.stages = (kRingBytes - T::kStageBytes) / p.stage_bytes + 1;
    if (p.stages > kMaxStages) p.stages = kMaxStages;
    static std::atomic<uint64_t> mask{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
    const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
    if (!bit || !(mask.load(std::memory_order_acquire) & bit)) {
        if (cudaFuncSetAttribute(ffn_kernel<kN>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess)
            return MOE_ERR_CUDA;
        mask.fetch_or(bit, std::memory_order_release);
    }
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * pairs);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = chained ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, ffn_kernel<kN>, p) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// The width of items: rounds over the pairs times what a stage takes (about 0.17, 0.23 and
// 0.33 us for 64 k: TMA's rows of A and B, and what a stage costs by itself).  Wide items read A less often, narrow ones leave fewer SMs
// idle.  hidden 4,096, inter 2,048, forward: 64 tokens 41 us with 256 columns and 21 with 64,
// 512 tokens 42 us with 64 and 29 with 128, 1,024 tokens 45 us with 128 and 41 with 256.  B
// along n comes in boxes of 64, the two CTAs' make 128.
moe_status run(const Product *w, int jobs, bool chained, int *status, uint64_t limit, cudaStream_t stream, int num_sms) {
    bool b_mn = false;
    for (int j = 0; j < jobs; ++j) b_mn = b_mn || w[j].b.mn;
    const auto cost = [&](int kN, int stage) { return plan(w, jobs, kN, num_sms / 2).stages * stage; };
    const int64_t c256 = cost(256, 33), c128 = cost(128, 23), c64 = b_mn ? INT64_MAX : cost(64, 17);
    if (c256 <= c128 && c256 <= c64) return launch<256>(w, jobs, chained, status, limit, stream, num_sms);
    if (c128 <= c64) return launch<128>(w, jobs, chained, status, limit, stream, num_sms);
    return launch<64>(w, jobs, chained, status, limit, stream, num_sms);
}

}  // namespace ffn

moe_status launch_ffn_forward(const Ffn &f, cudaStream_t stream, int num_sms, int *launches) {
    *launches = 0;
    if (f.T == 0) return MOE_OK;
    const int64_t T = f.T, H = f.hidden, I = f.inter;
    if (T <= ffn::kFewRows && !f.gu && H <= MOE_MATVEC_MAX_K && I <= MOE_MATVEC_MAX_K) {
        Matvec m = {f.x, f.x_stride, 1, nullptr, f.T, f.hidden, 1, f.inter, f.w13, nullptr, nullptr,
                    Matvec::kBf16, true, f.h, 1, f.status, f.wait_limit_ns, false};
        moe_status st = launch_matvec(m, stream, num_sms);
        if (st != MOE_OK) return st;
        m = {f.h, I, 1, nullptr, f.T, f.inter, 1, f.hidden, f.w2, nullptr, nullptr,
             Matvec::kBf16, false, f.out, f.out_bf16, f.status, f.wait_limit_ns, true};
        *launches = 2;
        return launch_matvec(m, stream, num_sms);
    }
    const ffn::Product up = {{f.x, f.x_stride, false}, {f.w13, H, false}, T, I, H, ffn::kGate, f.h, 0, f.gu};
    moe_status st = ffn::run(&up, 1, false, f.status, f.wait_limit_ns, stream, num_sms);
    if (st != MOE_OK) return st;
    ++*launches;
    const ffn::Product down = {{f.h, I, false}, {f.w2, I, false}, T, H, I, ffn::kStore, f.out, !f.out_bf16, nullptr};
    st = ffn::run(&down, 1, true, f.status, f.wait_limit_ns, stream, num_sms);
    if (st == MOE_OK) ++*launches;
    return st;
}

moe_status launch_ffn_backward(const Ffn &f, const FfnGrad &d, cudaStream_t stream, int num_sms, int *launches) {
    *launches = 0;
    const int64_t T = f.T, H = f.hidden, I = f.inter;
    const size_t size = d.dw_f32 ? 4 : 2;
    if (T == 0) {                      // sums of nothing
        if (d.dw13 && cudaMemsetAsync(d.dw13, 0, 2 * I * H * size, stream) != cudaSuccess) return MOE_ERR_CUDA;
        if (d.dw2 && cudaMemsetAsync(d.dw2, 0, H * I * size, stream) != cudaSuccess) return MOE_ERR_CUDA;
        return MOE_OK;
    }
    ffn::Product w[2];
    int n = 0;
    if (d.dx || d.dw13)
        w[n++] = {{d.dout, H, false}, {f.w2, I, true}, T, I, H, ffn::kGateBack, d.dgu, 0, f.gu};
    if (d.dw2)
        w[n++] = {{d.dout, H, true}, {f.h, I, true}, H, I, T, ffn::kStore, d.dw2, d.dw_f32, nullptr};
    if (n > 0) {
        const moe_status st = ffn::run(w, n, false, f.status, f.wait_limit_ns, stream, num_sms);
        if (st != MOE_OK) return st;
        ++*launches;
    }
    n = 0;
    if (d.dw13)
        w[n++] = {{d.dgu, 2 * I, true}, {f.x, f.x_stride, true}, 2 * I, H, T, ffn::kStore, d.dw13, d.dw_f32, nullptr};
    if (d.dx)
        w[n++] = {{d.dgu, 2 * I, false}, {f.w13, H, true}, T, H, 2 * I, ffn::kStore, d.dx, 0, nullptr};
    if (n > 0) {
        const moe_status st = ffn::run(w, n, true, f.status, f.wait_limit_ns, stream, num_sms);
        if (st != MOE_OK) return st;
        ++*launches;
    }
    return MOE_OK;
}

}  // namespace moe
