// What the barriers of a ring's stages still wait for besides their copies once every warp
// of the CTA has stopped after an abort.  Host code as well, so that the count can be tested
// without a GPU.
//
// Stages are numbered through a CTA's items: stage ks of its n-th item is n k_stages + ks,
// and belongs to converter set ks & 1.  A barrier counts the producer (which has arrived at
// every stage that it issued), the four warps of the stage's set and, in the even CTA of a
// pair, the odd CTA's relay.  Each of these goes through its stages in order and has arrived
// at every one before the stage where it stopped, of which its ring position is known: the
// number modulo twice the ring's n stages.
//
// Of stages all of whose predecessors are complete the first that is not, `from`, makes the
// number whole: nobody has stopped before it, and nobody is more than n + 2 stages past it
// (a warp arrives at a stage after the MMAs of the stage n before, and its next one is at
// most three on).  n + 3 <= 2 n from n = 3 on.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define MOE_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define MOE_HOST_DEVICE inline
#endif

namespace moe {

constexpr int kStopWarps = 8;        // converter warps, four a set
constexpr uint32_t kMinDrainStages = 3;

// Stage where somebody at ring position `at` stopped.
MOE_HOST_DEVICE uint32_t stopped_at(uint32_t at, uint32_t from, uint32_t n) {
    return from + (at + 2 * n - from % (2 * n)) % (2 * n);
}

// Arrivals that `stage` (>= from) still waits for; relay: its position, or null.
MOE_HOST_DEVICE uint32_t missing_arrivals(uint32_t stage, uint32_t from, uint32_t n, uint32_t k_stages,
                                          const uint32_t *stops, const uint32_t *relay) {
    const uint32_t *set = stops + 4 * (stage % k_stages & 1u);
    uint32_t missing = relay && stage >= stopped_at(*relay, from, n) ? 1u : 0u;
    for (int w = 0; w < 4; ++w) missing += stage >= stopped_at(set[w], from, n) ? 1u : 0u;
    return missing;
}

}  // namespace moe
