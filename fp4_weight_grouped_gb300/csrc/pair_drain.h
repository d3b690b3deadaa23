// What a CTA pair's stage barriers still wait for once both CTAs have stopped after a wait
// that gave up.  Host code as well, so that the rule can be tested without a GPU.
//
// The barrier of a stage, in the even CTA, counts one arrival (the even producer's, which
// expects the bytes of both CTAs) and the bytes that either CTA copies.  The producers have
// issued n0 (even) and n1 (odd) stages.  A barrier completes, and all copies on it have
// landed, once what never came has been made up for: the odd CTA's bytes of a stage that only
// the even CTA issued, and of one that only the odd CTA issued the arrival, expecting them.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define MOE_PAIR_FN __host__ __device__ __forceinline__
#else
#define MOE_PAIR_FN inline
#endif

namespace moe {

struct PairFix {
    bool arrive;         // make the even producer's arrival, expecting `expect` bytes
    uint32_t expect;
    uint32_t complete;   // bytes to count as landed
};

// Stage i < max(n0, n1), of which the odd CTA copies odd_bytes.
MOE_PAIR_FN PairFix pair_fix(uint32_t i, uint32_t n0, uint32_t n1, uint32_t odd_bytes) {
    if (i >= n0) return {true, odd_bytes, 0};
    if (i >= n1) return {false, 0, odd_bytes};
    return {false, 0, 0};
}

// First stage that may be incomplete: a producer issues a stage only after the one `stages`
// before it has been consumed.
MOE_PAIR_FN uint32_t pair_first(uint32_t n0, uint32_t n1, uint32_t stages) {
    const uint32_t n = n0 > n1 ? n0 : n1;
    return n > stages ? n - stages : 0;
}

}  // namespace moe
