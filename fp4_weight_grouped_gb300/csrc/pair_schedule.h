// Which items of a launch a CTA pair takes, one after another, and how long an epilogue waits for
// one.  Host code as well, so that both can be tested without a GPU.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define MOE_SCHEDULE_FN __host__ __device__ __forceinline__
#else
#define MOE_SCHEDULE_FN inline
#endif

namespace moe {

// Pair p starts with item p and goes on by the number of pairs; but where the first job's items
// are few and long (long_items of them, fewer than pairs, one a pair), the other pairs take
// `ahead` rounds of the rest first, up to item `from`.  A pair's items ascend; it stops at the
// first one past the last.
struct PairSchedule {
    int pairs, long_items, from;
    MOE_SCHEDULE_FN PairSchedule() : pairs(1), long_items(0), from(0) {}
    MOE_SCHEDULE_FN PairSchedule(int n, int few, int ahead) : pairs(n), long_items(few), from(few + ahead * (n - few)) {}
    MOE_SCHEDULE_FN int next(int pair, int item) const {
        if (item >= from) return item + pairs;
        const int after = item + pairs - long_items;
        return item < long_items || after >= from ? from + pair : after;
    }
};

// Nanoseconds after which the wait for an item's accumulator gives up: the feeding threads wait for
// one stage at a time, this for all of them.  2 us a stage; it takes 0.17 to 0.33.
MOE_SCHEDULE_FN uint64_t accumulator_limit(uint64_t limit_ns, int k_stages) {
    return limit_ns + 2000ull * static_cast<uint64_t>(k_stages);
}

}  // namespace moe
