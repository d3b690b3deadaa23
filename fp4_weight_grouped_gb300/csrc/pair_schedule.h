// Which items of a launch a CTA pair takes, one after another.  Host code as well, so that the
// order can be tested without a GPU.
#pragma once

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

}  // namespace moe
