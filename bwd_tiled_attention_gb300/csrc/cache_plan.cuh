// cache_plan.cuh -- what the planning CTAs of the page operations and of eviction share:
// the scratch words, sums over a CTA, and how its threads go round a call's entries.
#pragma once
#include <cuda_runtime.h>

#include "cache.cuh"

namespace fa {
namespace {

constexpr int kPlan = 1024;  // threads of the planning CTA

// Scratch words: [0] status, [1] go flag of the running call, then per slot an
// entry (4 words) and a mark, the list of pages taken, and a copy of the table
// entries behind an accepted base.
struct Scratch {
    int* status;
    int* go;
    int4* entry;
    int* mark;
    int* taken;
    int* shadow;
};
inline long long scratch_ints(long long pages, long long slots, long long max_pages) {
    return 8 + 4 * slots + slots + pages + slots * max_pages;
}
__device__ __forceinline__ Scratch scratch_of(const fa_cache& c) {
    Scratch s;
    s.status = c.scratch;
    s.go = c.scratch + 1;
    s.entry = reinterpret_cast<int4*>(c.scratch + 8);
    s.mark = c.scratch + 8 + 4 * (long long)c.slots;
    s.taken = s.mark + c.slots;
    s.shadow = s.taken + c.pages;
    return s;
}

__device__ __forceinline__ bool slot_ok(const fa_cache& c, int slot) { return slot >= 0 && slot < c.slots; }

// A slot's length, or -1 when it is not one.
__device__ __forceinline__ int length_of(const fa_cache& c, int slot) {
    const int n = c.lengths[slot];
    return n < 0 || n > (long long)c.max_pages * c.page_size ? -1 : n;
}

// The planning CTA's threads by entry: groups of g lanes, as many as put all
// entries to work at once (32 lanes for up to 32 entries, 4 for 256 and more).
struct Groups {
    int g, sub, entry, stride;
    unsigned mask;
    __device__ __forceinline__ explicit Groups(int n) {
        g = 32;
        while (g > 4 && n * g > kPlan) g >>= 1;
        sub = threadIdx.x & (g - 1);
        entry = threadIdx.x / g;
        stride = kPlan / g;
        mask = g == 32 ? 0xffffffffu : ((1u << g) - 1u) << (threadIdx.x & 31 & ~(g - 1));
    }
    __device__ __forceinline__ bool any(bool x) const { return __ballot_sync(mask, x) != 0; }
    __device__ __forceinline__ int first(int x) const { return __shfl_sync(mask, x, 0, g); }
};

}  // namespace
}  // namespace fa
