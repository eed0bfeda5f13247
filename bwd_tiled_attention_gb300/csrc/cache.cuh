// cache.cuh -- the paged key/value cache as the kernels see it, and the
// geometry of a call over some of its sequences.
//
// Keys and values live in pages of page_size tokens, [layers, pages, heads,
// page_size, d]: the rows of one head in one page are contiguous, so that a
// TMA box is one stretch of memory.  Sequence slot s holds lengths[s] tokens;
// token p is row p % page_size of page table[s][p / page_size].  refs counts
// the sequences that share a page.  A page that is only partly filled is never
// shared: fork copies it, and accept refuses to leave one.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/fa.h"

namespace fa {

// Bits of the cache's device status word (the first word of its scratch).
constexpr int kCacheBadSlot = 1;     // a slot or page index out of range, or a slot named twice
constexpr int kCacheBadLength = 2;   // a length, count or path that does not fit
constexpr int kCacheNoPages = 4;     // not enough free pages
constexpr int kCacheShared = 8;      // the call would write to a shared page
constexpr int kCacheTimeout = 16;    // a bounded wait inside a kernel gave up

// Sequences of a call, or slots of a cache, at most: indexes of loops over them,
// and sums of two, stay within 32 bits.
constexpr int kMostSequences = 1 << 30;

// The sequences of one call: sequence i is cache slot slots[i] and owns tokens
// [cu[i], cu[i + 1]) of the packed batch, or [i * N, (i + 1) * N) of a dense
// one.  Its tokens are the last ones that the slot holds.
struct SeqRange {
    int t0, n;  // first token and count; n < 0: the boundaries are not usable
};

__device__ __forceinline__ SeqRange seq_range(const int* cu, int N, int T, int i) {
    SeqRange r;
    if (cu) {
        r.t0 = cu[i];
        r.n = cu[i + 1] - r.t0;
        if (r.t0 < 0 || r.n < 0 || r.t0 > T - r.n) r.n = -1;
    } else {
        r.t0 = i * N;
        r.n = N;
    }
    return r;
}

// The sequence that owns token t, or -1: the first i with cu[i + 1] > t, if
// cu[i] <= t (empty sequences before it share the boundary).
__device__ __forceinline__ int seq_of_token(const int* cu, int B, int N, int t) {
    if (!cu) return t / N;
    int lo = 0, hi = B;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid + 1] <= t) lo = mid + 1; else hi = mid;
    }
    return lo < B && cu[lo] <= t ? lo : -1;
}

}  // namespace fa
