// cache.cu -- page operations of the paged key/value cache: making room for
// tokens, forking a sequence, accepting a path of drafted tokens, freeing.
//
// All state lives on the device and every call is asynchronous, so a serving
// step with its changing lengths can be captured into a graph.  A call is one
// planning CTA, and a copying kernel where rows move (fork, accept).
//
// Planning is whole-number work on a few kilobytes: what bounds it is latency,
// so one CTA does it with barriers instead of several launches.  It checks
// everything first and then either carries the whole call out or only sets the
// status word.  Free pages (refs == 0) are handed out lowest index first, in
// the order of the call's entries: results do not depend on timing.
//
// Copying is bound by memory, in 16-byte accesses of only the rows that a page
// holds: a CTA a (branch, layer, K or V) in fork, a (sequence, four layers, K or V)
// in accept.
//
// Measured (GPU time of calls among queued ones): freeing and forking 64 branches of
// 8 sequences of 400-2000 tokens, 8 layers, 8 heads of 128, 28 us, of which the copy
// is 21 us for 155 MB (reads of a parent's page meet in L2).  Dropping, reserving and
// accepting drafts of 64 in 64 sequences over 32 layers, four launches, 28.5 us: each
// planning CTA is a chain of four or five trips to memory.
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "../../include/fa.h"
#include "cache.cuh"
#include "common.cuh"
#include "internal.h"

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

// Sum over the CTA's threads before this one, and the total.
__device__ __forceinline__ long long block_scan(long long x, long long* sums, long long& total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto warp_scan = [&](long long v) {
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += y;
        }
        return v;
    };
    const long long incl = warp_scan(x);
    __syncthreads();  // (the last call's sums have been read)
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        const long long all = warp_scan(sums[lane]);
        sums[lane] = all - sums[lane];
        if (lane == 31) sums[32] = all;
    }
    __syncthreads();
    total = sums[32];
    return sums[warp] + incl - x;
}

// entry[i].z = first place in `taken` of entry i, for needs entry[i].x; returns
// the number of pages wanted in all.
__device__ __forceinline__ long long place_needs(int4* entry, int n, long long* sums) {
    long long all = 0;
    for (int i0 = 0; i0 < n; i0 += kPlan) {
        const int i = i0 + threadIdx.x;
        long long total;
        const long long at = all + block_scan(i < n ? entry[i].x : 0, sums, total);
        if (i < n) entry[i].z = (int)min(at, 0x7FFFFFFFLL);
        all += total;
    }
    __syncthreads();
    return all;
}

// Free pages, four to a thread from page p0 on: a mask.  The first stretch is
// looked up before the call knows how many it wants.
__device__ __forceinline__ int free_pages(const fa_cache& c, long long p0) {
    const long long p = p0 + threadIdx.x * 4;
    int mask = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (p + e < c.pages && c.refs[p + e] == 0) mask |= 1 << e;
    return mask;
}

// The `want` lowest free pages into taken[]; false when there are fewer.
__device__ __forceinline__ bool take_pages(const fa_cache& c, int* taken, long long want, int mask,
                                           long long* sums) {
    long long have = 0;
    for (long long p0 = 0; p0 < c.pages && have < want; p0 += kPlan * 4) {
        if (p0 > 0) mask = free_pages(c, p0);
        long long total, at = have + block_scan(__popc(mask), sums, total);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if ((mask >> e) & 1) {
                if (at < want) taken[at] = (int)(p0 + threadIdx.x * 4 + e);
                ++at;
            }
        have += total;
    }
    __syncthreads();
    return have >= want;
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

// Lists of up to kPlan entries and kFew pages stay in shared memory.
constexpr int kFew = 2048;
struct PlanSmem {
    long long sums[kPlan / 32 + 1];
    int4 entry[kPlan];
    int taken[kFew];
    int error;
};

__global__ void __launch_bounds__(kPlan) reserve_kernel(const fa_cache c, const int* slots,
                                                        const int* counts, int count, int n) {
    pdl_begin();
    __shared__ PlanSmem sm;
    const Scratch s = scratch_of(c);
    int4* entry = n <= kPlan ? sm.entry : s.entry;
    if (threadIdx.x == 0) sm.error = 0;
    const int free_mask = free_pages(c, 0);
    for (int i = threadIdx.x; i < n; i += kPlan)
        if (slot_ok(c, slots[i])) s.mark[slots[i]] = -1;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPlan) {
        const int slot = slots[i], m = counts ? counts[i] : count;
        int4 e = make_int4(0, 0, 0, slot);  // pages wanted, pages held, place in the list, slot
        int bad = 0;
        if (!slot_ok(c, slot)) bad = kCacheBadSlot;
        else {
            const int len = length_of(c, slot);
            if (atomicCAS(&s.mark[slot], -1, i) != -1) bad = kCacheBadSlot;
            else if (len < 0 || m < 0 || (long long)len + m > (long long)c.max_pages * c.page_size)
                bad = kCacheBadLength;
            else {
                e.y = (len + c.page_size - 1) / c.page_size;
                e.x = (int)(((long long)len + m + c.page_size - 1) / c.page_size) - e.y;
                if (m > 0 && len % c.page_size) {  // tokens will go to the last page
                    const int page = c.table[(long long)slot * c.max_pages + e.y - 1];
                    if (page < 0 || page >= c.pages) bad = kCacheBadSlot;
                    else if (c.refs[page] != 1) bad = kCacheShared;
                }
            }
        }
        if (bad) atomicOr(&sm.error, bad);
        entry[i] = e;
    }
    __syncthreads();
    const long long want = place_needs(entry, n, sm.sums);
    int* taken = want <= kFew ? sm.taken : s.taken;
    if (!sm.error && want > 0 && !(want <= c.pages && take_pages(c, taken, want, free_mask, sm.sums)))
        if (threadIdx.x == 0) atomicOr(&sm.error, kCacheNoPages);
    __syncthreads();
    if (sm.error) {
        if (threadIdx.x == 0) atomicOr(s.status, sm.error);
        return;
    }
    for (int r = threadIdx.x; r < want; r += kPlan) {
        int lo = 0, hi = n - 1;  // the last entry whose place is <= r
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (entry[mid].z <= r) lo = mid; else hi = mid - 1;
        }
        const int4 e = entry[lo];
        const int page = taken[r];
        c.table[(long long)e.w * c.max_pages + e.y + (r - e.z)] = page;
        c.refs[page] = 1;
    }
    for (int i = threadIdx.x; i < n; i += kPlan) c.lengths[entry[i].w] += counts ? counts[i] : count;
}

__global__ void __launch_bounds__(kPlan) fork_plan_kernel(const fa_cache c, const int* parents,
                                                          const int* children, int n) {
    pdl_begin();
    __shared__ PlanSmem sm;
    const Scratch s = scratch_of(c);
    const Groups grp(n);
    int4* entry = n <= kPlan ? sm.entry : s.entry;
    if (threadIdx.x == 0) sm.error = 0;
    const int free_mask = free_pages(c, 0);
    for (int i = threadIdx.x; i < n; i += kPlan) {
        const int from = parents[i], to = children[i];
        if (slot_ok(c, to)) s.mark[to] = -1;
        if (slot_ok(c, from)) s.mark[from] = -1;
    }
    __syncthreads();
    for (int i = grp.entry; i < n; i += grp.stride) {
        const int from = parents[i], to = children[i];
        int4 e = make_int4(0, 0, 0, 0);  // pages wanted (0 or 1), whole pages, place, rows copied
        int bad = 0;
        if (!slot_ok(c, from) || !slot_ok(c, to)) bad = kCacheBadSlot;
        else {
            const int* row = c.table + (long long)from * c.max_pages;
            const int page0 = grp.sub < c.max_pages ? row[grp.sub] : -1;  // (in the lengths' trip)
            const int len = length_of(c, from), old = c.lengths[to];
            if (grp.sub == 0 && atomicCAS(&s.mark[to], -1, i) != -1) bad = kCacheBadSlot;
            if (len < 0 || old != 0) bad |= kCacheBadLength;
            else {
                e.y = len / c.page_size;
                e.w = len % c.page_size;
                e.x = e.w > 0;
                for (int k = grp.sub; k < e.y + e.x; k += grp.g) {
                    const int p = k == grp.sub ? page0 : row[k];
                    if (p < 0 || p >= c.pages) bad |= kCacheBadSlot;
                }
            }
        }
        if (bad) atomicOr(&sm.error, bad);
        if (grp.sub == 0) entry[i] = e;
    }
    __syncthreads();
    // a slot cannot be read and made in one call
    for (int i = threadIdx.x; i < n; i += kPlan) {
        const int from = parents[i];
        if (slot_ok(c, from) && s.mark[from] != -1) atomicOr(&sm.error, kCacheBadSlot);
    }
    const long long want = place_needs(entry, n, sm.sums);  // (begins and ends with a barrier)
    int* taken = want <= kFew ? sm.taken : s.taken;
    if (!sm.error && want > 0 && !(want <= c.pages && take_pages(c, taken, want, free_mask, sm.sums)))
        if (threadIdx.x == 0) atomicOr(&sm.error, kCacheNoPages);
    __syncthreads();
    if (threadIdx.x == 0) {
        *s.go = sm.error == 0;
        if (sm.error) atomicOr(s.status, sm.error);
    }
    if (sm.error) return;
    for (int i = grp.entry; i < n; i += grp.stride) {
        const int4 e = entry[i];
        __syncwarp(grp.mask);  // (all have read it: past kPlan entries the record below lies there)
        const int from_slot = parents[i], to_slot = children[i];
        const int* from = c.table + (long long)from_slot * c.max_pages;
        int* to = c.table + (long long)to_slot * c.max_pages;
        for (int k = grp.sub; k < e.y; k += grp.g) {
            const int p = from[k];
            to[k] = p;
            atomicAdd(&c.refs[p], 1);
        }
        if (grp.sub == 0) {
            int src = 0, dst = 0;
            if (e.x) {
                src = from[e.y];
                dst = taken[e.z];
                to[e.y] = dst;
                c.refs[dst] = 1;
            }
            c.lengths[to_slot] = e.y * c.page_size + e.w;
            s.entry[i] = make_int4(src, dst, e.w, 0);  // for the copying kernel
        }
    }
}

// Copies the first rows of a page to another page: entry (source page,
// destination page, rows).
__global__ void __launch_bounds__(256, 4) fork_copy_kernel(const fa_cache c) {
    pdl_begin();
    const Scratch s = scratch_of(c);
    if (!*s.go) return;
    const int4 e = s.entry[blockIdx.x];
    if (e.z == 0) return;
    const int layer = blockIdx.y >> 1;
    uint4* base = static_cast<uint4*>(blockIdx.y & 1 ? c.v : c.k);
    const int row16 = c.d / 8;                       // 16-byte units of a row
    const int head16 = c.page_size * row16, run = e.z * row16;
    const uint4* src = base + ((long long)layer * c.pages + e.x) * c.heads * head16;
    uint4* dst = base + ((long long)layer * c.pages + e.y) * c.heads * head16;
    // (heads in fours, so that no index has to be divided: the copy is close to
    // bound by instructions otherwise)
    for (int h = 0; h < c.heads; h += 4) {
        const uint4* from = src + (long long)h * head16;
        uint4* to = dst + (long long)h * head16;
        const int heads = min(4, c.heads - h);
        for (int i = threadIdx.x; i < run; i += 256) {
            uint4 x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (u < heads) x[u] = from[u * head16 + i];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (u < heads) __stcs(&to[u * head16 + i], x[u]);  // (parents are read again)
        }
    }
}

__global__ void __launch_bounds__(kPlan) free_kernel(const fa_cache c, const int* slots, int n) {
    pdl_begin();
    __shared__ int error;
    const Scratch s = scratch_of(c);
    const Groups grp(n);
    if (threadIdx.x == 0) error = 0;
    __syncthreads();
    for (int i = grp.entry; i < n; i += grp.stride) {
        const int slot = slots[i];
        int bad = 0;
        if (!slot_ok(c, slot)) bad = kCacheBadSlot;
        else {
            const int* row = c.table + (long long)slot * c.max_pages;
            const int page0 = grp.sub < c.max_pages ? row[grp.sub] : -1;  // (in the length's trip)
            const int len = length_of(c, slot);
            if (len < 0) bad = kCacheBadLength;
            else {
                const int used = (len + c.page_size - 1) / c.page_size;
                for (int k = grp.sub; k < used; k += grp.g) {
                    const int p = k == grp.sub ? page0 : row[k];
                    if (p < 0 || p >= c.pages) bad = kCacheBadSlot;
                }
            }
        }
        if (bad) atomicOr(&error, bad);
    }
    __syncthreads();
    if (error) {
        if (threadIdx.x == 0) atomicOr(s.status, error);
        return;
    }
    for (int i = grp.entry; i < n; i += grp.stride) {
        const int slot = slots[i];
        int len = 0;
        // whoever takes the length frees the pages: a slot named twice is freed once
        if (grp.sub == 0) len = atomicExch(&c.lengths[slot], 0);
        len = grp.first(len);
        const int used = (len + c.page_size - 1) / c.page_size;
        for (int k = grp.sub; k < used; k += grp.g) {
            int* at = c.table + (long long)slot * c.max_pages + k;
            atomicSub(&c.refs[*at], 1);
            *at = -1;
        }
    }
}

__global__ void __launch_bounds__(kPlan) accept_plan_kernel(const fa_cache c, const int* slots,
                                                            const int* base, const int* path,
                                                            int width, const int* accepted, int n) {
    pdl_begin();
    __shared__ int error;
    const Scratch s = scratch_of(c);
    const Groups grp(n);
    if (threadIdx.x == 0) error = 0;
    for (int i = threadIdx.x; i < n; i += kPlan) {
        const int slot = slots[i];
        if (slot_ok(c, slot)) s.mark[slot] = -1;
    }
    __syncthreads();
    for (int i = grp.entry; i < n; i += grp.stride) {
        const int slot = slots[i], b = base[i], m = accepted[i];
        const int* at = path + (long long)i * width;
        int bad = 0;
        if (!slot_ok(c, slot)) bad = kCacheBadSlot;
        else {
            // what the checks look at first comes in one trip with the length: this
            // lane's entry of the path and its page, wherever the length ends
            const int* row = c.table + (long long)slot * c.max_pages;
            const int k0 = b / c.page_size + grp.sub;
            const int page0 = b >= 0 && k0 < c.max_pages ? row[k0] : -1;
            int step0 = 0, prev0 = -1;
            if (grp.sub < m && grp.sub < width) {
                step0 = at[grp.sub];
                if (grp.sub > 0) prev0 = at[grp.sub - 1];
            }
            const int len = length_of(c, slot);
            const bool again = grp.sub == 0 && atomicCAS(&s.mark[slot], -1, i) != -1;
            if (grp.any(again)) bad = kCacheBadSlot;
            else if (len < 0 || b < 0 || b > len || m < 0 || m > width || m > len - b) bad = kCacheBadLength;
            else {
                const int used = (len + c.page_size - 1) / c.page_size;
                const int kept = (b + m + c.page_size - 1) / c.page_size;
                for (int j = grp.sub; j < m; j += grp.g) {  // strictly ascending, within the draft
                    const int t = j == grp.sub ? step0 : at[j];
                    const int before = j == grp.sub ? prev0 : at[j - 1];  // (-1 before the first)
                    if (t < 0 || t >= len - b || before >= t) bad |= kCacheBadLength;
                }
                for (int k = k0; k < used; k += grp.g) {
                    const int p = k == k0 ? page0 : row[k];
                    if (p < 0 || p >= c.pages) bad |= kCacheBadSlot;
                    else if (k < kept && c.refs[p] != 1) bad |= kCacheShared;
                    s.shadow[(long long)slot * c.max_pages + k] = p;
                }
            }
        }
        if (bad) atomicOr(&error, bad);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        *s.go = error == 0;
        if (error) atomicOr(s.status, error);
    }
    if (error) return;
    for (int i = grp.entry; i < n; i += grp.stride) {
        const int slot = slots[i], now = base[i] + accepted[i], len = c.lengths[slot];
        __syncwarp(grp.mask);  // (all have read the length)
        const int used = (len + c.page_size - 1) / c.page_size;
        for (int k = (now + c.page_size - 1) / c.page_size + grp.sub; k < used; k += grp.g) {
            const long long at = (long long)slot * c.max_pages + k;
            atomicSub(&c.refs[c.table[at]], 1);
            c.table[at] = -1;
        }
        if (grp.sub == 0) c.lengths[slot] = now;
    }
}

// Moves token base + path[j] to base + j, for every head of one layer's K or
// V.  path ascends strictly, so path[j] >= j: a thread owns its 16 bytes of a
// row and walks j upward in runs, reading a run's rows before it writes them;
// what it has written lies below every row still to be read.
// The rows' places are the same in all layers: a CTA takes kMoveLayers of them.
constexpr int kRun = 8, kMoveLayers = 4, kMoveThreads = 128;
__global__ void __launch_bounds__(kMoveThreads) accept_move_kernel(const fa_cache c, const int* slots,
                                                                   const int* base, const int* path,
                                                                   int width, const int* accepted) {
    pdl_begin();
    const Scratch s = scratch_of(c);
    const int i = blockIdx.x;
    if (!*s.go) return;
    const int m = accepted[i], b = base[i];
    const int* pages = s.shadow + (long long)slots[i] * c.max_pages;
    const int* at = path + (long long)i * width;
    const int first = (blockIdx.y >> 1) * kMoveLayers, last = min(first + kMoveLayers, c.layers);
    uint4* data = static_cast<uint4*>(blockIdx.y & 1 ? c.v : c.k);
    const int row16 = c.d / 8;                                     // 16-byte units of a row
    const unsigned plane = (unsigned)c.page_size * row16;          // of a head in a page
    const long long layer_units = (long long)c.pages * c.heads * plane;
    for (int x = threadIdx.x; x < c.heads * row16; x += kMoveThreads) {
        const int head = x / row16, col = x - head * row16;
        auto place = [&](int tok) {
            return ((long long)pages[tok / c.page_size] * c.heads + head) * plane +
                   (unsigned)(tok % c.page_size) * row16 + col;
        };
        for (int j0 = 0; j0 < m; j0 += kRun) {
            long long from[kRun], to[kRun];                        // from < 0: stays
#pragma unroll
            for (int u = 0; u < kRun; ++u) {
                const int j = j0 + u, t = j < m ? at[j] : j;
                from[u] = -1;
                if (t != j) {
                    from[u] = place(b + t);
                    to[u] = place(b + j);
                }
            }
            for (int layer = first; layer < last; ++layer) {
                uint4* rows = data + layer * layer_units;
                uint4 v[kRun];
#pragma unroll
                for (int u = 0; u < kRun; ++u)
                    if (from[u] >= 0) v[u] = __ldcs(&rows[from[u]]);  // (read for the last time)
#pragma unroll
                for (int u = 0; u < kRun; ++u)
                    if (from[u] >= 0) __stcs(&rows[to[u]], v[u]);
            }
        }
    }
}

// Takes the bits that have been read out of the status word, and no others: calls
// on other streams may have set some since.
__global__ void clear_kernel(int* status, int bits) {
    pdl_begin();
    atomicAnd(status, ~bits);
}

bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
fa_status launched(cudaError_t e) { return e == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

// A list of device integers.
bool list_ok(const int* p) { return p && aligned(p, 4); }

}  // namespace

fa_status check_cache(const fa_cache* c) {
    if (!c || !c->k || !c->v || !c->table || !c->lengths || !c->refs || !c->scratch)
        return FA_ERR_INVALID_ARG;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->table, 4) || !aligned(c->lengths, 4) ||
        !aligned(c->refs, 4) || !aligned(c->scratch, 16))
        return FA_ERR_INVALID_ARG;
    if (c->layers <= 0 || c->pages <= 0 || c->heads <= 0 || c->slots <= 0 || c->max_pages <= 0)
        return FA_ERR_INVALID_ARG;
    if (c->d != 64 && c->d != 96 && c->d != 128 && c->d != 192 && c->d != 256)
        return FA_ERR_UNSUPPORTED;
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
        return FA_ERR_UNSUPPORTED;
    if (c->heads > 65535 || c->layers > 32767 || c->slots > kMostSequences ||
        (long long)c->layers * c->pages > 0x7FFFFFFFLL / c->heads ||
        (long long)c->max_pages * c->page_size > 0x40000000LL)
        return FA_ERR_UNSUPPORTED;
    return FA_OK;
}

}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_cache_scratch_size(int pages, int slots, int max_pages) {
    if (pages <= 0 || slots <= 0 || max_pages <= 0) return 0;
    return (size_t)scratch_ints(pages, slots, max_pages) * sizeof(int);
}

fa_status fa_cache_reserve(const fa_cache* cache, const int* slots, const int* counts, int count,
                           int n, fa_stream_t stream) {
    const fa_status st = check_cache(cache);
    if (st != FA_OK) return st;
    if (n < 0 || n > cache->slots || (!counts && count < 0)) return FA_ERR_INVALID_ARG;
    if (n == 0) return FA_OK;
    if (!list_ok(slots) || !aligned(counts, 4)) return FA_ERR_INVALID_ARG;
    return launched(launch_pdl(reserve_kernel, dim3(1), dim3(kPlan), 0,
                               reinterpret_cast<cudaStream_t>(stream), *cache, slots, counts, count, n));
}

fa_status fa_cache_fork(const fa_cache* cache, const int* parents, const int* children, int n,
                        fa_stream_t stream) {
    const fa_status st = check_cache(cache);
    if (st != FA_OK) return st;
    if (n < 0 || n > cache->slots) return FA_ERR_INVALID_ARG;
    if (n == 0) return FA_OK;
    if (!list_ok(parents) || !list_ok(children)) return FA_ERR_INVALID_ARG;
    cudaStream_t strm = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = launch_pdl(fork_plan_kernel, dim3(1), dim3(kPlan), 0, strm, *cache, parents,
                                     children, n);
    if (e != cudaSuccess) return FA_ERR_CUDA;
    return launched(launch_pdl(fork_copy_kernel, dim3(n, cache->layers * 2), dim3(256), 0, strm, *cache));
}

fa_status fa_cache_free(const fa_cache* cache, const int* slots, int n, fa_stream_t stream) {
    const fa_status st = check_cache(cache);
    if (st != FA_OK) return st;
    if (n < 0) return FA_ERR_INVALID_ARG;
    if (n > kMostSequences) return FA_ERR_UNSUPPORTED;
    if (n == 0) return FA_OK;
    if (!list_ok(slots)) return FA_ERR_INVALID_ARG;
    return launched(launch_pdl(free_kernel, dim3(1), dim3(kPlan), 0,
                               reinterpret_cast<cudaStream_t>(stream), *cache, slots, n));
}

fa_status fa_cache_accept(const fa_cache* cache, const int* slots, const int* base, const int* path,
                          int path_width, const int* accepted, int n, fa_stream_t stream) {
    const fa_status st = check_cache(cache);
    if (st != FA_OK) return st;
    if (n < 0 || n > cache->slots || path_width < 0) return FA_ERR_INVALID_ARG;
    if (n == 0) return FA_OK;
    if (!list_ok(slots) || !list_ok(base) || !list_ok(accepted) || (path_width > 0 && !list_ok(path)))
        return FA_ERR_INVALID_ARG;
    cudaStream_t strm = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = launch_pdl(accept_plan_kernel, dim3(1), dim3(kPlan), 0, strm, *cache, slots,
                                     base, path, path_width, accepted, n);
    if (e != cudaSuccess) return FA_ERR_CUDA;
    if (path_width == 0) return FA_OK;
    return launched(launch_pdl(accept_move_kernel, dim3(n, cdiv(cache->layers, kMoveLayers) * 2),
                               dim3(kMoveThreads), 0, strm,
                               *cache, slots, base, path, path_width, accepted));
}

fa_status fa_cache_check(const fa_cache* cache, int* bits, fa_stream_t stream) {
    const fa_status st = check_cache(cache);
    if (st != FA_OK) return st;
    cudaStream_t strm = reinterpret_cast<cudaStream_t>(stream);
    int word = 0;
    if (cudaMemcpyAsync(&word, cache->scratch, sizeof(int), cudaMemcpyDeviceToHost, strm) != cudaSuccess ||
        cudaStreamSynchronize(strm) != cudaSuccess)
        return FA_ERR_CUDA;
    if (word && (launch_pdl(clear_kernel, dim3(1), dim3(1), 0, strm, cache->scratch, word) != cudaSuccess ||
                 cudaStreamSynchronize(strm) != cudaSuccess))
        return FA_ERR_CUDA;
    if (bits) *bits = word;
    if (word & kCacheTimeout) return FA_ERR_TIMEOUT;
    return word ? FA_ERR_INVALID_ARG : FA_OK;
}

}  // extern "C"
