// evict.cu -- cutting sequences of the paged cache down to a budget: the first tokens and
// the last ones stay, and of those between the ones whose keys have received the most
// attention, in every layer and head on its own.
//
// With S sinks, R recent tokens and a budget of `keep`, a head's kept rows come to stand
// as [sinks | heavy | recent].  Rows are not pushed together: a heavy one before
// keep - R stays where it is, and only those beyond fill the holes that dropped ones
// leave, in ascending order both.  So a step that drops E of `keep` + E tokens moves R rows and
// at most E others instead of nearly all (2048 of 2304 tokens, R = 512: 0.7 of 1.8 thousand
// rows).
//
// Bound: memory, the moved rows (read and written once) and one read of the weights; with
// few heads in all the latency of a CTA's chain: search, two sums over the CTA, moves.
//
// A planning CTA checks the call, copies the page lists of its slots (the moves need
// them), and does the bookkeeping; then a CTA a (sequence, layer, head):
//   - weights become 32-bit keys in their order, in shared memory where they fit;
//   - the lowest kept key is found by a search over its bits, two at a time, by counting
//     keys; those that share its first bits are listed once they are few.  (Counting needs
//     no histogram: most weights share their exponent, so that most of a radix digit's
//     atomics would meet in a few words.)
//   - a second and third look count ties, holes and rows to move along each thread's
//     stretch; ranks from sums over the CTA pair the r-th hole with the r-th such row;
//   - 16-byte pieces of K and V move, then the recent rows close up from below, in runs
//     that are read before they are written.
//
// Measured (GPU time, the call alone): 16 sequences of 2.1-2.3k tokens back to 2048, R = 512, 16
// layers, 8 heads of 128: 253 us for 1.41 GB, 82% of a copy; 4 prompts of 8-16k down to 1024:
// 138 us for 0.60 GB (512 CTAs of one long chain: ~22 us of search and lists, ~27 of moves, in
// two uneven waves).  One sequence, one layer, 8 heads: 34 us.  Those are tables as wide as what they
// hold; shared memory and threads go by the table's width, and tables of 32k places take 389 and
// 199 us, of 8192 the first 314.
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "../../include/fa.h"
#include "cache.cuh"
#include "cache_plan.cuh"
#include "common.cuh"
#include "internal.h"

#ifndef FA_DYNAMIC_SHARED
#define FA_DYNAMIC_SHARED(type, name) extern __shared__ type name[]
#endif

namespace fa {
namespace {

constexpr int kMostKeys = 32768;  // keys in shared memory
constexpr int kPairs = 2048;      // moves listed at once
constexpr int kRun = 8;           // 16-byte pieces in flight a thread

__global__ void __launch_bounds__(kPlan) evict_plan_kernel(const fa_cache c, const int* slots,
                                                           const int* keep, int keep_all, int recent,
                                                           int sinks, int n) {
    pdl_begin();
    __shared__ int error;
    const Scratch s = scratch_of(c);
    const Groups grp(n);
    if (threadIdx.x == 0) error = 0;
    for (int i = threadIdx.x; i < n; i += kPlan)
        if (slot_ok(c, slots[i])) s.mark[slots[i]] = -1;
    __syncthreads();
    for (int i = grp.entry; i < n; i += grp.stride) {
        const int slot = slots[i], now = keep ? keep[i] : keep_all;
        int bad = 0;
        if (!slot_ok(c, slot)) bad = kCacheBadSlot;
        else {
            const int* row = c.table + (long long)slot * c.max_pages;
            const int page0 = grp.sub < c.max_pages ? row[grp.sub] : -1;  // (in the length's trip)
            const int len = length_of(c, slot);
            const bool again = grp.sub == 0 && atomicCAS(&s.mark[slot], -1, i) != -1;
            if (grp.any(again)) bad = kCacheBadSlot;
            else if (len < 0 || (long long)now < (long long)recent + sinks) bad = kCacheBadLength;
            else if (len > now) {
                const int used = (len + c.page_size - 1) / c.page_size;
                const int kept = (now + c.page_size - 1) / c.page_size;
                for (int k = grp.sub; k < used; k += grp.g) {
                    const int p = k == grp.sub ? page0 : row[k];
                    if (p < 0 || p >= c.pages) bad |= kCacheBadSlot;
                    else if (k >= sinks / c.page_size && k < kept && c.refs[p] != 1) bad |= kCacheShared;
                    s.shadow[(long long)slot * c.max_pages + k] = p;
                }
            }
            if (grp.sub == 0) s.entry[i] = make_int4(slot, len, now, 0);  // for the CTAs that move
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
        const int4 e = s.entry[i];
        if (e.y <= e.z) continue;
        const int used = (e.y + c.page_size - 1) / c.page_size;
        for (int k = (e.z + c.page_size - 1) / c.page_size + grp.sub; k < used; k += grp.g) {
            const long long at = (long long)e.x * c.max_pages + k;
            atomicSub(&c.refs[c.table[at]], 1);
            c.table[at] = -1;
        }
        if (grp.sub == 0) c.lengths[e.x] = e.z;
    }
}

// Weights in their order as whole numbers: NaN above all, -0 as 0.
__device__ __forceinline__ unsigned key_of(float w) {
    if (w != w) return 0xffffffffu;
    unsigned u;
    w += 0.f;
    memcpy(&u, &w, 4);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct EvictSmem {
    int counts[16][3], listed;
    long long sums[16];
    int hole[2 * kPairs];   // and where they are filled from: hole[kPairs + i]
};

// Sum over the CTA's threads before this one, and the total.
template <int kEvict>
__device__ __forceinline__ long long cta_scan(long long x, long long* sums, long long& total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    long long incl = x;
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    __syncthreads();  // (the last call's sums have been read)
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    long long before = 0;
    total = 0;
    for (int w = 0; w < kEvict / 32; ++w) {
        if (w < warp) before += sums[w];
        total += sums[w];
    }
    return before + incl - x;
}

// kEvict: threads.
template <int kEvict>
__global__ void __launch_bounds__(kEvict, 1024 / kEvict) evict_kernel(const fa_cache c, float* weights, int recent,
                                                          int sinks, int room_keys) {
    pdl_begin();
    FA_DYNAMIC_SHARED(unsigned, keys);
    __shared__ EvictSmem sm;
    const Scratch s = scratch_of(c);
    if (!*s.go) return;
    const int unit = blockIdx.x, planes = c.layers * c.heads;
    const int i = unit / planes, layer = unit % planes / c.heads, head = unit % c.heads;
    const int4 e = s.entry[i];
    const int slot = e.x, len = e.y, keep = e.z, tid = threadIdx.x;
    if (len <= keep) return;
    const int gap = keep - recent, last = len - recent;  // the recent ones: [last, len) -> [gap, keep)
    const int top = gap - sinks, many = last - sinks;    // kept of so many
    const long long room = (long long)c.max_pages * c.page_size;
    float* w = weights + (((long long)layer * c.slots + slot) * c.heads + head) * room;
    const bool cached = many <= room_keys;
    auto key = [&](int j) { return cached ? keys[j] : key_of(w[sinks + j]); };

    // ---- rows: a thread has one 16-byte piece of them, of K or of V, and takes every
    // `rows`-th row, kRun in flight
    const int* pages = s.shadow + (long long)slot * c.max_pages;
    const int row16 = c.d / 8, row0 = tid / (2 * row16), rows = kEvict / (2 * row16);
    const int piece = tid - row0 * 2 * row16, col = piece < row16 ? piece : piece - row16;
    const bool moving = row0 < rows;  // (a few threads are left over where rows do not divide them)
    const int shift = __ffs(c.page_size) - 1;
    const long long plane = (long long)c.page_size * row16, page = plane * c.heads;
    uint4* base = static_cast<uint4*>(piece < row16 ? c.k : c.v) +
                  ((long long)layer * c.pages * c.heads + head) * plane + col;
    auto at = [&](int tok) {
        return base + pages[tok >> shift] * page + (tok & (c.page_size - 1)) * row16;
    };

    if (top > 0) {
        for (int j = tid; j < 48; j += kEvict) sm.counts[j / 3][j % 3] = 0;
        if (tid == 0) sm.listed = 0;
        if (cached)
            for (int j = tid; j < many; j += kEvict) keys[j] = key_of(w[sinks + j]);
        __syncthreads();
        // ---- the lowest kept key: its bits from above, two at a time.  `need` of the `group`
        // keys that begin like it are kept.  Once few keys do, they alone are looked at, and
        // once all of them are kept (soon, without ties) the other bits do not matter.
        unsigned edge = 0;
        int need = top, group = many;
        bool listed = false;
        unsigned* list = reinterpret_cast<unsigned*>(sm.hole);  // (not used yet)
        for (int step = 0; step < 16; ++step) {
            const int shift = 30 - 2 * step;
            if (!listed && group <= 2 * kPairs && group < many / 2) {
                for (int j = tid; j < many; j += kEvict) {
                    const unsigned x = key(j);
                    if ((x >> shift >> 2) == edge) list[atomicAdd(&sm.listed, 1)] = x;
                }
                __syncthreads();
                listed = true;
            }
            int more[3] = {0, 0, 0};
            const int end = listed ? sm.listed : many;
            for (int j = tid; j < end; j += kEvict) {
                const unsigned x = (listed ? list[j] : key(j)) >> shift;
                if ((x >> 2) != edge) continue;
                const unsigned digit = x & 3u;
                more[0] += digit >= 1;
                more[1] += digit >= 2;
                more[2] += digit >= 3;
            }
            for (int d = 0; d < 3; ++d) {
                const int all = __reduce_add_sync(0xffffffffu, more[d]);
                if ((tid & 31) == 0 && all) atomicAdd(&sm.counts[step][d], all);
            }
            __syncthreads();
            int digit = 0, from = group, above = sm.counts[step][0];  // keys of this digit on, of the next on
            for (int d = 1; d <= 3; ++d) {
                if (sm.counts[step][d - 1] < need) break;
                digit = d;
                from = sm.counts[step][d - 1];
                above = d < 3 ? sm.counts[step][d] : 0;
            }
            need -= above;
            group = from - above;
            edge = edge * 4 + digit;
            if (need == group) {
                edge <<= shift;
                break;
            }
        }
        const bool ranked = need < group;  // some ties are dropped: those of the highest places
        // ---- each thread's stretch (an odd number of keys: no two threads in one bank)
        const int stretch = ((many + kEvict - 1) / kEvict) | 1;
        const int j0 = (int)min((long long)many, (long long)tid * stretch), j1 = min(many, j0 + stretch);
        long long total;
        int ties = 0, low_ties = 0;  // of all, and of those before `top`
        for (int j = j0; ranked && j < j1; ++j)
            if (key(j) == edge) {
                ++ties;
                low_ties += j < top;
            }
        const int tie0 = ranked ? (int)cta_scan<kEvict>(ties, sm.sums, total) : 0;
        // visits the holes and the rows that move, in ascending order
        auto visit = [&](auto&& hole, auto&& from) {
            int tie = tie0;
            for (int j = j0; j < j1; ++j) {
                if (j == top) tie = tie0 + low_ties;  // (a hole that has been filled may be a tie now)
                const unsigned x = key(j);
                bool stays = x >= edge;
                if (ranked && x == edge) stays = tie++ < need;
                if (stays && j >= top) from(j);
                if (!stays && j < top) hole(j);
            }
        };
        int holes = 0, froms = 0;
        visit([&](int) { ++holes; }, [&](int) { ++froms; });
        const long long before = cta_scan<kEvict>(((long long)holes << 32) | froms, sm.sums, total);
        const int hole0 = (int)(before >> 32), from0 = (int)before, moves = (int)total;
        // The last moves first: a moved weight changes the key of a hole, where keys are not in
        // shared memory, and a stretch's holes are counted from below.
        for (int first = (moves - 1) / kPairs * kPairs; first >= 0 && moves > 0; first -= kPairs) {
            int h = hole0 - first, f = from0 - first;
            visit([&](int j) { if (h >= 0 && h < kPairs) sm.hole[h] = sinks + j; ++h; },
                  [&](int j) { if (f >= 0 && f < kPairs) sm.hole[kPairs + f] = sinks + j; ++f; });
            __syncthreads();
            const int now = min(kPairs, moves - first);
            for (int m = row0; moving && m < now; m += kRun * rows) {
                uint4 v[kRun];
#pragma unroll
                for (int r = 0; r < kRun; ++r)
                    if (m + r * rows < now) v[r] = __ldcs(at(sm.hole[kPairs + m + r * rows]));
#pragma unroll
                for (int r = 0; r < kRun; ++r)
                    if (m + r * rows < now) __stcs(at(sm.hole[m + r * rows]), v[r]);
            }
            for (int m = tid; m < now; m += kEvict) w[sm.hole[m]] = w[sm.hole[kPairs + m]];
            __syncthreads();
        }
    }

    // ---- the recent rows close up: a run lies above all that earlier runs have written
    const bool apart = recent <= len - keep;  // (nothing that is written is read)
    for (int m0 = 0; m0 < recent; m0 += kRun * rows) {
        const int m = moving ? m0 + row0 : recent;
        uint4 v[kRun];
#pragma unroll
        for (int r = 0; r < kRun; ++r)
            if (m + r * rows < recent) v[r] = __ldcs(at(last + m + r * rows));
        if (!apart) __syncthreads();
#pragma unroll
        for (int r = 0; r < kRun; ++r)
            if (m + r * rows < recent) __stcs(at(gap + m + r * rows), v[r]);
    }
    for (int m0 = 0; m0 < recent; m0 += kEvict) {
        const int m = m0 + tid;
        float x = 0.f;
        if (m < recent) x = w[last + m];
        if (!apart) __syncthreads();
        if (m < recent) w[gap + m] = x;
    }
    __syncthreads();
    for (int m = keep + tid; m < len; m += kEvict) w[m] = 0.f;
}

bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" fa_status fa_cache_evict(const fa_cache* cache, const int* slots, const int* keep, int keep_all,
                                    int recent, int sinks, float* weights, int n, fa_stream_t stream) {
    const fa_status st = check_cache(cache);
    if (st != FA_OK) return st;
    if (n < 0 || n > cache->slots || recent < 0 || sinks < 0 || recent > 0x7FFFFFFF - sinks ||
        (!keep && keep_all < recent + sinks))
        return FA_ERR_INVALID_ARG;
    if (n == 0) return FA_OK;
    if (!slots || !weights || !aligned(slots, 4) || !aligned(keep, 4) || !aligned(weights, 4))
        return FA_ERR_INVALID_ARG;
    const long long units = (long long)n * cache->layers * cache->heads;
    if (units > 0x7FFFFFFFLL) return FA_ERR_UNSUPPORTED;
    cudaStream_t strm = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = launch_pdl(evict_plan_kernel, dim3(1), dim3(kPlan), 0, strm, *cache, slots, keep,
                               keep_all, recent, sinks, n);
    if (e != cudaSuccess) return FA_ERR_CUDA;
    const long long room = (long long)cache->max_pages * cache->page_size;
    const int keys = (int)(room < kMostKeys ? room : kMostKeys);
    // The search takes the longer the more places there are, the moves the longer the fewer
    // CTAs an SM has: 512 threads for tables of more than 8192 places (16k: 140 us against
    // 170 with 256 threads), 256 below (5120 places: 231 against 234; 2304: 253 against 270; 640: 226
    // against 358; sequences that fill their tables).
    const bool many = room > 8192;
    auto kern = many ? evict_kernel<512> : evict_kernel<256>;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kMostKeys * (int)sizeof(unsigned));
    if (e != cudaSuccess) return FA_ERR_CUDA;
    e = launch_pdl(kern, dim3((unsigned)units), dim3(many ? 512 : 256), (size_t)keys * sizeof(unsigned), strm,
                   *cache, weights, recent, sinks, keys);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
