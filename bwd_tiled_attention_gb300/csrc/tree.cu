// tree.cu -- attention of new tokens over a paged key/value cache, for sm_103a:
// single tokens, chunks of a prompt (causal) and trees of drafted tokens.
//
// A sequence holds len = ctx + n tokens in the cache, the last n of which are
// the call's.  Row t sees every key of the context, and of its own n tokens
// those with index <= t (no mask) or those whose bit is set in its mask row.
//   m = max_j s_j,  l = sum_j 2^(s_j - m),  O = sum_j 2^(s_j - m) v_j / l,
// with s = q.k * scale * log2 e over the visible keys j; LSE = (m + log2 l) ln 2.
// The sums split: any two disjoint key ranges with their own (m, l, O~) join by
// rescaling both to the larger m.  That identity carries the kernel twice: the
// two softmax streams of a CTA take alternate key tiles, and the CTAs take
// equal stretches of all tiles together, whatever item those belong to.
//
// Bound: reading the cache once.  The query rows are the group's heads times
// the tokens (row = token * G + head), so a decoding step has few of them and
// the tensor core runs mostly padded rows; a 128 x 128 x 128 tile pair costs
// ~1040 tensor cycles against the ~2800 that its 64 KB take at this SM's share
// of the memory bandwidth, so padding is free and the work per SM is all that
// matters.  Hence:
//   - linear split: all (sequence, kv head, row tile) items' key tiles stand in
//     one line and CTA c takes [c * per, (c + 1) * per).  Every SM streams the
//     same number of tiles for any mix of lengths; an item that spans CTAs
//     leaves partials, joined in a fixed order: with few rows by the CTA that
//     finishes last, otherwise by a second kernel.
//   - the K and V tiles of a CTA run through one ring of stages in the order
//     the tensor core consumes them, filled by TMA boxes of one page each, K
//     and V by a warp each.
//   - up to d = 128 two streams (softmax warpgroups, S/P and O in TMEM) work on
//     alternate key tiles of one row tile; with more than 128 rows they take
//     two row tiles and share each key tile (PAIR), since then the tensor core
//     is the bound.  Above d = 128 TMEM holds one O: one stream with two S
//     buffers, on tiles of 64 keys.
//   - up to 32 rows at d = 64 (FEW) stand four times in the tile, and each lane
//     quarter's warp works on a quarter of the keys: its P is 0 elsewhere, and the
//     quarters' O add up at the end as the streams' do.  A tile's 32 KB take 1400
//     cycles of memory there, and one warp's chain over 128 keys as many (64
//     sequences of 4-8k tokens, 8 kv heads, 142 -> 135 us; trees of 5-26 over
//     0.7-2k, 36.9 -> 35.0).  At d = 128 memory takes twice that, and loading Q four
//     times and adding up O cost more than they gave (16 x 4 tokens 47 -> 50 us).
//
// Measured (GPU time of a call among queued ones; the pairs of figures at single
// choices are replays of a graph of one call, which take ~3 us more): 64 sequences
// of 4-8k tokens, 32 + 8 heads of 128, one token each, 240 us = 6.7 TB/s, the rate
// of a copy (d = 64, 8 heads, 132 us at 6.1 TB/s; d = 96 190 us at 6.3; d = 192 and
// 256, 32 sequences, 16 + 4 heads, 101 us at 6.0 and 128 us at 6.3).  2048-token
// chunks over 4000 and 6000 keys, 32 + 8 heads of 128: 367 us = 1168 TF/s (d = 96
// 342 us; 16 + 4 heads of 192 330 us); 1500- and 2048-token chunks over 4-6k, 16 + 4
// heads of 256: 340 us = 1167 TF/s; 4 trees of 64 over 30-33k keys 125 us.  One token
// over 501 keys 11.8 us: ~2.6 us of lookups and arithmetic, ~2 us until the first
// tile is there, its chain, the join.
//
// With a window of W keys and S first ones (sinks; tree_window.cu compiles these kernels),
// a row at position p sees of the keys j before `limit` those with p - j < W or j < S.
// An item's tiles are then those of the sinks and a stretch that begins where its first
// row's window does; everything else -- the line, the split, the join -- counts tiles as
// before, and a tile of the count is turned into one of the sequence where keys are
// named.  A drafted token stands as many places behind the context as its row names
// others of the call's own tokens, or as its depth says, and the window hides keys of the
// context alone: where drafts may be deeper than the window, the mask leaves out what it hides
// of them (tree_near_kernel, once a step for all layers).
// Measured, 64 sequences of 8-16k tokens, 32 + 8 heads of 128, one token each, W = 4096, S =
// 16: 171 us = 6.3 TB/s of visible keys and values; one token over 5001, W = 512, 16 heads
// 12.5 us; 16 sequences of 16k, 512 tokens each, W = 1024: 249 us = 555 TF/s.
//
// Pages hold whatever was there before: keys past the length never reach a
// sum (their scores are replaced, their V rows zeroed in shared memory), and
// a drafted token's V that is not finite is kept from the rows that do not
// see it: it is zeroed in shared memory and added to the rows that do see it
// at the end.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstring>

#include "../../include/fa.h"
#include "cache.cuh"
#include "common.cuh"
#include "internal.h"
#include "sm100_ptx.cuh"

namespace fa {
namespace {

#ifdef FA_WINDOW
constexpr bool kWin = true;
#else
constexpr bool kWin = false;
#endif

constexpr int kThreads = 384;
constexpr float kRescale = 8.0f;  // log2 units: P <= 256 before the reference moves

// PAIR: two row tiles.  FEW (d = 64): up to 32 rows, which stand in all four lane
// quarters of the tile; each quarter's warp takes a quarter of the keys.
template <int D, bool PAIR, bool FEW>
struct Cfg {
    static constexpr int kBN = D > 128 ? 64 : 128;       // keys of a tile
    static constexpr int kCols = D / 64;                 // 64-column boxes
    static constexpr int kQTiles = PAIR ? 2 : 1;
    static constexpr int kQBytes = 128 * D * 2;
    static constexpr int kStageBytes = kBN * D * 2;      // one K or V tile
    static constexpr int kXStep = 36;                    // FEW: floats of 32 columns of O in shared memory
    static constexpr int kXBytes = FEW ? 2 * 128 * kXStep * 4 : 0;
    // what 227 KB leave beside Q, the alignment, and the barriers and statistics
    static constexpr int kRoom = 232448 - 1024 - 5120 - kQTiles * kQBytes - kXBytes;
    static constexpr int kMaxStages = kRoom / kStageBytes;
    static constexpr int kStages = kMaxStages > 8 ? 8 : kMaxStages;
    static constexpr int kStreams = D > 128 ? 1 : 2;     // O accumulators
    // d = 64 and d > 128 leave TMEM for P in columns of its own (behind two O of 64
    // columns, or between the S buffers of 64), so that the next scores need not
    // wait until PV has read the P of those two tiles before (decoding 64 sequences
    // of 4-8k tokens, 8 kv heads of 64: 154 -> 146 us; 2048-token chunks over 4-6k
    // keys, d = 256: 392 -> 367 us).
    static constexpr bool kSepP = D != 128;
    // scores of a row held in registers: 64 of them, or where the tensor core is the bound
    static constexpr bool kWhole = PAIR || kBN == 64;
    static constexpr int kOStep = D == 64 ? 64 : 128;    // columns from O_0 to O_1
    static constexpr int kPCol = D == 64 ? 384 : (kSepP ? 64 : 0), kPStep = D == 64 ? 64 : 128;
    static_assert(kStages >= 4, "the ring holds two K and two V tiles");
    static_assert(!PAIR || D <= 128, "two row tiles need two O accumulators");
    static_assert(!FEW || (D == 64 && !PAIR), "a warpgroup adds up half of 64 columns at once");
};

// A stretch of one item's key tiles, worked on by one CTA.
struct Piece {
    int b, h;            // sequence (< 0: none left), kv head
    int tok0, ntok;      // first token of the row tile(s) in the packed batch, tokens
    int trow0;           // the first token's index in the sequence
    int slot, ctx, len;
    int k0, n;           // key tiles [k0, k0 + n)
#ifdef FA_WINDOW
    int nsk, lo;         // of the item's tiles the first nsk hold sinks, the others begin at lo
#endif
    int part;            // partial slot, or -1: the whole item
    int first_cta, last_cta;  // the CTAs that share the item
    // First key of the piece's tile j.
    __device__ __forceinline__ int tile_key(int j, int bn) const {
#ifdef FA_WINDOW
        return (k0 + j < nsk ? k0 + j : lo + (k0 + j - nsk)) * bn;
#else
        return (k0 + j) * bn;
#endif
    }
};

// What the window leaves of a piece (everything, without one).  A row sees key j when
// j >= from or j < sinks, apart from what `limit` and the mask say.
struct Sight {
    int open;            // every row of the piece sees all keys before that ...
    int open_lo;         // ... from here on, and the sinks
    int all_lo;          // no row sees keys before that but the sinks
    int sinks;
    __device__ __forceinline__ Sight(const TreeParams& p, const Piece& x) {
        open = p.mask ? x.ctx : min(x.len, x.ctx + x.trow0 + 1);
        open_lo = all_lo = sinks = 0;
        if constexpr (kWin) {
            sinks = p.sinks;
            if (p.mask) {
                open_lo = min(x.ctx, x.len - p.window);
                all_lo = x.ctx - p.window + 1;
            } else {
                open_lo = x.ctx + x.trow0 + x.ntok - p.window;
                all_lo = x.ctx + x.trow0 - p.window + 1;
            }
        }
    }
    // Is some key of [key, key + n) hidden from some row?
    __device__ __forceinline__ bool ragged(int key, int n) const {
        return key + n > open || (kWin && key < open_lo && key + n > sinks);
    }
    __device__ __forceinline__ bool hidden_from_some(int key) const {
        return key >= open || (kWin && key < open_lo && key >= sinks);
    }
    __device__ __forceinline__ bool hidden_from_all(int key, int len) const {
        return key >= len || (kWin && key < all_lo && key >= sinks);
    }
};

// Tokens of its sequence's n own ones, other than itself, that token `trow` names in its row of
// the mask.
__device__ __forceinline__ int named_others(const uint32_t* row, int words, int n, int trow) {
    int others = 0;
#pragma unroll 1
    for (int w = 0; w * 32 < n && w < 2 * words; ++w) {
        uint32_t bits = row[w];
        if (n - w * 32 < 32) bits &= (1u << (n - w * 32)) - 1u;
        if (trow >> 5 == w) bits &= ~(1u << (trow & 31));
        others += __popc(bits);
    }
    return others;
}

// First key of the window of token `trow` of its sequence (0: no window); words: its row
// of the mask, or null; tok: its place in the batch.
__device__ __forceinline__ int window_from(const TreeParams& p, const Piece& x, const uint32_t* words,
                                           int trow, size_t tok) {
    if constexpr (!kWin) return 0;
    if (!p.mask) return x.ctx + trow - p.window + 1;
    const int n = x.len - x.ctx;
    const int others = p.depth ? max(0, min(p.depth[tok], n - 1)) : named_others(words, p.words, n, trow);
    return min(x.ctx, x.ctx + others - p.window + 1);
}

// Bits of the keys of [kb, kb + 32) that a window from `from` with its sinks leaves.
__device__ __forceinline__ uint32_t window_bits(int kb, int from, int sinks) {
    const int low = from - kb, few = sinks - kb;
    uint32_t hidden = low <= 0 ? 0u : (low >= 32 ? 0xffffffffu : (1u << low) - 1u);
    if (few > 0) hidden &= few >= 32 ? 0u : ~((1u << few) - 1u);
    return ~hidden;
}

template <int D, bool PAIR, bool FEW>
struct Smem {
    using C = Cfg<D, PAIR, FEW>;
    alignas(1024) uint8_t q[C::kQTiles][C::kQBytes];
    alignas(1024) uint8_t kv[C::kStages][C::kStageBytes];
    alignas(8) uint64_t full[C::kStages], empty[C::kStages];
    uint64_t q_full, q_empty, piece_full[2], piece_empty[2];
    uint64_t s_full[2], p_full[2], p_hi[2], o_done[2], o_free[2], stat_full, drain, begun, stored, x_full[2];
    Piece piece[2];
    int start[4];        // this CTA's first item: sequence, kv head, row tile, key tile
    long long line[3];   // tiles of a CTA, and this CTA's stretch
    long long sums[kThreads / 32];
    Piece shared[2];     // fused: this CTA's pieces of items that it shares
    int n_shared, join_last[2];
    int early;           // the first piece ends an item begun elsewhere: brought as soon as it is stored
    uint32_t tmem_base;
    int abort_flag, zero;
    int poison;          // a drafted V that is not finite has been met (never cleared)
    // row statistics that the two warpgroups exchange: [piece parity][stream][m, l]
    float stats[2][2][2][128];
    alignas(16) float x[FEW ? 2 : 1][FEW ? 128 : 1][C::kXStep];  // FEW: O of a warpgroup's lanes
};

template <int D, bool PAIR, bool FEW>
constexpr size_t smem_bytes() {
    static_assert(sizeof(Smem<D, PAIR, FEW>) + 1024 <= 232448, "shared memory exceeds 227 KB");
    return sizeof(Smem<D, PAIR, FEW>) + 1024;
}

// A sequence whose boundaries decrease or leave the batch owns nothing (the
// status word says so).  Where there is one, each token is looked for in all
// sequences, by one warp of `warps`, and the rows of those found in none are
// written as empty.
template <int DR>
__device__ __forceinline__ void clear_unowned(const TreeParams& p, int warp, int warps) {
    bool odd = false;
#pragma unroll 1
    for (int i = lane_id(); i < p.B; i += 32) odd |= seq_range(p.cu, p.N, p.T, i).n < 0;
    if (!__any_sync(0xffffffffu, odd)) return;
#pragma unroll 1
    for (long long t = warp; t < p.T; t += warps) {
        bool owned = false;
#pragma unroll 1
        for (int i = lane_id(); i < p.B && !owned; i += 32) {
            const SeqRange r = seq_range(p.cu, p.N, p.T, i);
            owned = t >= r.t0 && t < (long long)r.t0 + r.n;
        }
        if (__any_sync(0xffffffffu, owned)) continue;
        uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + t * p.Hq * DR);
#pragma unroll 1
        for (int i = lane_id(); i < p.Hq * (DR / 8); i += 32) o[i] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
        for (int h = lane_id(); h < p.Hq; h += 32) p.lse[(long long)h * p.T + t] = -INFINITY;
    }
}

struct SeqInfo {
    int t0, n, slot, len, ctx, bad;
};

__device__ __forceinline__ SeqInfo seq_info(const TreeParams& p, int i) {
    SeqInfo s;
    const int slot = p.slots[i];  // (in one trip with the boundaries)
    const SeqRange r = seq_range(p.cu, p.N, p.T, i);
    s.t0 = r.t0;
    s.n = r.n;
    s.slot = s.len = s.ctx = s.bad = 0;
    if (r.n < 0) {  // boundaries out of order: no rows
        s.n = 0;
        s.bad = kCacheBadLength;
        return s;
    }
    if (r.n == 0) return s;
    s.slot = slot;
    if (s.slot < 0 || s.slot >= p.cache.slots) {
        s.slot = 0;
        s.bad = kCacheBadSlot;
        return s;
    }
    const int len = p.cache.lengths[s.slot];
    if (len < s.n || s.n > p.N || len > (long long)p.cache.max_pages * p.cache.page_size) {
        s.bad = kCacheBadLength;  // its rows see no key
        return s;
    }
    s.len = len;
    s.ctx = len - s.n;
    return s;
}

// With a window: the first tile behind the sinks' that row tile q visits, and the sinks'.
__device__ __forceinline__ int window_tiles(const TreeParams& p, const SeqInfo& s, int q, int tokens,
                                            int bn, int& sink_tiles) {
    const int pos = p.mask ? s.ctx : s.ctx + q * tokens;  // of its first row (at least)
    const int lo = s.len > 0 ? max(0, pos - p.window + 1) / bn : 0;
    sink_tiles = min((p.sinks + bn - 1) / bn, lo);
    return lo;
}

// Key tiles that row tile q of a sequence visits (one even when it sees no
// key, so that its rows are written).
__device__ __forceinline__ int item_tiles(const TreeParams& p, const SeqInfo& s, int q, int tokens,
                                          int bn) {
    int keys = s.len;
    if (!p.mask && s.len > 0) keys = min(s.len, s.ctx + min(s.n, (q + 1) * tokens));
    int tiles = (keys + bn - 1) / bn;
    if constexpr (kWin) {
        int few;
        tiles -= window_tiles(p, s, q, tokens, bn, few);
        tiles += few;
    }
    return max(1, tiles);
}

__device__ __forceinline__ long long head_tiles(const TreeParams& p, const SeqInfo& s, int tokens,
                                                int bn) {
    const int nq = (s.n + tokens - 1) / tokens;
    if (p.mask || s.len == 0) return (long long)nq * item_tiles(p, s, 0, tokens, bn);
    long long sum = 0;
#pragma unroll 1
    for (int q = 0; q < nq; ++q) sum += item_tiles(p, s, q, tokens, bn);
    return sum;
}

// a / b without a 64-bit division where both fit 32 bits (nearly always).
__device__ __noinline__ long long divide_far(long long a, long long b) { return a / b; }
__device__ __forceinline__ long long divide(long long a, long long b) {
    if (((a | b) >> 32) == 0) return (long long)((uint32_t)a / (uint32_t)b);
    return divide_far(a, b);
}

// Finds tile `at` (counted from the sequence's first) of sequence s.
__device__ __forceinline__ void locate(const TreeParams& p, const SeqInfo& s, long long at,
                                       long long head, int tokens, int bn, int& h, int& q, int& k) {
    h = (int)divide(at, head);
    k = (int)(at - h * head);
    if (p.mask || s.len == 0) {
        const int t = item_tiles(p, s, 0, tokens, bn);
        q = k / t;
        k -= q * t;
        return;
    }
#pragma unroll 1
    for (q = 0;; ++q) {
        const int t = item_tiles(p, s, q, tokens, bn);
        if (k < t) return;
        k -= t;
    }
}

// Bounded wait; on giving up the CTA stops and the status word says so.
__device__ __forceinline__ bool poll(uint32_t bar, uint32_t parity, volatile int* flag, int* status) {
    if (mbar_wait(bar, parity, flag)) return true;
    *flag = 1;
    atomicOr(status, kCacheTimeout);
    return false;
}
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* flag,
                                          int* status) {
    return __all_sync(0xffffffffu, poll(bar, parity, flag, status));
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, uint32_t bar, int c0,
                                            int c1, int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

__device__ __forceinline__ void fence_gpu() { asm volatile("fence.acq_rel.gpu;" ::: "memory"); }

// Bits 15 and 31: the low or high bf16 of a pair is an infinity or NaN (its
// exponent, all ones, carries).
__device__ __forceinline__ uint32_t not_finite(uint32_t pair) {
    return ((pair & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
}
__device__ __forceinline__ bool finite_bf16(uint32_t lo16) { return (lo16 & 0x7F80u) != 0x7F80u; }

// Bits of the 32 keys from `j0` (an index among the sequence's own tokens;
// negative: the context) that a row sees.
__device__ __forceinline__ uint32_t mask_bits(const uint32_t* words, int nwords, int j0) {
    const int w = j0 >> 5;  // floor
    const uint32_t lo = w < 0 ? 0xffffffffu : (w < nwords ? words[w] : 0u);
    const uint32_t hi = w + 1 < 0 ? 0xffffffffu : (w + 1 < nwords ? words[w + 1] : 0u);
    return __funnelshift_r(lo, hi, j0 & 31);
}

// One warp's loads of K or V tiles into the ring: a box is one page's keys (or
// 64 of them) by 64 columns, and each box of a tile is a lane's.  K and V have a
// warp each: a lane's TMA takes ~95 cycles to issue, and a tile of 16-token
// pages at d = 128 has 16 boxes.
//
// The wait for a stage looks at a phase's parity only.  That is enough: tile
// loads are consumed in ring order, and this warp's previous load has waited
// for the consumer to pass the place S before it, so the stage is at most one
// phase behind.
template <int BN, int S, int COLS>
struct Loader {
    const TreeParams& p;
    const CUtensorMap* map;
    uint8_t* ring;
    uint64_t *full, *empty;
    volatile int* stop;
    int ps, shift, rows, rows_shift, boxes, box, col, box_key;
    uint32_t dst;
    // of the piece: page ids of a window of 32 pages, and of the next one
    const int* table;
    int used, win, ids, nxt, key0, len, head;
#ifdef FA_WINDOW
    int left, jump_key, jump_ids, jump_nxt;  // tiles before the window's stretch, and where it begins
    int sinks, all_lo;                       // no row sees keys of [sinks, all_lo)
#endif
    int place = -1;  // ring place of this lane's turn among the last 32 loads
    int count = 0;

    __device__ __forceinline__ Loader(const TreeParams& p_, const CUtensorMap* map_, uint8_t* ring_,
                                      uint64_t* full_, uint64_t* empty_, volatile int* stop_)
        : p(p_), map(map_), ring(ring_), full(full_), empty(empty_), stop(stop_) {
        ps = p.cache.page_size;
        shift = p.page_shift;
        rows = min(ps, BN);
        rows_shift = rows == ps ? shift : 6;  // (pages of 128 tokens, tiles of 64)
        boxes = BN >> rows_shift;
        box = lane_id() / COLS;
        col = lane_id() % COLS;
        box_key = box << rows_shift;
        dst = col * (BN * 128) + box_key * 128;
    }
    __device__ __forceinline__ int table_at(int i) const { return i < used ? table[i] : -1; }
    __device__ __forceinline__ void begin(const Piece& x) {
        table = p.cache.table + (long long)x.slot * p.cache.max_pages;
        len = x.len;
        head = x.h;
        used = (len + ps - 1) >> shift;
        key0 = x.tile_key(0, BN);
        win = key0 >> shift;
        ids = table_at(win + lane_id());
        nxt = table_at(win + 32 + lane_id());
#ifdef FA_WINDOW
        const Sight sight(p, x);
        sinks = sight.sinks;
        all_lo = sight.all_lo;
        left = x.nsk - x.k0;
        jump_key = x.lo * BN;
        if (left > 0) {
            jump_ids = table_at((jump_key >> shift) + lane_id());
            jump_nxt = table_at((jump_key >> shift) + 32 + lane_id());
        }
#endif
    }
    // The piece's next tile into place f of the ring.
    __device__ __forceinline__ bool tile(int f, int* status) {
        const int first = key0 >> shift;
        if (first >= win + 32) {
            win += 32;
            ids = nxt;
            nxt = table_at(win + 32 + lane_id());
        }
        const int page = __shfl_sync(0xffffffffu, ids, (first - win + box) & 31);
        const int st = f % S;
        if (!warp_wait(smem_u32(&empty[st]), ((f / S) & 1) ^ 1, stop, status)) return false;
        const int have = max(0, min(boxes, (len - key0 + rows - 1) >> rows_shift));
        const uint32_t bar = smem_u32(&full[st]);
        int gone0 = 0, gone1 = 0;
#ifdef FA_WINDOW
        // Boxes of keys that no row sees are left out (64 sequences, W = 4096, 16 sinks:
        // 173.5 -> 170.7 us): their scores are replaced and their V zeroed, as behind the length.
        gone0 = min(have, max(0, (sinks - key0 + rows - 1) >> rows_shift));
        gone1 = max(gone0, min(have, (all_lo - key0) >> rows_shift));
#endif
        if (lane_id() == 0) mbar_arrive_expect_tx(bar, (have - (gone1 - gone0)) * rows * 128 * COLS);
        __syncwarp();
        if (box < have && (box < gone0 || box >= gone1)) {
            // a page id out of range reads the fill value (zeros) and is reported
            int plane = -1;
            if (page >= 0 && page < p.cache.pages)
                plane = (p.layer * p.cache.pages + page) * p.cache.heads + head;
            else
                atomicOr(status, kCacheBadSlot);
            tma_load_3d(smem_u32(ring) + st * (BN * COLS * 128) + dst, map, bar, col * 64,
                        (key0 + box_key) & (ps - 1), plane);
        }
        if ((count & 31) == (int)lane_id()) place = f;
        ++count;
        key0 += BN;
#ifdef FA_WINDOW
        if (--left == 0) {
            key0 = jump_key;
            win = key0 >> shift;
            ids = jump_ids;
            nxt = jump_nxt;
        }
#endif
        return true;
    }
    // After an abort: waits (bounded) for the loads that may still fly.
    __device__ __forceinline__ void drain(const volatile int* never) {
        int last = place;
        for (int o = 16; o; o >>= 1) last = max(last, __shfl_xor_sync(0xffffffffu, last, o));
        if (place >= 0 && place > last - S) mbar_wait(smem_u32(&full[place % S]), (place / S) & 1, never);
        __syncwarp();
    }
};

// P = 2^(s c - m) of 32 columns as bf16 pairs (each rounded once: P enters the
// tensor core in the type of V), and their fp32 sum before that rounding.
__device__ __forceinline__ void exp_chunk(const float* s, float c, float neg, uint64_t (&acc)[2],
                                          uint32_t (&pk)[16]) {
    const uint64_t c2 = f2_pack(c, c), n2 = f2_pack(neg, neg);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint64_t x = f2_fma(f2_pack(s[2 * i], s[2 * i + 1]), c2, n2);
        float x0, x1;
        f2_unpack(x, x0, x1);
        x0 = ex2_approx(x0);
        x1 = ex2_approx(x1);
        acc[i & 1] = f2_add(acc[i & 1], f2_pack(x0, x1));
        pk[i] = pack_bf16x2(x0, x1);
    }
}

// FIFO place, within a piece of n tiles, of tile j's K and V.
template <bool PAIR>
__device__ __forceinline__ int fifo_k(int j) {
    return PAIR ? 2 * j : (j == 0 ? 0 : 2 * j - 1);
}
template <bool PAIR>
__device__ __forceinline__ int fifo_v(int j, int n) {
    return PAIR ? 2 * j + 1 : (j < n - 1 ? 2 * j + 2 : 2 * n - 1);
}

// One row of an item that CTAs c0 .. c0 + n - 1 shared, by one warp: partials
// stand in slot 2c + 1 of the first CTA and slot 2c of the others, and are
// added in that order.
template <int DR>
__device__ __forceinline__ void join_row(const TreeParams& p, int slot_row, int c0, int n, size_t tok,
                                         int head) {
    const int lane = lane_id();
    constexpr int V = DR / 32;                       // columns of a lane, contiguous
    constexpr int W = V % 4 == 0 ? 4 : (V % 2 == 0 ? 2 : 1);
    auto slot = [&](int i) { return (size_t)(2 * (c0 + i) + (i == 0)) * p.part_rows + slot_row; };
    const float2* stats = reinterpret_cast<const float2*>(p.part_stats);
    // This lane's partial's statistics, and the first partials' columns: one trip
    // to memory where there are few.
    constexpr int R = DR > 128 ? 2 : 4;              // partials in flight
    float x[R][V];
    auto fetch = [&](int i0) {
#pragma unroll
        for (int u = 0; u < R; ++u) {
            if (i0 + u >= n) continue;
            const float* at = p.part_o + slot(i0 + u) * DR + lane * V;
#pragma unroll
            for (int v = 0; v < V; v += W) {
                if (W == 4) {
                    const float4 y = __ldcg(reinterpret_cast<const float4*>(at + v));
                    x[u][v] = y.x; x[u][v + 1 % W] = y.y; x[u][v + 2 % W] = y.z; x[u][v + 3 % W] = y.w;
                } else if (W == 2) {
                    const float2 y = __ldcg(reinterpret_cast<const float2*>(at + v));
                    x[u][v] = y.x; x[u][v + 1 % W] = y.y;
                } else {
                    x[u][v] = __ldcg(at + v);
                }
            }
        }
    };
    float2 st = make_float2(-INFINITY, 0.f);
    if (lane < n) st = __ldcg(stats + slot(lane));
    fetch(0);
    float m = st.x;
    for (int i = lane + 32; i < n; i += 32) m = fmaxf(m, __ldcg(stats + slot(i)).x);
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float base = m == -INFINITY ? 0.f : m;
    float acc[V], l = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.f;
    float w = 0.f, lw = 0.f;
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += R) {
        if (i0 > 0) fetch(i0);
        if ((i0 & 31) == 0) {                        // weights of the next 32 partials
            if (i0 > 0)
                st = i0 + lane < n ? __ldcg(stats + slot(i0 + lane)) : make_float2(-INFINITY, 0.f);
            w = ex2_approx(st.x - base);
            lw = st.y * w;
        }
#pragma unroll
        for (int u = 0; u < R; ++u) {
            if (i0 + u >= n) break;
            const float wi = __shfl_sync(0xffffffffu, w, (i0 + u) & 31);
            l += __shfl_sync(0xffffffffu, lw, (i0 + u) & 31);
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] = fmaf(x[u][v], wi, acc[v]);
        }
    }
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    struct alignas(2 * W) Half { __nv_bfloat16 x[W]; };
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o) + (tok * p.Hq + head) * DR + lane * V;
#pragma unroll
    for (int v = 0; v < V; v += W) {
        Half y;
#pragma unroll
        for (int e = 0; e < W; ++e) y.x[e] = __float2bfloat16_rn(acc[v + e] * inv);
        *reinterpret_cast<Half*>(o + v) = y;
    }
    if (lane == 0) p.lse[(size_t)head * p.T + tok] = (m + __log2f(l)) * 0.69314718055994531f;
}

// FEW: the sums over lane quarters of columns [32 cc, 32 cc + 32) of a piece's
// rows, eight of them by each warp: stored, or left as the piece's partial.
template <int DR, int BN>
__device__ __forceinline__ void store_few(const TreeParams& p, const Piece& x, const float (*o)[36],
                                          const float (*stats)[2][128], bool two, int poison,
                                          const Sight& sight, int q4, int cc) {
    const int lane = lane_id(), row = q4 * 8 + (lane >> 2), col = (lane & 3) * 8;
    const int row_tok = row / p.group, head = x.h * p.group + row - row_tok * p.group;
    if (row_tok >= x.ntok) return;
    const size_t tok = (size_t)x.tok0 + row_tok;
    float y[8];
    bool odd = false;
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
        float4 a[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) a[k] = *reinterpret_cast<const float4*>(&o[k * 32 + row][col + i]);
        y[i] = (a[0].x + a[1].x) + (a[2].x + a[3].x);
        y[i + 1] = (a[0].y + a[1].y) + (a[2].y + a[3].y);
        y[i + 2] = (a[0].z + a[1].z) + (a[2].z + a[3].z);
        y[i + 3] = (a[0].w + a[1].w) + (a[2].w + a[3].w);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) odd |= !(fabsf(y[i]) < INFINITY);
    if (odd || poison) {
        // A visible V that is not finite adds itself, its weight being positive: a
        // drafted one was zeroed, and one of the context has made NaN of the quarters
        // whose P is 0 there.  A row whose sum is NaN stays NaN.
        float sum = 0.f, add[8] = {};
        for (int i = 0; i < (two ? 2 : 1); ++i)
            for (int k = 0; k < 4; ++k) sum += stats[i][1][k * 32 + row];
        const uint32_t* words = p.mask
            ? reinterpret_cast<const uint32_t*>(p.mask) + tok * (2 * (size_t)p.words) : nullptr;
        const int limit = p.mask ? x.len : min(x.len, x.ctx + x.trow0 + row_tok + 1);
        const int ps = p.cache.page_size;
        const int from = window_from(p, x, words, x.trow0 + row_tok, tok);
        const int skip = kWin || odd ? 0 : max(0, sight.open - x.tile_key(0, BN));  // (tiles in a row)
        for (int i = skip; i < x.n * BN && sum == sum; ++i) {
            const int key = x.tile_key(i / BN, BN) + i % BN;
            if (key >= limit) break;
            if (kWin && ((!odd && !sight.hidden_from_some(key)) || (key < from && key >= sight.sinks)))
                continue;
            if (p.mask && !(mask_bits(words, 2 * p.words, key - x.ctx) & 1u)) continue;
            const int page = p.cache.table[(long long)x.slot * p.cache.max_pages + key / ps];
            if (page < 0 || page >= p.cache.pages) continue;
            const uint16_t* v = static_cast<const uint16_t*>(p.cache.v) +
                                ((((long long)p.layer * p.cache.pages + page) * p.cache.heads + x.h) * ps +
                                 key % ps) * DR + cc * 32 + col;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t bits = v[i];
                if (!finite_bf16(bits)) add[i] += __uint_as_float(bits << 16);
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (add[i] != 0.f) y[i] = add[i];
    }
    if (x.part < 0) {
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + (tok * p.Hq + head) * DR + cc * 32 + col) =
            make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                       pack_bf16x2(y[6], y[7]));
    } else {
        float4* dst = reinterpret_cast<float4*>(p.part_o + ((size_t)x.part * p.part_rows + row) * DR +
                                                cc * 32 + col);
        dst[0] = make_float4(y[0], y[1], y[2], y[3]);
        dst[1] = make_float4(y[4], y[5], y[6], y[7]);
    }
}

// One thread says that this CTA's partial of an item is there; true: it was the
// last one.  The item's word counts those brought under this call's number;
// anything else that it holds counts as none, and the last one clears it.
__device__ __forceinline__ bool bring(const TreeParams& p, const Piece& x) {
    fence_gpu();  // all partials of the CTA, before it says that they are there
    unsigned long long* word = p.arrived + x.last_cta;
    unsigned long long old = 0, now;  // (what the last call left, most often)
    for (;;) {
        now = (old >> 8) == p.call ? old + 1 : (p.call << 8) + 1;
        const unsigned long long seen = atomicCAS(word, old, now);
        if (seen == old) break;
        old = seen;
    }
    const bool last = (int)(now & 255) == x.last_cta - x.first_cta + 1;
    if (last) {
        *word = 0;
        fence_gpu();
    }
    return last;
}

// D: tile columns; DR: head dimension in memory (96 runs on 128 columns whose
// last 32 the TMA fills with zeros).
template <int D, int DR, bool PAIR, bool FEW>
__global__ void __launch_bounds__(kThreads, 1) tree_kernel(const __grid_constant__ TreeParams p) {
    pdl_trigger();
    using C = Cfg<D, PAIR, FEW>;
    using SM = Smem<D, PAIR, FEW>;
    constexpr int S = C::kStages, BN = C::kBN;
    extern __shared__ uint8_t smem_raw[];
    SM& sm = *reinterpret_cast<SM*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                    ~uintptr_t(1023));
    const int warp = warp_id(), lane = lane_id();
    volatile int* stop = &sm.abort_flag;
    int* status = p.cache.scratch;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(smem_u32(&sm.full[s]), 1);
            mbar_init(smem_u32(&sm.empty[s]), 1);
        }
        mbar_init(smem_u32(&sm.q_full), 1);
        mbar_init(smem_u32(&sm.q_empty), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sm.piece_full[i]), 1);
            mbar_init(smem_u32(&sm.piece_empty[i]), 1 + 8 + 1);
            mbar_init(smem_u32(&sm.s_full[i]), 1);
            mbar_init(smem_u32(&sm.p_full[i]), 4);
            mbar_init(smem_u32(&sm.p_hi[i]), 4);
            mbar_init(smem_u32(&sm.o_done[i]), 1);
            mbar_init(smem_u32(&sm.o_free[i]), PAIR ? 4 : 8);
            mbar_init(smem_u32(&sm.x_full[i]), 4);
        }
        mbar_init(smem_u32(&sm.stat_full), 8);
        mbar_init(smem_u32(&sm.drain), 1);
        mbar_init(smem_u32(&sm.begun), 1);
        mbar_init(smem_u32(&sm.stored), 8);
        sm.abort_flag = sm.zero = sm.poison = 0;
        sm.start[0] = -1;
        sm.n_shared = sm.early = 0;
        fence_barrier_init();
    }
    if (warp == 2) {
        tmem_alloc(smem_u32(&sm.tmem_base), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    const int tokens = p.tile_tokens * C::kQTiles;  // tokens of an item
    if (warp == 1 && lane == 0) {
        tma_prefetch_desc(&p.tm_q);
        tma_prefetch_desc(&p.tm_k);
        tma_prefetch_desc(&p.tm_v);
    }
    pdl_wait();

    // ---- the line of all key tiles, and where this CTA's stretch begins: the
    // producer warp's own business for small batches, all threads' for large ones
    SeqInfo mine_info = {0, 0, 0, 0, 0, 0};  // (one sequence a lane: B <= 32)
    if (p.B <= 128 ? warp == 0 : true) {
        const bool all_threads = p.B > 128;
        const int chunk = all_threads ? (p.B + kThreads - 1) / kThreads : (p.B + 31) / 32;
        const int i0 = (all_threads ? (int)threadIdx.x : lane) * chunk, i1 = min(p.B, i0 + chunk);
        long long mine = 0;
        int bad = 0;
#pragma unroll 1
        for (int i = i0; i < i1; ++i) {
            const SeqInfo s = seq_info(p, i);
            bad |= s.bad;
            mine_info = s;
            mine += head_tiles(p, s, tokens, BN) * p.cache.heads;
        }
        if (bad && blockIdx.x == 0) atomicOr(status, bad);
        long long incl = mine;
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        long long before = 0, total = __shfl_sync(0xffffffffu, incl, 31);
        if (all_threads) {
            if (lane == 31) sm.sums[warp] = incl;
            __syncthreads();
            total = 0;
#pragma unroll 1
            for (int w = 0; w < kThreads / 32; ++w) {
                if (w < warp) before += sm.sums[w];
                total += sm.sums[w];
            }
        }
        const long long per = max(divide(total + gridDim.x - 1, gridDim.x), (long long)p.min_tiles);
        const long long begin = min(total, per * blockIdx.x), end = min(total, begin + per);
        if (threadIdx.x == 0) {
            sm.line[0] = per;
            sm.line[1] = begin;
            sm.line[2] = end;
        }
        long long at = before + incl - mine;  // first tile of this thread's sequences
        if (begin < end && begin >= at && begin < at + mine) {
#pragma unroll 1
            for (int i = i0; i < i1; ++i) {
                const SeqInfo s = chunk == 1 ? mine_info : seq_info(p, i);
                const long long ht = head_tiles(p, s, tokens, BN), all = ht * p.cache.heads;
                if (begin >= at + all) {
                    at += all;
                    continue;
                }
                sm.start[0] = i;
                locate(p, s, begin - at, ht, tokens, BN, sm.start[1], sm.start[2], sm.start[3]);
                break;
            }
        }
        if (all_threads) __syncthreads(); else __syncwarp();
    }
    // Registers: the launch gives every thread 168.  Two row tiles hold whole rows
    // of scores; one row tile's loops hold half, and the producer wants the rest.
    constexpr int kFewRegs = PAIR ? 72 : 104, kManyRegs = PAIR ? 216 : 200;
    static_assert(128 * kFewRegs + 256 * kManyRegs == 384 * 168, "register split must match the launch");

    if (warp == 0) {
        // ------------------------------------------------------------ pieces, Q and K
        setmaxnreg_dec<kFewRegs>();
        int it = 0, f = 0, nq = 0;  // pieces, ring places before this piece, query loads
        bool ok = true;
        int own_first = -1, own_tok0 = 0, own_ntok = 0, own_h = 0;  // an item that ends here
        int b = sm.start[0], h = sm.start[1], q = sm.start[2], k0 = sm.start[3];
        const long long per = sm.line[0], end = sm.line[2];
        long long at = sm.line[1];             // place in the line
        // sequence i's geometry: a small batch stays in the lanes that looked it up
        auto sequence = [&](int i) {
            if (p.B > 32) return seq_info(p, i);
            SeqInfo y;
            y.t0 = __shfl_sync(0xffffffffu, mine_info.t0, i);
            y.n = __shfl_sync(0xffffffffu, mine_info.n, i);
            y.slot = __shfl_sync(0xffffffffu, mine_info.slot, i);
            y.len = __shfl_sync(0xffffffffu, mine_info.len, i);
            y.ctx = __shfl_sync(0xffffffffu, mine_info.ctx, i);
            return y;
        };
        SeqInfo s;
        s.n = 0;
        if (at < end) s = sequence(b);
        Loader<BN, S, C::kCols> load(p, &p.tm_k, sm.kv[0], sm.full, sm.empty, stop);
        while (ok) {
            const int slot = it & 1;
            if (!(ok = warp_wait(smem_u32(&sm.piece_empty[slot]), ((it >> 1) & 1) ^ 1, stop, status)))
                break;
            Piece x;
            if (at >= end) {
                if (lane == 0) {
                    sm.piece[slot].b = -1;
                    mbar_arrive(smem_u32(&sm.piece_full[slot]));
                    if (it == 0) mbar_arrive(smem_u32(&sm.begun));
                }
                break;
            }
            const int tiles = item_tiles(p, s, q, tokens, BN);
            x.b = b;
            x.h = h;
            x.trow0 = q * tokens;
            x.tok0 = s.t0 + x.trow0;
            x.ntok = min(tokens, s.n - x.trow0);
            x.slot = s.slot;
            x.ctx = s.ctx;
            x.len = s.len;
            x.k0 = k0;
#ifdef FA_WINDOW
            x.lo = window_tiles(p, s, q, tokens, BN, x.nsk);
#endif
            x.n = (int)min((long long)(tiles - k0), end - at);
            const bool whole_end = k0 + x.n == tiles;
            x.part = k0 == 0 ? (whole_end ? -1 : 2 * (int)blockIdx.x + 1) : 2 * (int)blockIdx.x;
            x.first_cta = x.last_cta = blockIdx.x;
            if (k0 > 0) x.first_cta = (int)divide(at - k0, per);
            if (!whole_end) x.last_cta = (int)divide(at - k0 + tiles - 1, per);
            if (k0 > 0 && whole_end) {  // this CTA's first piece ends an item begun elsewhere
                own_first = x.first_cta;
                own_tok0 = x.tok0;
                own_ntok = x.ntok;
                own_h = h;
            }
            if (lane == 0) {
                sm.piece[slot] = x;
                if (x.part >= 0) sm.shared[sm.n_shared++] = x;  // the first and the last at most
                mbar_arrive(smem_u32(&sm.piece_full[slot]));
                if (!PAIR && it == 0) {
                    sm.early = k0 > 0;
                    mbar_arrive(smem_u32(&sm.begun));
                }
            }
            __syncwarp();

            auto load_q = [&] {
                if (!(ok = warp_wait(smem_u32(&sm.q_empty), (it & 1) ^ 1, stop, status))) return;
                if (lane == 0) {
                    const uint32_t bar = smem_u32(&sm.q_full);
                    const int nt = PAIR && x.ntok > p.tile_tokens ? 2 : 1;
                    constexpr int copies = FEW ? 4 : 1;
                    mbar_arrive_expect_tx(bar, nt * copies * p.tile_tokens * p.group * 128 * C::kCols);
                    for (int t = 0; t < nt; ++t)
                        for (int c = 0; c < C::kCols; ++c)
                            for (int y = 0; y < copies; ++y)  // (32 rows of 128 bytes apart)
                                tma_load_4d(smem_u32(sm.q[t]) + c * 16384 + y * 4096, &p.tm_q, bar,
                                            c * 64, 0, x.h, x.tok0 + t * p.tile_tokens);
                }
                __syncwarp();
                ++nq;
            };
            if (it == 0) load_q();  // (later pieces: behind the first key tile)
            load.begin(x);
            for (int j = 0; j < x.n && ok; ++j) {
                ok = load.tile(f + fifo_k<PAIR>(j), status);
                if (ok && j == 0 && it > 0) load_q();
            }
            f += 2 * x.n;
            ++it;
            // -- the next item
            at += x.n;
            k0 = 0;
            if (at < end) {
                ++q;
                if (q * tokens >= s.n) {
                    q = 0;
                    if (++h == p.cache.heads) {
                        h = 0;
                        do {
                            ++b;
                            if (b >= p.B) {  // (cannot be: the line counts real tiles)
                                at = end;
                                break;
                            }
                            s = sequence(b);
                        } while (s.n == 0);
                    }
                }
            }
        }
        if (lane == 0 && !p.fused) p.meta[blockIdx.x] = make_int4(own_first, own_tok0, own_ntok, own_h);
        if (!ok) {  // never leave a TMA write in flight
            load.drain(&sm.zero);
            if (lane == 0 && nq > 0) mbar_wait(smem_u32(&sm.q_full), (nq - 1) & 1, &sm.zero);
        }
    } else if (warp == 3) {
        // ------------------------------------------------------------ V
        setmaxnreg_dec<kFewRegs>();
        int it = 0, f = 0;
        bool ok = true;
        Loader<BN, S, C::kCols> load(p, &p.tm_v, sm.kv[0], sm.full, sm.empty, stop);
        while (ok) {
            const int slot = it & 1;
            if (!(ok = warp_wait(smem_u32(&sm.piece_full[slot]), (it >> 1) & 1, stop, status))) break;
            const Piece x = sm.piece[slot];
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.piece_empty[slot]));
            if (x.b < 0) break;
            load.begin(x);
            for (int j = 0; j < x.n && ok; ++j) ok = load.tile(f + fifo_v<PAIR>(j, x.n), status);
            f += 2 * x.n;
            ++it;
        }
        if (!ok) load.drain(&sm.zero);
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        setmaxnreg_dec<kFewRegs>();
        {
            constexpr uint32_t idS = make_idesc_bf16(128, BN, false, false);
            constexpr uint32_t idPV = make_idesc_bf16(128, D, false, true);
            int it = 0, f = 0;
            const uint32_t lead = elect_lead();
            int cnt[2] = {0, 0};  // tiles through each S buffer
            int done[2] = {0, 0}; // PAIR: pieces of each stream
            bool ok = true;
            // A tile that is nearly always there is looked up beside an earlier wait (a wait
            // costs ~140 cycles even when nothing is missing).  The place S before it has been
            // consumed by then, so that the parity tells.
            auto there = [&](int place) {
                return mbar_test_wait(smem_u32(&sm.full[place % S]), (place / S) & 1);
            };
            auto wait = [&](uint64_t& bar, int n) {
                return ok = ok && warp_wait(smem_u32(&bar), n & 1, stop, status);
            };
            auto issue_s = [&](int stage_no, int buf, int qt) {
                const uint64_t da = make_sdesc(smem_u32(sm.q[qt]), 16, 1024);
                const uint64_t db = make_sdesc(smem_u32(sm.kv[stage_no % S]), 16, 1024);
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < DR / 16; ++kk)
                    warp_mma_ss(lead, tmem + buf * 128, sdesc_add(da, (kk >> 2) * 16384 + (kk & 3) * 32),
                           sdesc_add(db, (kk >> 2) * (BN * 128) + (kk & 3) * 32), idS, kk > 0);
            };
            auto issue_pv = [&](int stage_no, int buf, int o, int c, bool first) {
                // keys [0, BN/2) of P, then the others once the softmax has them
                const uint64_t db = make_sdesc(smem_u32(sm.kv[stage_no % S]), BN * 128, 1024);
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < BN / 16; ++kk) {
                    if (!FEW && kk == BN / 32) {
                        if (!wait(sm.p_hi[buf], c)) return;
                        tc_fence_after();
                    }
                    warp_mma_ts(lead, tmem + 256 + o * C::kOStep, tmem + C::kPCol + buf * C::kPStep + kk * 8,
                                sdesc_add(db, kk * 2048), idPV, (first && kk == 0) ? 0u : 1u);
                }
            };
            while (ok) {
                const int slot = it & 1;
                if (!wait(sm.piece_full[slot], it >> 1)) break;
                const int pb = __shfl_sync(0xffffffffu, sm.piece[slot].b, 0);
                const int n = __shfl_sync(0xffffffffu, sm.piece[slot].n, 0);
                const int nt = __shfl_sync(0xffffffffu, sm.piece[slot].ntok, 0);
                if (lane == 0) mbar_arrive(smem_u32(&sm.piece_empty[slot]));
                __syncwarp();
                if (pb < 0) break;
                if (!wait(sm.q_full, it)) break;
                if constexpr (PAIR) {
                    // Each stream's next scores right behind its PV, so that it does not wait
                    // for the other's softmax: S0 S1 | PV0 S0 PV1 S1 | PV0 S0 ...
                    const int ns = nt > p.tile_tokens ? 2 : 1;
                    for (int j = -1; j < n && ok; ++j) {
                        const int fv = f + 2 * j + 1, fk = fv + 1;  // V(j), K(j + 1)
                        const bool v_in = j >= 0 && there(fv), k_in = j + 1 < n && there(fk);
                        for (int s = 0; s < ns && ok; ++s) {
                            if (j >= 0) {
                                // (stream 0 mends V before its P is ready, so both may follow it)
                                if (!wait(sm.p_full[s], cnt[s])) break;
                                if (s == 0 && !v_in && !wait(sm.full[fv % S], fv / S)) break;
                                if (j == 0 && done[s] > 0 && !wait(sm.o_free[s], done[s] - 1)) break;
                                issue_pv(fv, s, s, cnt[s], j == 0);
                                if (!ok) break;
                                if (s == ns - 1) warp_mma_commit(lead, smem_u32(&sm.empty[fv % S]));
                                warp_mma_commit(lead, smem_u32(&sm.o_done[s]));
                                ++cnt[s];
                            }
                            if (j + 1 < n) {
                                if (s == 0 && !k_in && !wait(sm.full[fk % S], fk / S)) break;
                                // S_s is free once the P written over it has been read
                                if (!C::kSepP && cnt[s] > 0 && !wait(sm.o_done[s], cnt[s] - 1)) break;
                                issue_s(fk, s, s);
                                warp_mma_commit(lead, smem_u32(&sm.s_full[s]));
                                if (s == ns - 1) {
                                    warp_mma_commit(lead, smem_u32(&sm.empty[fk % S]));
                                    if (j + 1 == n - 1) warp_mma_commit(lead, smem_u32(&sm.q_empty));
                                }
                            }
                        }
                    }
                    if (!ok) break;
                    for (int s = 0; s < ns; ++s) ++done[s];
                } else {
                    // S runs one tile ahead: S(0), S(1), PV(0), S(2), PV(1), ...
                    bool k_in = false;
                    auto do_s = [&](int j) {
                        const int fk = f + fifo_k<false>(j), bf = j & 1;
                        if (!k_in && !wait(sm.full[fk % S], fk / S)) return;
                        k_in = false;
                        // the buffer's P of two tiles ago has been read
                        const int c = cnt[bf] + (j >> 1);
                        if (!C::kSepP && c > 0 && !wait(sm.o_done[bf], c - 1)) return;
                        issue_s(fk, bf, 0);
                        warp_mma_commit(lead, smem_u32(&sm.empty[fk % S]));
                        warp_mma_commit(lead, smem_u32(&sm.s_full[bf]));
                        if (j == n - 1) warp_mma_commit(lead, smem_u32(&sm.q_empty));
                    };
                    for (int j = -2; j < n && ok; ++j) {
                        if (j >= 0) {
                            const int fv = f + fifo_v<false>(j, n), bf = j & 1;
                            const int c = cnt[bf] + (j >> 1);
                            const bool v_in = there(fv);
                            k_in = j + 2 < n && there(f + fifo_k<false>(j + 2));
                            if (!wait(sm.p_full[bf], c)) break;
                            if (!v_in && !wait(sm.full[fv % S], fv / S)) break;
                            if (j == 0 && it > 0 && !wait(sm.o_free[0], it - 1)) break;
                            issue_pv(fv, bf, C::kStreams == 2 ? bf : 0, c,
                                     C::kStreams == 2 ? j < 2 : j == 0);
                            if (!ok) break;
                            warp_mma_commit(lead, smem_u32(&sm.empty[fv % S]));
                            warp_mma_commit(lead, smem_u32(&sm.o_done[bf]));
                        }
                        if (j + 2 < n) do_s(j + 2);
                    }
                    cnt[0] += (n + 1) / 2;
                    cnt[1] += n / 2;
                }
                if (!ok) break;
                f += 2 * n;
                ++it;
            }
            warp_mma_commit(lead, smem_u32(&sm.drain));
            mbar_wait(smem_u32(&sm.drain), 0, &sm.zero);
        }
    } else if (warp >= 4) {
        // ------------------------------------------------------------ softmax and epilogue
        setmaxnreg_inc<kManyRegs>();
        const int w = (warp - 4) >> 2;          // stream
        const int q4 = warp & 3;                // TMEM lane quarter
        const int at = q4 * 32 + lane;          // lane of TMEM
        const int row = FEW ? lane : at;
        const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
        const int row_tok = row / p.group, row_head = row - row_tok * p.group;
        const bool row_used = row_tok < p.tile_tokens;
        int it = 0, f = 0, cnt[2] = {0, 0};
        bool ok = true;
        if constexpr (FEW) {  // a lane's P of the other quarters' keys: none, for good
            const uint32_t none[16] = {};
            for (int i = 0; i < BN / 2; i += 16)
                tmem_st16(tmem + lane_off + C::kPCol + w * C::kPStep + i, none);
            tmem_st_wait();
        }
        while (ok) {
            const int slot = it & 1;
            if (!(ok = warp_wait(smem_u32(&sm.piece_full[slot]), (it >> 1) & 1, stop, status))) break;
            const Piece x = sm.piece[slot];
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.piece_empty[slot]));
            if (x.b < 0) break;
            const int tok_first = PAIR ? w * p.tile_tokens : 0;  // of this stream's rows
            const int ntok = min(p.tile_tokens, x.ntok - tok_first);  // <= 0: no rows
            const bool valid = row_used && row_tok < ntok;
            const bool warp_valid = __any_sync(0xffffffffu, valid);
            const int trow = x.trow0 + tok_first + row_tok;  // index in the sequence
            const size_t tok = (size_t)x.tok0 + tok_first + row_tok;
            // no key from `limit` on is visible; without a mask all before it are
            const int limit = p.mask ? x.len : min(x.len, x.ctx + trow + 1);
            const Sight sight(p, x);
            const uint32_t* words = p.mask
                ? reinterpret_cast<const uint32_t*>(p.mask) + (valid ? tok : 0) * (2 * (size_t)p.words)
                : nullptr;
            const int from = window_from(p, x, words, trow, valid ? tok : 0);
            const bool active = PAIR ? ntok > 0 : (C::kStreams == 2 || w == 0);
            const int step = PAIR || C::kStreams == 1 ? 1 : 2;
            float m_ref = -INFINITY, l = 0.f;
            bool first = true;  // this stream has had no tile yet
            if (active) {
                for (int j = PAIR || C::kStreams == 1 ? 0 : w; j < x.n; j += step) {
                    const int buf = PAIR ? w : j & 1;
                    const int c = PAIR ? cnt[w] + j : cnt[buf] + (j >> 1);
                    const int key0 = x.tile_key(j, BN);
                    if (!(ok = warp_wait(smem_u32(&sm.s_full[buf]), c & 1, stop, status))) break;
                    tc_fence_after();
                    const uint32_t s_at = tmem + lane_off + buf * 128;
                    const uint32_t p_at = tmem + lane_off + C::kPCol + buf * C::kPStep;
                    const bool ragged = sight.ragged(key0, BN);
                    // V rows past the length are whatever the page held, and a drafted V
                    // may be anything: both are mended before P is handed over (before the
                    // scores take up the registers; only once S(j) is there, so that the stage's
                    // barrier is at most one phase behind).
                    if (ragged && (!PAIR || w == 0)) {
                        const int fv = f + fifo_v<PAIR>(j, x.n);
                        if (!(ok = warp_wait(smem_u32(&sm.full[fv % S]), (fv / S) & 1, stop, status)))
                            break;
                        if (at < BN && sight.hidden_from_some(key0 + at)) {
                            uint8_t* rest = sm.kv[fv % S] + at * 128;
                            const bool past = sight.hidden_from_all(key0 + at, x.len);
#pragma unroll 1
                            for (int cb = 0; cb < C::kCols; ++cb, rest += BN * 128) {
                                // (chunks in an order of the row's own, which spreads the banks)
                                uint4* line = reinterpret_cast<uint4*>(rest);
                                uint4 v[8];
                                uint32_t bad = 0;
#pragma unroll
                                for (int e = 0; e < 8; ++e) v[e] = line[(e + at) & 7];
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    bad |= not_finite(v[e].x) | not_finite(v[e].y) | not_finite(v[e].z) |
                                           not_finite(v[e].w);
                                if (past) {
#pragma unroll
                                    for (int e = 0; e < 8; ++e) line[(e + at) & 7] = make_uint4(0u, 0u, 0u, 0u);
                                } else if (bad) {
                                    *reinterpret_cast<volatile int*>(&sm.poison) = 1;
                                    uint16_t* value = reinterpret_cast<uint16_t*>(rest);
                                    for (int e = 0; e < 64; ++e)
                                        if (!finite_bf16(value[e])) value[e] = 0;
                                }
                            }
                            fence_proxy_async_smem();
                        }
                        __syncwarp();
                    }
                    float alpha = 1.f, neg = 0.f;
                    bool need = false;
                    // the reference moves when the row maximum outgrows it
                    auto take_max = [&](float mx) {
                        if (first) {
                            m_ref = mx;
                        } else if (mx > m_ref + kRescale) {
                            need = true;
                            alpha = ex2_approx(m_ref - mx);
                            m_ref = mx;
                            l *= alpha;
                        }
                        neg = m_ref == -INFINITY ? 0.f : -m_ref;
                    };
                    auto key_bits = [&](int kb) {
                        uint32_t bits = p.mask ? mask_bits(words, 2 * p.words, kb - x.ctx) : 0xffffffffu;
                        const int room = limit - kb;
                        if (room <= 0) bits = 0;
                        else if (room < 32) bits &= (1u << room) - 1u;
                        if constexpr (kWin) bits &= window_bits(kb, from, sight.sinks);
                        return bits;
                    };
                    float s[FEW ? 32 : C::kWhole ? BN : 1];
                    if constexpr (FEW) {
                        // this quarter's 32 keys
                        if (warp_valid) {
                            uint32_t r[32];
                            tmem_ld32(s_at + q4 * 32, r);
                            tmem_ld_wait();
                            const uint32_t bits = ragged ? key_bits(key0 + q4 * 32) : 0xffffffffu;
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                s[i] = (bits >> i) & 1u ? __uint_as_float(r[i]) : -INFINITY;
                            float m4[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                float m = fmaxf(s[k], s[28 + k]);
#pragma unroll
                                for (int i = 4; i < 28; i += 8) m = fmax3(m, s[i + k], s[i + 4 + k]);
                                m4[k] = m;
                            }
                            take_max(fmax3(fmaxf(m4[0], m4[1]), m4[2], m4[3]) * p.scale_log2);
                        }
                    } else if constexpr (C::kWhole) {
                        // the whole row in registers, all loads in flight
                        if (warp_valid) {
                            uint32_t r[BN / 32][32];
#pragma unroll
                            for (int i = 0; i < BN / 32; ++i) tmem_ld32(s_at + i * 32, r[i]);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < BN; ++i) s[i] = __uint_as_float(r[i / 32][i % 32]);
                            if (ragged) {
#pragma unroll
                                for (int i = 0; i < BN / 32; ++i) {
                                    const uint32_t bits = key_bits(key0 + i * 32);
#pragma unroll
                                    for (int e = 0; e < 32; ++e)
                                        if (!((bits >> e) & 1u)) s[i * 32 + e] = -INFINITY;
                                }
                            }
                            float m8[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                float m = fmax3(s[k], s[8 + k], s[16 + k]);
#pragma unroll
                                for (int i = 24; i + 8 < BN; i += 16) m = fmax3(m, s[i + k], s[i + 8 + k]);
                                m8[k] = fmaxf(m, s[BN - 8 + k]);
                            }
                            take_max(fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]),
                                           fmaxf(m8[6], m8[7])) * p.scale_log2);
                        }
                    } else if (warp_valid) {
                        // memory-bound, and often only a few tiles in a CTA: S is read twice in
                        // loops of 64 columns, whose code is a quarter of the unrolled form's (a
                        // CTA's first pass through it waits for every instruction line)
                        if (ragged) {
#pragma unroll 1
                            for (int i = 0; i < BN / 32; ++i) {
                                const uint32_t bits = key_bits(key0 + i * 32);
                                uint32_t r[32], lo[16], hi[16];
                                tmem_ld32(s_at + i * 32, r);
                                tmem_ld_wait();
#pragma unroll
                                for (int e = 0; e < 16; ++e) {
                                    lo[e] = (bits >> e) & 1u ? r[e] : 0xff800000u;
                                    hi[e] = (bits >> (16 + e)) & 1u ? r[16 + e] : 0xff800000u;
                                }
                                tmem_st16(s_at + i * 32, lo);
                                tmem_st16(s_at + i * 32 + 16, hi);
                            }
                            tmem_st_wait();
                        }
                        float mx = -INFINITY;
#pragma unroll 1
                        for (int i = 0; i < BN; i += 64) {
                            uint32_t r0[32], r1[32];
                            tmem_ld32(s_at + i, r0);
                            tmem_ld32(s_at + i + 32, r1);
                            tmem_ld_wait();
                            float m4[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                float m = fmaxf(__uint_as_float(r0[k]), __uint_as_float(r1[k]));
#pragma unroll
                                for (int e = 4; e < 32; e += 4)
                                    m = fmax3(m, __uint_as_float(r0[e + k]), __uint_as_float(r1[e + k]));
                                m4[k] = m;
                            }
                            mx = fmax3(mx, fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                        }
                        take_max(mx * p.scale_log2);
                    }
                    first = false;
                    // P in columns of its own is free once the last PV has read it
                    if (C::kSepP && c > 0) {
                        if (!(ok = warp_wait(smem_u32(&sm.o_done[buf]), (c - 1) & 1, stop, status))) break;
                        tc_fence_after();
                    }
                    // O~ is stable when its last PV is done: with two streams that has
                    // been waited for, here or before S(j); with one, PV(j - 1) may still run.
                    if (__any_sync(0xffffffffu, need)) {
                        const int o = PAIR ? w : (C::kStreams == 2 ? buf : 0);
                        if (C::kStreams == 1) {
                            const int pb = (j - 1) & 1;
                            if (!(ok = warp_wait(smem_u32(&sm.o_done[pb]),
                                                 (cnt[pb] + ((j - 1) >> 1)) & 1, stop, status)))
                                break;
                            tc_fence_after();
                        }
                        const uint32_t o_at = tmem + lane_off + 256 + o * C::kOStep;
#pragma unroll 1
                        for (int cc = 0; cc < DR / 32; ++cc) {
                            uint32_t ov[32];
                            tmem_ld32(o_at + cc * 32, ov);
                            tmem_ld_wait();
                            uint32_t lo[16], hi[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                lo[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
                                hi[i] = __float_as_uint(__uint_as_float(ov[16 + i]) * alpha);
                            }
                            tmem_st16(o_at + cc * 32, lo);
                            tmem_st16(o_at + cc * 32 + 16, hi);
                        }
                    }
                    uint64_t acc[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
                    if constexpr (FEW) {
                        if (warp_valid) {
                            uint32_t pk[16];
                            exp_chunk(s, p.scale_log2, neg, acc, pk);
                            tmem_st16(p_at + q4 * 16, pk);
                            tmem_st_wait();
                        }
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_u32(&sm.p_full[buf]));
                    } else if constexpr (C::kWhole) {
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            if (warp_valid) {
#pragma unroll
                                for (int cc = hf * (BN / 64); cc < (hf + 1) * (BN / 64); ++cc) {
                                    uint32_t pk[16];
                                    exp_chunk(s + cc * 32, p.scale_log2, neg, acc, pk);
                                    tmem_st16(p_at + cc * 16, pk);
                                }
                                tmem_st_wait();
                            }
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(smem_u32(hf == 0 ? &sm.p_full[buf] : &sm.p_hi[buf]));
                        }
                    } else {
                        // (a chunk's P lies over scores that have been read)
#pragma unroll 1
                        for (int hf = 0; hf < 2; ++hf) {
                            if (warp_valid) {
                                constexpr int W = BN / 64;  // chunks of a half
                                uint32_t r[W][32];
#pragma unroll
                                for (int c2 = 0; c2 < W; ++c2) tmem_ld32(s_at + (hf * W + c2) * 32, r[c2]);
                                tmem_ld_wait();
#pragma unroll
                                for (int c2 = 0; c2 < W; ++c2) {
                                    uint32_t pk[16];
                                    exp_chunk(reinterpret_cast<const float*>(r[c2]), p.scale_log2, neg,
                                              acc, pk);
                                    tmem_st16(p_at + (hf * W + c2) * 16, pk);
                                }
                                tmem_st_wait();
                            }
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(smem_u32(hf == 0 ? &sm.p_full[buf] : &sm.p_hi[buf]));
                        }
                    }
                    if (warp_valid) {
                        float a0, a1, b0, b1;
                        f2_unpack(acc[0], a0, a1);
                        f2_unpack(acc[1], b0, b1);
                        l += (a0 + a1) + (b0 + b1);
                    }
                }
            }
            if (!ok) break;

            // ---- epilogue
            float w0 = 1.f, w1 = 0.f;      // weights of the two accumulators
            const bool two = !PAIR && C::kStreams == 2 && x.n > 1;
            if constexpr (!PAIR) {
                // both warpgroups need both streams' statistics: each then stores
                // every other 32 columns
                auto& st = sm.stats[it & 1];
                if (w < C::kStreams) {
                    st[w][0][at] = m_ref;
                    st[w][1][at] = l;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sm.stat_full));
                if (!(ok = warp_wait(smem_u32(&sm.stat_full), it & 1, stop, status))) break;
                m_ref = st[0][0][at];
                l = st[0][1][at];
                if constexpr (FEW) {
                    // this lane's weights, and the row's sums over quarters and streams
                    const float m0 = m_ref, m1 = st[1][0][at];
                    for (int i = 0; i < (two ? 2 : 1); ++i)
                        for (int k = 0; k < 4; ++k) m_ref = fmaxf(m_ref, st[i][0][k * 32 + lane]);
                    const float base = m_ref == -INFINITY ? 0.f : m_ref;
                    l = 0.f;
                    for (int i = 0; i < (two ? 2 : 1); ++i)
                        for (int k = 0; k < 4; ++k)
                            l += st[i][1][k * 32 + lane] * ex2_approx(st[i][0][k * 32 + lane] - base);
                    w0 = ex2_approx(m0 - base);
                    if (two) w1 = ex2_approx(m1 - base);
                } else if (two) {
                    const float m1 = st[1][0][at], l1 = st[1][1][at];
                    const float m = fmaxf(m_ref, m1), base = m == -INFINITY ? 0.f : m;
                    w0 = ex2_approx(m_ref - base);
                    w1 = ex2_approx(m1 - base);
                    l = l * w0 + l1 * w1;
                    m_ref = m;
                }
                // the last PV of each buffer
                const int n0 = (x.n + 1) / 2, n1 = x.n / 2;
                if (!(ok = warp_wait(smem_u32(&sm.o_done[0]), (cnt[0] + n0 - 1) & 1, stop, status)))
                    break;
                if (x.n > 1 &&
                    !(ok = warp_wait(smem_u32(&sm.o_done[1]), (cnt[1] + n1 - 1) & 1, stop, status)))
                    break;
                cnt[0] += n0;
                cnt[1] += n1;
            } else if (active) {
                if (!(ok = warp_wait(smem_u32(&sm.o_done[w]), (cnt[w] + x.n - 1) & 1, stop, status)))
                    break;
                cnt[w] += x.n;
            }
            tc_fence_after();
            if (active || !PAIR) {
                const int poison = *reinterpret_cast<volatile int*>(&sm.poison);
                const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
                const int head = x.h * p.group + row_head;
                if (valid && (PAIR || w == 0) && (!FEW || q4 == 0)) {
                    if (x.part < 0) {
                        p.lse[(size_t)head * p.T + tok] = (m_ref + __log2f(l)) * 0.69314718055994531f;
                    } else {
                        float* st = p.part_stats + ((size_t)x.part * p.part_rows +
                                                    (PAIR ? w * 128 : 0) + row) * 2;
                        st[0] = m_ref;
                        st[1] = l;
                    }
                }
                if (warp_valid) {
#pragma unroll 1
                    for (int cc = PAIR ? 0 : w; cc < DR / 32; cc += PAIR ? 1 : 2) {
                        float o[32];
                        {
                            uint32_t ov[32];
                            tmem_ld32(tmem + lane_off + 256 + (PAIR ? w * C::kOStep : 0) + cc * 32, ov);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = __uint_as_float(ov[i]) * w0;
                        }
                        if (two) {
                            uint32_t ov[32];
                            tmem_ld32(tmem + lane_off + 256 + C::kOStep + cc * 32, ov);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                o[i] = fmaf(__uint_as_float(ov[i]), w1, o[i]);
                        }
                        if (x.part < 0) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] *= inv;
                        }
                        if constexpr (FEW) {
                            // The quarters' O add up through shared memory; each warp then
                            // stores eight of the rows.  (All have read the last piece's: they
                            // have brought this piece's statistics.)
                            float4* line = reinterpret_cast<float4*>(sm.x[w][at]);
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                line[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                            __syncwarp();
                            if (lane == 0) mbar_arrive(smem_u32(&sm.x_full[w]));
                            if (!(ok = warp_wait(smem_u32(&sm.x_full[w]), it & 1, stop, status))) break;
                            store_few<DR, BN>(p, x, sm.x[w], sm.stats[it & 1], two, poison, sight, q4, cc);
                            continue;
                        }
                        if (poison && valid) {
                            // a visible drafted V that is not finite: its weight is
                            // positive, so it adds itself
                            const int ps = p.cache.page_size;
                            const int skip = kWin ? 0 : max(0, sight.open - x.tile_key(0, BN));
                            for (int i = skip; i < x.n * BN; ++i) {
                                const int key = x.tile_key(i / BN, BN) + i % BN;
                                if (key >= limit) break;
                                if (kWin && (!sight.hidden_from_some(key) ||
                                             (key < from && key >= sight.sinks)))
                                    continue;
                                if (p.mask && !(mask_bits(words, 2 * p.words, key - x.ctx) & 1u))
                                    continue;
                                const int page = p.cache.table[(long long)x.slot * p.cache.max_pages +
                                                               key / ps];
                                if (page < 0 || page >= p.cache.pages) continue;
                                const uint16_t* v =
                                    static_cast<const uint16_t*>(p.cache.v) +
                                    ((((long long)p.layer * p.cache.pages + page) * p.cache.heads +
                                      x.h) * ps + key % ps) * DR + cc * 32;
#pragma unroll
                                for (int i = 0; i < 32; ++i) {
                                    const uint32_t u = v[i];
                                    if (!finite_bf16(u)) o[i] += __uint_as_float(u << 16);
                                }
                            }
                        }
                        if (valid && x.part < 0) {
                            uint4* dst = reinterpret_cast<uint4*>(
                                static_cast<__nv_bfloat16*>(p.o) + (tok * p.Hq + head) * DR + cc * 32);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                dst[i] = make_uint4(pack_bf16x2(o[8 * i], o[8 * i + 1]),
                                                    pack_bf16x2(o[8 * i + 2], o[8 * i + 3]),
                                                    pack_bf16x2(o[8 * i + 4], o[8 * i + 5]),
                                                    pack_bf16x2(o[8 * i + 6], o[8 * i + 7]));
                        } else if (valid) {
                            // many rows: columns in fours, rows next to one another, so that a
                            // warp's stores are contiguous
                            const int step = p.fused ? 1 : p.part_rows;
                            const int r = (PAIR ? w * 128 : 0) + row;
                            float4* dst = reinterpret_cast<float4*>(p.part_o) +
                                          (size_t)x.part * p.part_rows * (DR / 4) +
                                          (p.fused ? r * (DR / 4) + cc * 8 : r + cc * 8 * step);
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                dst[i * step] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                        }
                    }
                }
                if (FEW && !ok) break;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_u32(&sm.o_free[PAIR ? w : 0]));
                    if (!PAIR && it == 0) mbar_arrive(smem_u32(&sm.stored));
                }
            }
            f += 2 * x.n;
            ++it;
        }
    } else {
        // ------------------------------------------------------------ warp 2
        setmaxnreg_dec<kFewRegs>();
        if (p.zero_rest && p.cu) {
            // Tokens before all boundaries and behind all of them.  (What this warp runs
            // moves the loops of the others in the instruction cache: with the search for
            // tokens between odd boundaries here too, 2048-token chunks over 4-6k keys took
            // 1-4% longer.)
            int skip = p.T, used = 0;
#pragma unroll 1
            for (int i = lane; i <= p.B; i += 32) {
                skip = min(skip, p.cu[i]);
                used = max(used, p.cu[i]);
            }
            skip = max(__reduce_min_sync(0xffffffffu, skip), 0);
            used = min(__reduce_max_sync(0xffffffffu, used), p.T);
            const long long step = (long long)gridDim.x * 32;
            const long long at = (long long)blockIdx.x * 32 + lane;
            auto clear = [&](int t0, int n) {
                const long long rows = (long long)n * p.Hq;
                uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) +
                                                    (long long)t0 * p.Hq * DR);
                for (long long i = at; i < rows * (DR / 8); i += step) o[i] = make_uint4(0u, 0u, 0u, 0u);
                for (long long i = at; i < rows; i += step)
                    p.lse[(i / n) * p.T + t0 + i % n] = -INFINITY;
            };
            clear(0, skip);
            if (used < p.T) clear(used, p.T - used);
            if constexpr (!PAIR) {  // (those between: the join kernel's, where there is one)
                if (p.fused) clear_unowned<DR>(p, blockIdx.x, gridDim.x);
            }
        }
        if constexpr (!PAIR) {
            // An item's end is brought while the CTA goes on, so that its beginning, which
            // a CTA finishes last, is what completes it nearly always: a CTA then joins one
            // item at its end, not up to two.
            if (p.fused && warp_wait(smem_u32(&sm.begun), 0, stop, status) && sm.early &&
                warp_wait(smem_u32(&sm.stored), 0, stop, status) && lane == 0)
                sm.join_last[0] = bring(p, sm.shared[0]);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if constexpr (!PAIR) {
        // Whoever brings an item's last partial joins them.
        const int n = p.fused && !sm.abort_flag ? sm.n_shared : 0;
        if (n == 0) return;
        if (threadIdx.x >= sm.early && threadIdx.x < n)
            sm.join_last[threadIdx.x] = bring(p, sm.shared[threadIdx.x]);
        __syncthreads();
        for (int r = warp; r < n * p.part_rows; r += kThreads / 32) {
            const int i = r >= p.part_rows, row = r - i * p.part_rows;
            const Piece& x = sm.shared[i];
            const int rt = row / p.group;
            if (sm.join_last[i] && rt < x.ntok)
                join_row<DR>(p, row, x.first_cta, x.last_cta - x.first_cta + 1, (size_t)x.tok0 + rt,
                             x.h * p.group + row - rt * p.group);
        }
    }
}

// Joins the partials of every item that more than one CTA worked on: the CTA
// whose first piece ends the item left (first CTA, token, tokens, head) in
// meta.  A thread takes eight columns of a row, the rows of a warp are
// neighbours; partials are added in the CTAs' order, rescaled as the maximum
// moves.  Mostly two or three partials, and latency: more blocks to an SM count
// for as much as more loads in flight (2048-token chunks, 2 / 3 / 4 / 8 in flight:
// 338.8 / 338.9 / 340.3 / 344 us; 19 partials of 128 rows: 39.4 / 38.8 / 38.4 / 38.8).
template <int DR>
__global__ void __launch_bounds__(256, 4) tree_join_kernel(const __grid_constant__ TreeParams p) {
    pdl_begin();
    if (p.clear_odd && blockIdx.y == gridDim.y - 1) {
        clear_unowned<DR>(p, blockIdx.x * 8 + warp_id(), gridDim.x * 8);
        return;
    }
    const int4 own = p.meta[blockIdx.x];
    const int e = blockIdx.y * 256 + threadIdx.x;
    const int c8 = e / p.part_rows, slot_row = e - c8 * p.part_rows;
    const int stream = slot_row >> 7, row = slot_row & 127;
    const int row_tok = row / p.group;
    const int t = stream * p.tile_tokens + row_tok;
    if (own.x < 0 || c8 >= DR / 8 || row_tok >= p.tile_tokens || t >= own.z) return;
    constexpr int R = 3;
    const int n = (int)blockIdx.x - own.x + 1;
    float m = -INFINITY, l = 0.f, acc[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] = 0.f;
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += R) {
        float2 st[R];
        float4 x[R][2];
#pragma unroll
        for (int u = 0; u < R; ++u) {
            st[u] = make_float2(-INFINITY, 0.f);
            x[u][0] = x[u][1] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i0 + u < n) {  // slot 2c + 1 of the first CTA, 2c of the others
                const size_t slot = 2 * (own.x + i0 + u) + (i0 + u == 0);
                const float4* at = reinterpret_cast<const float4*>(p.part_o) +
                                   (slot * (DR / 4) + 2 * c8) * p.part_rows + slot_row;
                st[u] = __ldcg(reinterpret_cast<const float2*>(p.part_stats) + slot * p.part_rows + slot_row);
                x[u][0] = __ldcg(at);
                x[u][1] = __ldcg(at + p.part_rows);
            }
        }
        float top = m;
#pragma unroll
        for (int u = 0; u < R; ++u) top = fmaxf(top, st[u].x);
        const float base = top == -INFINITY ? 0.f : top, keep = ex2_approx(m - base);
        m = top;
        l *= keep;
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] *= keep;
#pragma unroll
        for (int u = 0; u < R; ++u) {
            if (i0 + u >= n) continue;
            const float w = ex2_approx(st[u].x - base);
            l = fmaf(st[u].y, w, l);
            acc[0] = fmaf(x[u][0].x, w, acc[0]); acc[1] = fmaf(x[u][0].y, w, acc[1]);
            acc[2] = fmaf(x[u][0].z, w, acc[2]); acc[3] = fmaf(x[u][0].w, w, acc[3]);
            acc[4] = fmaf(x[u][1].x, w, acc[4]); acc[5] = fmaf(x[u][1].y, w, acc[5]);
            acc[6] = fmaf(x[u][1].z, w, acc[6]); acc[7] = fmaf(x[u][1].w, w, acc[7]);
        }
    }
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    const size_t tok = (size_t)own.y + t;
    const int head = own.w * p.group + row - row_tok * p.group;
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + (tok * p.Hq + head) * DR + c8 * 8) =
        make_uint4(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv),
                   pack_bf16x2(acc[4] * inv, acc[5] * inv), pack_bf16x2(acc[6] * inv, acc[7] * inv));
    if (c8 == 0) p.lse[(size_t)head * p.T + tok] = (m + __log2f(l)) * 0.69314718055994531f;
}

template <int D, int DR, bool PAIR, bool FEW = false>
cudaError_t launch_t(const TreeParams& p, int ctas, cudaStream_t stream) {
    auto kern = tree_kernel<D, DR, PAIR, FEW>;
    constexpr size_t smem = smem_bytes<D, PAIR, FEW>();
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3(ctas), dim3(kThreads), smem, stream, p);
    if (e != cudaSuccess || p.fused) return e;
    const int slices = cdiv(p.part_rows * (DR / 8), 256) + p.clear_odd;
    return launch_pdl(tree_join_kernel<DR>, dim3(ctas, slices), dim3(256), 0, stream, p);
}

cudaError_t launch_d(const TreeParams& p, bool pair, int ctas, cudaStream_t strm) {
    const int d = p.cache.d;
    if (d == 128)
        return pair ? launch_t<128, 128, true>(p, ctas, strm) : launch_t<128, 128, false>(p, ctas, strm);
    if (d == 96)
        return pair ? launch_t<128, 96, true>(p, ctas, strm) : launch_t<128, 96, false>(p, ctas, strm);
    if (d == 64)
        return pair      ? launch_t<64, 64, true>(p, ctas, strm)
               : p.fused ? launch_t<64, 64, false, true>(p, ctas, strm)
                         : launch_t<64, 64, false>(p, ctas, strm);
    if (d == 192) return launch_t<192, 192, false>(p, ctas, strm);
    return launch_t<256, 256, false>(p, ctas, strm);
}

#ifdef FA_WINDOW

}  // namespace

cudaError_t launch_tree_window(const TreeParams& p, bool pair, int ctas, cudaStream_t stream) {
    return launch_d(p, pair, ctas, stream);
}

}  // namespace fa

#else

// Ancestor bits of drafted trees: token t of a sequence sees itself, its
// parent, its parent's parent, ... up to a token whose parent is -1 (or is not
// an earlier token of the sequence).  A thread a row.
__global__ void tree_mask_kernel(const int* parents, const int* cu, int B, int N, int T, int words,
                                 unsigned long long* mask) {
    pdl_begin();
    const int t = blockIdx.x * blockDim.x + threadIdx.x;
    if (t >= T) return;
    unsigned long long* row = mask + (size_t)t * words;
    for (int i = 0; i < words; ++i) row[i] = 0ull;
    const int b = seq_of_token(cu, B, N, t);
    if (b < 0) return;
    const int t0 = cu ? max(cu[b], 0) : b * N;
    int j = t - t0;
    while (j >= 0) {
        if (j < words * 64) row[j >> 6] |= 1ull << (j & 63);
        const int up = parents[t0 + j];
        if (up >= j) break;
        j = up;
    }
}

// The window among the call's own tokens: depth[t] is the number of others that token t names,
// and of these it keeps in `out` those less than `window` above it, and those whose position is
// one of the first `sinks`.  A thread a row, then a thread a word of one.
__global__ void tree_depth_kernel(const uint32_t* mask, const int* cu, int B, int N, int T, int words, int* depth) {
    pdl_begin();
    const int t = blockIdx.x * blockDim.x + threadIdx.x;
    if (t >= T) return;
    const int b = seq_of_token(cu, B, N, t);
    int d = 0;
    if (b >= 0) {
        const SeqRange r = seq_range(cu, N, T, b);
        if (t - r.t0 < r.n) d = named_others(mask + (size_t)t * 2 * words, words, r.n, t - r.t0);
    }
    depth[t] = d;
}
__global__ void tree_near_kernel(const fa_cache c, const int* slots, const unsigned long long* mask, const int* cu,
                                 int B, int N, int T, int words, int window, int sinks, unsigned long long* out,
                                 const int* depth) {
    pdl_begin();
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= (long long)T * words) return;
    const int t = (int)(i / words), first = (int)(i - (long long)t * words) * 64;
    const int b = seq_of_token(cu, B, N, t);
    unsigned long long left = 0;
    if (b >= 0) {
        const SeqRange r = seq_range(cu, N, T, b);
        const int slot = slots[b];
        const int ctx = slot >= 0 && slot < c.slots ? c.lengths[slot] - r.n : 0;
        unsigned long long bits = t - r.t0 < r.n ? mask[i] : 0;
        if (r.n - first < 64) bits &= r.n > first ? (1ull << (r.n - first)) - 1 : 0;
        const int mine = depth[t];
        for (; bits; bits &= bits - 1) {
            const int a = first + __ffsll((long long)bits) - 1, at = depth[r.t0 + a];
            if (r.t0 + a == t || (long long)mine - at < window || (long long)ctx + at < sinks)
                left |= bits & -bits;
        }
    }
    out[i] = left;
}

// Row tiles: as many whole tokens (of group rows each) as 128 rows hold; more
// rows than that take them in pairs where TMEM has two accumulators.
struct Tiles {
    int tokens, rows;
    bool pair;
};
Tiles row_tiles(int group, int N, int d) {
    Tiles t;
    t.tokens = 128 / group < N ? 128 / group : N;
    t.pair = d <= 128 && N > 128 / group;
    t.rows = t.pair ? 256 : t.tokens * group;
    return t;
}

// Items of up to this many rows are joined by the CTA that finishes last:
// one launch less (~5 us of the caller's time, and as much on the GPU), while
// more rows would leave one CTA too much to read.
constexpr int kFusedRows = 32;

struct TreeWs {
    size_t arrived, stats, o, bytes;
};
TreeWs tree_ws(int rows, int d) {
    TreeWs w;
    w.arrived = align_up(kTreeMaxCtas * sizeof(int4), kAlign);
    w.stats = align_up(w.arrived + kTreeMaxCtas * sizeof(long long), kAlign);
    w.o = align_up(w.stats + (size_t)kTreeMaxCtas * 2 * rows * 2 * sizeof(float), kAlign);
    w.bytes = align_up(w.o + (size_t)kTreeMaxCtas * 2 * rows * d * sizeof(float), kAlign);
    return w;
}

// A number that no other call of this process has, and whose 56 bits what a
// workspace happens to hold does not repeat.
unsigned long long next_call() {
    static std::atomic<unsigned long long> last{0};
    unsigned long long x = last.fetch_add(1, std::memory_order_relaxed) + 1;
    x *= 0x9E3779B97F4A7C15ull;  // (odd: different calls stay different)
    return x & 0x00FFFFFFFFFFFFFFull;
}

bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// window = 0: none.
fa_status tree_impl(const fa_cache* cache, int layer, const int* slots, int B, int N,
                    const int* cu_seqlens, int T, const void* q, int Hq, long long q_token_stride,
                    long long q_head_stride, const void* mask, int mask_words, void* o, float* lse,
                    float scale, int window, int sinks, const int* depth, int zero_rest,
                    void* workspace, size_t workspace_bytes, fa_stream_t stream) {
    const fa_status cs = check_cache(cache);
    if (cs != FA_OK) return cs;
    const int d = cache->d, Hkv = cache->heads;
    if (layer < 0 || layer >= cache->layers || B < 0 || N < 0 || T < 0 || Hq <= 0 || Hq % Hkv)
        return FA_ERR_INVALID_ARG;
    if (Hq / Hkv > 128 || Hq > 65535 || (long long)T * Hq * d > (1LL << 40) || B > kMostSequences)
        return FA_ERR_UNSUPPORTED;
    if (!(scale > 0.f) || !std::isfinite(scale)) return FA_ERR_UNSUPPORTED;
    if (!cu_seqlens && (long long)B * N != T) return FA_ERR_INVALID_ARG;
    if (mask && (mask_words <= 0 || (long long)mask_words * 64 < N)) return FA_ERR_INVALID_ARG;
    if (T == 0) return FA_OK;
    if ((B > 0 && !slots) || !q || !o || !lse || !workspace) return FA_ERR_INVALID_ARG;
    if (N == 0) N = 1;  // (a packed batch of empty sequences)
    if (!aligned(slots, 4) || !aligned(cu_seqlens, 4) || !aligned(q, 16) || !aligned(o, 16) ||
        !aligned(lse, 4) || !aligned(mask, 8) || !aligned(depth, 4) || !aligned(workspace, 16))
        return FA_ERR_INVALID_ARG;
    if (T == 1) q_token_stride = (long long)Hq * d;  // (a stride that is never taken)
    if (Hq == 1) q_head_stride = d;
    if (q_token_stride <= 0 || q_head_stride <= 0 || q_token_stride % 8 || q_head_stride % 8 ||
        q_token_stride >= (1LL << 38) || q_head_stride >= (1LL << 31))
        return FA_ERR_INVALID_ARG;
    TreeParams p;
    std::memset(&p, 0, sizeof(p));
    p.group = Hq / Hkv;
    const Tiles tiles = row_tiles(p.group, N, d);
    const TreeWs ws = tree_ws(tiles.rows, d);
    if (workspace_bytes < ws.bytes) return FA_ERR_INVALID_ARG;
    const int bn = d > 128 ? 64 : 128;
    if (!make_tree_maps(p, *cache, q, T, Hq, q_token_stride, q_head_stride, tiles.tokens, bn))
        return FA_ERR_CUDA;
    p.cache = *cache;
    p.slots = slots;
    p.cu = cu_seqlens;
    p.mask = mask;
    p.words = mask_words;
    p.o = o;
    p.lse = lse;
    char* base = static_cast<char*>(workspace);
    p.meta = reinterpret_cast<int4*>(base);
    p.arrived = reinterpret_cast<unsigned long long*>(base + ws.arrived);
    p.part_stats = reinterpret_cast<float*>(base + ws.stats);
    p.part_o = reinterpret_cast<float*>(base + ws.o);
    p.part_rows = tiles.rows;
    p.layer = layer;
    p.B = B; p.N = N; p.T = T; p.Hq = Hq;
    p.tile_tokens = tiles.tokens;
    // Two tiles a CTA at least: the streams alternate, and a join costs about as much
    // as a tile (one token over 501 keys, 16 heads: 15.8 -> 15.1 us).
    p.min_tiles = 2;
    p.page_shift = __builtin_ctz(cache->page_size);
    p.fused = !tiles.pair && tiles.rows <= kFusedRows;
    p.call = next_call();
    p.zero_rest = zero_rest ? 1 : 0;
    p.clear_odd = !p.fused && p.zero_rest && p.cu;
    // a window or sinks as long as any sequence hide nothing
    const long long room = (long long)cache->max_pages * cache->page_size;
    if (window > 0 && window < room && sinks < room) {
        p.window = window;
        p.sinks = sinks;
        p.depth = mask ? depth : nullptr;
    }
    p.scale_log2 = scale * 1.4426950408889634f;
    const int nsm = device_sms();
    if (nsm <= 0) return FA_ERR_CUDA;
    const int ctas = nsm < kTreeMaxCtas ? nsm : kTreeMaxCtas;
    cudaStream_t strm = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = p.window ? launch_tree_window(p, tiles.pair, ctas, strm)
                                   : launch_d(p, tiles.pair, ctas, strm);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_tree_workspace_size(int Hq, int Hkv, int N, int d) {
    if (Hq <= 0 || Hkv <= 0 || Hq % Hkv || Hq / Hkv > 128 || N <= 0 || d <= 0) return 0;
    return tree_ws(row_tiles(Hq / Hkv, N, d).rows, d).bytes;
}

fa_status fa_tree_mask(const int* parents, const int* cu_seqlens, int B, int N, int T, int words,
                       void* mask, fa_stream_t stream) {
    if (B < 0 || N < 0 || T < 0 || words <= 0 || (long long)words * 64 < N) return FA_ERR_INVALID_ARG;
    if (!cu_seqlens && (long long)B * N != T) return FA_ERR_INVALID_ARG;
    if (B > kMostSequences) return FA_ERR_UNSUPPORTED;
    if (T == 0) return FA_OK;
    if (!parents || !mask || !aligned(parents, 4) || !aligned(cu_seqlens, 4) || !aligned(mask, 8))
        return FA_ERR_INVALID_ARG;
    const cudaError_t e = launch_pdl(tree_mask_kernel, dim3(cdiv(T, 128)), dim3(128), 0,
                                     reinterpret_cast<cudaStream_t>(stream), parents, cu_seqlens, B,
                                     N, T, words, static_cast<unsigned long long*>(mask));
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_tree_fwd(const fa_cache* cache, int layer, const int* slots, int B, int N,
                      const int* cu_seqlens, int T, const void* q, int Hq, long long q_token_stride,
                      long long q_head_stride, const void* mask, int mask_words, void* o, float* lse,
                      float scale, int zero_rest, void* workspace, size_t workspace_bytes,
                      fa_stream_t stream) {
    return tree_impl(cache, layer, slots, B, N, cu_seqlens, T, q, Hq, q_token_stride, q_head_stride,
                     mask, mask_words, o, lse, scale, 0, 0, nullptr, zero_rest, workspace, workspace_bytes,
                     stream);
}

fa_status fa_tree_fwd_window(const fa_cache* cache, int layer, const int* slots, int B, int N,
                             const int* cu_seqlens, int T, const void* q, int Hq,
                             long long q_token_stride, long long q_head_stride, const void* mask,
                             int mask_words, void* o, float* lse, float scale, int window, int sinks,
                             int zero_rest, void* workspace, size_t workspace_bytes,
                             fa_stream_t stream) {
    if (window < 1 || sinks < 0) return FA_ERR_INVALID_ARG;
    return tree_impl(cache, layer, slots, B, N, cu_seqlens, T, q, Hq, q_token_stride, q_head_stride,
                     mask, mask_words, o, lse, scale, window, sinks, nullptr, zero_rest, workspace,
                     workspace_bytes, stream);
}

fa_status fa_tree_fwd_window_depth(const fa_cache* cache, int layer, const int* slots, int B, int N,
                                   const int* cu_seqlens, int T, const void* q, int Hq,
                                   long long q_token_stride, long long q_head_stride, const void* mask,
                                   int mask_words, const int* depth, void* o, float* lse, float scale,
                                   int window, int sinks, int zero_rest, void* workspace,
                                   size_t workspace_bytes, fa_stream_t stream) {
    if (window < 1 || sinks < 0 || (T > 0 && (!mask || !depth))) return FA_ERR_INVALID_ARG;
    return tree_impl(cache, layer, slots, B, N, cu_seqlens, T, q, Hq, q_token_stride, q_head_stride,
                     mask, mask_words, o, lse, scale, window, sinks, depth, zero_rest, workspace,
                     workspace_bytes, stream);
}

fa_status fa_tree_window_mask(const fa_cache* cache, const int* slots, int B, int N,
                              const int* cu_seqlens, int T, const void* mask, int words, int window,
                              int sinks, void* out, int* depth, fa_stream_t stream) {
    const fa_status cs = check_cache(cache);
    if (cs != FA_OK) return cs;
    if (B < 0 || N < 0 || T < 0 || words <= 0 || (long long)words * 64 < N || window < 1 || sinks < 0)
        return FA_ERR_INVALID_ARG;
    if (!cu_seqlens && (long long)B * N != T) return FA_ERR_INVALID_ARG;
    if (B > kMostSequences || (long long)T * words > (1LL << 38)) return FA_ERR_UNSUPPORTED;
    if (T == 0) return FA_OK;
    if ((B > 0 && !slots) || !mask || !out || !depth || !aligned(slots, 4) || !aligned(cu_seqlens, 4) ||
        !aligned(mask, 8) || !aligned(out, 8) || !aligned(depth, 4))
        return FA_ERR_INVALID_ARG;
    cudaStream_t strm = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = launch_pdl(tree_depth_kernel, dim3(cdiv(T, 128)), dim3(128), 0, strm,
                               static_cast<const uint32_t*>(mask), cu_seqlens, B, N, T, words, depth);
    if (e == cudaSuccess)
        e = launch_pdl(tree_near_kernel, dim3((unsigned)(((long long)T * words + 127) / 128)), dim3(128), 0, strm,
                       *cache, slots, static_cast<const unsigned long long*>(mask), cu_seqlens, B, N, T, words,
                       window, sinks, static_cast<unsigned long long*>(out), static_cast<const int*>(depth));
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"

#endif  // FA_WINDOW
