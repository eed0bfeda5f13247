// weights.cu -- the attention weight that each cached key receives from a call's
// queries, added up: for every slot, key/value head and key j
//   w_j += sum over the rows t and heads a of the group that see j of 2^(s_tj c - l_ta),
// with s = q.k, c = scale log2 e and l = LSE log2 e, which the attention over the cache
// has left.  It is what an eviction goes by.
//
// Bound: reading the keys once (decoding); with the last tokens of a prompt the sums over
// exponentials, ~1450 cycles of a warpgroup for 128 x 128 of them beside ~520 of the
// tensor core for their scores.
//
// The scores are computed transposed, S^T = K Q^T: a key is a lane of TMEM and a thread,
// which walks the query columns and adds up in registers, and no maximum is needed.  All
// sequences' and heads' key tiles stand in one line, each as long as its sequence has Q
// tiles, and every CTA takes an equal stretch; nothing has to be joined.
//   warp 0       K tiles through a ring of stages, a TMA box a page (or 128 keys of one)
//   warp 3       Q tiles and the LSE of their rows, for as long as a stretch of keys lasts
//   warp 1       MMA issuer
//   warps 4..7, 8..11  exponentials and sums
// Where one Q tile of up to 128 rows holds all (decoding), the two warpgroups take alternate
// key tiles, with two buffers of scores each, and the keys get all the shared memory.
// Otherwise (MANY) Q tiles have 256 rows (128 above d = 128): a 128 x 128 x 16 MMA reads
// 8 KB of operands in its 64 cycles, all that shared memory gives, and took 100.  Each
// warpgroup then adds up half of the columns of every tile, and the halves meet in shared
// memory.  More Q tiles than fit go through the stretch of keys in turns.
//
// Measured (GPU time of a call among queued ones): 64 sequences of 4-8k tokens, 32 + 8 heads
// of 128, one token each, 130 us = 6.4 TB/s, 94% of a copy (32 sequences, 16 heads: d = 64,
// 8 key heads, 41 us at 5.2 TB/s; d = 192 and 256, 4 key heads, 53 and 68 us at 5.9 and 6.1).
// 64-128 tokens over 8-16k in 4 sequences, 32 + 8 heads of 128: 60 us, of which ~8 are the
// start and the first Q tiles; 2048 tokens over 4-6k in 2: 315 us = 678 TF/s.  One token over
// 501 keys 6.1 us.
//
// A key's sum goes to memory as one addition of the whole call (one a turn, by the same
// thread), so that results do not vary from run to run; a slot that a call names twice gets
// both sums, in either order.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "../../include/fa.h"
#include "cache.cuh"
#include "common.cuh"
#include "internal.h"
#include "sm100_ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 384;
constexpr int kBN = 128;  // keys of a tile

struct Params {
    CUtensorMap tm_q, tm_k;
    fa_cache cache;
    const int* slots;
    const int* cu;
    const void* mask;
    const float* lse;
    float* weights;
    int layer, B, N, T, Hq, group, words, tile_tokens, page_shift;
    float scale_log2;
};

// D: tile columns (96 runs on 128).  NQ: query rows of a tile.  One Q tile has 64 above
// d = 128, to leave room for keys, unless a group is larger.
template <int D, int NQ, bool MANY>
struct Cfg {
    static constexpr int kCols = D / 64;
    static constexpr int kQBytes = NQ * D * 2, kStageBytes = kBN * D * 2;
    static constexpr int kRoom = 232448 - 1024 - 8192;
    static constexpr int kMostQ = (kRoom - 2 * kStageBytes) / kQBytes;
    static constexpr int kQBufs = kMostQ > (MANY ? 4 : 2) ? (MANY ? 4 : 2) : kMostQ;
    static constexpr int kMost = (kRoom - kQBufs * kQBytes) / kStageBytes;
    static constexpr int kStages = kMost > 8 ? 8 : kMost;
    static constexpr int kBuffers = MANY ? 2 : 4;         // of scores
    static constexpr int kSCols = MANY ? NQ : 128;        // from one to the next
    static constexpr int kSpan = MANY ? NQ / 2 : NQ;      // columns of a warpgroup
    static_assert(kStages >= 2 && kQBufs >= 1, "two key tiles and a Q tile");
    static_assert(kBuffers * kSCols <= 512 && kSpan <= 128, "TMEM holds the scores");
};

// A stretch of one (sequence, head)'s key tiles.
struct Piece {
    int h;               // < 0: none left
    int tok0, n;         // tokens in the packed batch, of this turn
    int first;           // the first one's index in its sequence
    int last;            // the item's last turn
    int slot, ctx, len;
    int k0, tiles;       // key tiles [k0, k0 + tiles)
};

template <int D, int NQ, bool MANY>
struct Smem {
    using C = Cfg<D, NQ, MANY>;
    alignas(1024) uint8_t q[C::kQBufs][C::kQBytes];
    alignas(1024) uint8_t k[C::kStages][C::kStageBytes];
    alignas(16) float nl[C::kQBufs][NQ];  // -LSE log2 e of the Q tile's rows
    alignas(8) uint64_t full[C::kStages], empty[C::kStages];
    uint64_t q_land[C::kQBufs];  // a Q tile's TMA
    uint64_t q_full[C::kQBufs], q_empty[C::kQBufs];  // its LSE (and rows cleared), its last reader
    uint64_t piece_full[2], piece_empty[2];
    uint64_t s_full[C::kBuffers], s_free[C::kBuffers];
    // MANY: the second warpgroup's sums, and that they are there.  It is less than four key
    // tiles ahead: the scores that it takes up wait for both to have read those before.
    uint64_t x_full[4];
    float x[MANY ? 4 : 1][kBN];
    uint64_t drain;
    Piece piece[2];
    long long sums[kThreads / 32];
    int start[3];        // this CTA's first item: sequence, head, key tile
    long long item;      // its place in the line
    uint32_t tmem_base;
    int abort_flag, zero;
};

__device__ __forceinline__ bool poll(uint32_t bar, uint32_t parity, volatile int* flag, int* status) {
    if (mbar_wait(bar, parity, flag)) return true;
    *flag = 1;
    atomicOr(status, kCacheTimeout);
    return false;
}
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* flag,
                                          int* status) {
    // the common case in one branch of the whole warp (2048 tokens over 4-6k 312 us against 318,
    // d = 256 576 against 596)
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
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

struct SeqInfo {
    int t0, n, slot, len, bad;
};

// Sequence i; one that does not fit, or has no tokens, has len = 0: no keys, no tiles.
__device__ __forceinline__ SeqInfo seq_info(const Params& p, int i) {
    SeqInfo s;
    const int slot = p.slots[i];  // (in one trip with the boundaries)
    const SeqRange r = seq_range(p.cu, p.N, p.T, i);
    s.t0 = r.t0;
    s.n = r.n;
    s.slot = s.len = s.bad = 0;
    if (r.n < 0) s.bad = kCacheBadLength;
    if (r.n <= 0) return s;
    if (slot < 0 || slot >= p.cache.slots) {
        s.bad = kCacheBadSlot;
        return s;
    }
    const int len = p.cache.lengths[slot];
    if (len < s.n || s.n > p.N || len > (long long)p.cache.max_pages * p.cache.page_size) {
        s.bad = kCacheBadLength;
        return s;
    }
    s.slot = slot;
    s.len = len;
    return s;
}

// The sum over columns [c0, ncols) of 2^(s c + nl), s from TMEM.  MASK: column
// `col` counts only where see(col).
template <bool MASK, typename See>
__device__ __forceinline__ float weigh(uint32_t s_at, const float* nl, float c, int c0, int ncols,
                                       See&& see) {
    float sum = 0.f;
    const uint64_t cc = f2_pack(c, c);
    if (!MASK && ncols >= c0 + 64) {
        uint64_t acc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = f2_pack(0.f, 0.f);
#pragma unroll 1
        for (; c0 + 64 <= ncols; c0 += 64) {
            uint32_t r[2][32];
            tmem_ld32(s_at + c0, r[0]);
            tmem_ld32(s_at + c0 + 32, r[1]);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const ulonglong2 l = reinterpret_cast<const ulonglong2*>(nl + c0)[e];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t* s = &r[e >> 3][(4 * e + 2 * h) & 31];
                    float x0, x1;
                    f2_unpack(f2_fma(f2_pack(__uint_as_float(s[0]), __uint_as_float(s[1])), cc, h ? l.y : l.x),
                              x0, x1);
                    acc[(e & 1) * 2 + h] = f2_add(acc[(e & 1) * 2 + h], f2_pack(ex2_approx(x0), ex2_approx(x1)));
                }
            }
        }
        float a, b;
        f2_unpack(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), a, b);
        sum = a + b;
    }
#pragma unroll 1
    for (; c0 < ncols; c0 += 32) {
        uint32_t r[32];
        tmem_ld32(s_at + c0, r);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            if (c0 + i >= ncols) break;
#pragma unroll
            for (int k = i; k < i + 4; ++k) {
                const int col = c0 + k;
                const float e = ex2_approx(fmaf(__uint_as_float(r[k]), c, nl[col]));
                if (col < ncols && (!MASK || see(col))) sum += e;
            }
        }
    }
    return sum;
}

template <int D, int DR, int NQ, bool MANY>
__global__ void __launch_bounds__(kThreads, 1) weights_kernel(const __grid_constant__ Params p) {
    pdl_trigger();
    using C = Cfg<D, NQ, MANY>;
    using SM = Smem<D, NQ, MANY>;
    constexpr int S = C::kStages, QB = C::kQBufs;
    static_assert(sizeof(SM) + 1024 <= 232448, "shared memory exceeds 227 KB");
    extern __shared__ uint8_t smem_raw[];
    SM& sm = *reinterpret_cast<SM*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = warp_id(), lane = lane_id();
    volatile int* stop = &sm.abort_flag;
    int* status = p.cache.scratch;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(smem_u32(&sm.full[s]), 1);
            mbar_init(smem_u32(&sm.empty[s]), 1);
        }
        for (int i = 0; i < QB; ++i) {
            mbar_init(smem_u32(&sm.q_land[i]), 1);
            mbar_init(smem_u32(&sm.q_full[i]), 1);
            mbar_init(smem_u32(&sm.q_empty[i]), 1 + 8);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sm.piece_full[i]), 1);
            mbar_init(smem_u32(&sm.piece_empty[i]), 1 + 1 + 8);
        }
        for (int i = 0; i < C::kBuffers; ++i) {
            mbar_init(smem_u32(&sm.s_full[i]), 1);
            mbar_init(smem_u32(&sm.s_free[i]), MANY ? 8 : 4);
        }
        for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&sm.x_full[i]), 4);
        mbar_init(smem_u32(&sm.drain), 1);
        sm.abort_flag = sm.zero = 0;
        sm.start[0] = -1;
        fence_barrier_init();
        tma_prefetch_desc(&p.tm_q);
        tma_prefetch_desc(&p.tm_k);
    }
    if (warp == 2) {
        tmem_alloc(smem_u32(&sm.tmem_base), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    pdl_wait();

    // Q tiles of a sequence, or of a turn: QB at most
    auto q_tiles = [&](int n) { return (n + p.tile_tokens - 1) / p.tile_tokens; };

    // ---- the line of all key tiles, each as long as its Q tiles are many, and where this
    // CTA's stretch begins: it takes the tiles that begin within
    long long at, end;
    {
        const int chunk = (p.B + kThreads - 1) / kThreads;
        const int i0 = min((long long)p.B, (long long)threadIdx.x * chunk), i1 = min(p.B, i0 + chunk);
        long long mine = 0;
        int bad = 0;
        for (int i = i0; i < i1; ++i) {
            const SeqInfo s = seq_info(p, i);
            bad |= s.bad;
            mine += (long long)cdiv(s.len, kBN) * q_tiles(s.n) * p.cache.heads;
        }
        if (bad && blockIdx.x == 0) atomicOr(status, bad);
        long long incl = mine;
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        if (lane == 31) sm.sums[warp] = incl;
        __syncthreads();
        long long before = 0, total = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before += sm.sums[w];
            total += sm.sums[w];
        }
        const long long per = (total + gridDim.x - 1) / gridDim.x;
        at = min(total, per * blockIdx.x);
        end = min(total, at + per);
        long long first = before + incl - mine;  // first tile of this thread's sequences
        if (at < end && at >= first && at < first + mine) {
            for (int i = i0; i < i1; ++i) {
                const SeqInfo s = seq_info(p, i);
                const int nq = q_tiles(s.n);
                const long long item = (long long)cdiv(s.len, kBN) * nq, all = item * p.cache.heads;
                if (at >= first + all) {
                    first += all;
                    continue;
                }
                sm.start[0] = i;
                sm.start[1] = (int)((at - first) / item);
                sm.item = first + sm.start[1] * item;
                sm.start[2] = (int)((at - sm.item + nq - 1) / nq);  // (may be behind the item's last)
                break;
            }
        }
        __syncthreads();
    }
    if (warp == 0) {
        // ------------------------------------------------------------ pieces and K
        int it = 0, f = 0, b = sm.start[0], h = sm.start[1], k0 = sm.start[2];
        const int ps = p.cache.page_size, shift = p.page_shift, boxes = kBN >> shift;
        const int box = lane / C::kCols, col = lane % C::kCols;
        bool ok = true;
        int place = -1, count = 0;  // ring place of this lane's turn among the last 32 loads
        long long item = sm.item;   // the item's place in the line
        int turn = 0;               // token that the item's next turn begins with
        SeqInfo s = {};
        bool any = at < end;
        if (any) s = seq_info(p, b);
        // the item behind this one
        auto next_item = [&] {
            item += (long long)cdiv(s.len, kBN) * q_tiles(s.n);
            k0 = 0;
            any = item < end;
            if (any && ++h == p.cache.heads) {
                h = 0;
                do {
                    if (++b >= p.B) {  // (cannot be: the line counts real tiles)
                        any = false;
                        break;
                    }
                    s = seq_info(p, b);
                } while (s.len == 0);
            }
        };
        if (any && k0 >= cdiv(s.len, kBN)) next_item();
        while (ok) {
            const int slot = it & 1;
            if (!(ok = warp_wait(smem_u32(&sm.piece_empty[slot]), ((it >> 1) & 1) ^ 1, stop, status)))
                break;
            Piece x = {};
            x.h = -1;
            const int nq = q_tiles(s.n);
            if (any && item + (long long)k0 * nq < end) {
                x.h = h;
                x.first = turn;
                x.tok0 = s.t0 + turn;
                x.n = min(s.n - turn, QB * p.tile_tokens);
                x.last = turn + x.n == s.n;
                x.slot = s.slot;
                x.len = s.len;
                x.ctx = s.len - s.n;
                x.k0 = k0;
                x.tiles = (int)min((long long)cdiv(s.len, kBN), (end - item + nq - 1) / nq) - k0;
            }
            if (lane == 0) {
                sm.piece[slot] = x;
                mbar_arrive(smem_u32(&sm.piece_full[slot]));
            }
            __syncwarp();
            ++it;
            if (x.h < 0) break;
            const int* table = p.cache.table + (long long)x.slot * p.cache.max_pages;
            const int used = (x.len + ps - 1) >> shift;
            int win = (x.k0 * kBN) >> shift;  // page ids of a window of 32 pages
            int ids = win + lane < used ? table[win + lane] : -1;
            int nxt = win + 32 + lane < used ? table[win + 32 + lane] : -1;
            for (int j = 0; j < x.tiles && ok; ++j) {
                const int key0 = (x.k0 + j) * kBN, first = key0 >> shift;
                if (first >= win + 32) {
                    win += 32;
                    ids = nxt;
                    nxt = win + 32 + lane < used ? table[win + 32 + lane] : -1;
                }
                const int page = __shfl_sync(0xffffffffu, ids, (first - win + box) & 31);
                const int st = f % S;
                if (!(ok = warp_wait(smem_u32(&sm.empty[st]), ((f / S) & 1) ^ 1, stop, status))) break;
                const int have = min(boxes, used - first);  // (pages that hold no key are not loaded)
                const uint32_t bar = smem_u32(&sm.full[st]);
                if (lane == 0) mbar_arrive_expect_tx(bar, have * ps * 128 * C::kCols);
                __syncwarp();
                if (box < have) {  // (8 boxes of 4 columns at most: a lane each)
                    int plane = -1;  // a page id out of range reads zeros and is reported
                    if (page >= 0 && page < p.cache.pages)
                        plane = (p.layer * p.cache.pages + page) * p.cache.heads + x.h;
                    else
                        atomicOr(status, kCacheBadSlot);
                    tma_load_3d(smem_u32(sm.k[st]) + col * (kBN * 128) + (box << shift) * 128, &p.tm_k,
                                bar, col * 64, 0, plane);
                }
                if ((count++ & 31) == lane) place = f;
                ++f;
            }
            turn += x.n;
            if (x.last) {
                turn = 0;
                next_item();
            }
        }
        if (!ok) {  // never leave a TMA write in flight
            int last = place;
            for (int o = 16; o; o >>= 1) last = max(last, __shfl_xor_sync(0xffffffffu, last, o));
            if (place >= 0 && place > last - S)
                mbar_wait(smem_u32(&sm.full[place % S]), (place / S) & 1, &sm.zero);
            __syncwarp();
        }
    } else if (warp == 3) {
        // ------------------------------------------------------------ Q and LSE
        int it = 0, g = 0;
        bool ok = true;
        while (ok) {
            const int slot = it & 1;
            if (!(ok = warp_wait(smem_u32(&sm.piece_full[slot]), (it >> 1) & 1, stop, status))) break;
            const Piece x = sm.piece[slot];
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.piece_empty[slot]));
            ++it;
            if (x.h < 0) break;
            {
                const int nq = q_tiles(x.n);
                for (int qt = 0; qt < nq && ok; ++qt, ++g) {
                    const int qs = g % QB;
                    if (!(ok = warp_wait(smem_u32(&sm.q_empty[qs]), ((g / QB) & 1) ^ 1, stop, status)))
                        break;
                    const uint32_t bar = smem_u32(&sm.q_land[qs]);
                    const int tok = x.tok0 + qt * p.tile_tokens;
                    const int rows = min(p.tile_tokens, x.n - qt * p.tile_tokens) * p.group;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(bar, p.tile_tokens * p.group * 128 * C::kCols);
                        for (int c = 0; c < C::kCols; ++c)
                            tma_load_4d(smem_u32(sm.q[qs]) + c * (NQ * 128), &p.tm_q, bar, c * 64, 0, x.h,
                                        tok);
                    }
                    __syncwarp();
                    float l[NQ / 32];
#pragma unroll
                    for (int i = 0; i < NQ / 32; ++i) {
                        const int r = i * 32 + lane, t = r / p.group;
                        l[i] = 0.f;
                        if (r < rows) l[i] = p.lse[(size_t)(x.h * p.group + r - t * p.group) * p.T + tok + t];
                    }
#pragma unroll
                    for (int i = 0; i < NQ / 32; ++i)  // (a row that sees nothing gives nothing)
                        sm.nl[qs][i * 32 + lane] = l[i] == -INFINITY ? -INFINITY : -l[i] * 1.4426950408889634f;
                    // ... whatever its q holds: scores that are not finite would not vanish (-inf + inf
                    // is NaN), so such rows are cleared.  (This 312 -> 315 us; looking at each sum for NaN: 317)
                    bool gone = false;
#pragma unroll
                    for (int i = 0; i < NQ / 32; ++i) gone |= l[i] == -INFINITY;
                    if (__any_sync(0xffffffffu, gone)) {
                        if (!(ok = warp_wait(bar, (g / QB) & 1, stop, status))) {
                            ++g;
                            break;
                        }
#pragma unroll
                        for (int i = 0; i < NQ / 32; ++i)
                            if (l[i] == -INFINITY)
                                for (int c = 0; c < C::kCols * 8; ++c)
                                    *reinterpret_cast<uint4*>(sm.q[qs] + (c >> 3) * (NQ * 128) + (i * 32 + lane) * 128 +
                                                              (c & 7) * 16) = make_uint4(0, 0, 0, 0);
                        fence_proxy_async_smem();
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sm.q_full[qs]));
                }
            }
        }
        if (!ok && lane == 0)
            for (int i = 0; i < QB && i < g; ++i)
                mbar_wait(smem_u32(&sm.q_land[(g - 1 - i) % QB]), ((g - 1 - i) / QB) & 1, &sm.zero);
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        constexpr uint32_t id = make_idesc_bf16(128, NQ, false, false);
        const uint32_t lead = elect_lead();
        int it = 0, f = 0, g = 0, cnt[2] = {0, 0};  // (MANY: cnt[0])
        bool ok = true;
        auto wait = [&](uint64_t& bar, int parity) {
            return ok = ok && warp_wait(smem_u32(&bar), parity & 1, stop, status);
        };
        while (ok) {
            const int slot = it & 1;
            if (!wait(sm.piece_full[slot], it >> 1)) break;
            const int h = __shfl_sync(0xffffffffu, sm.piece[slot].h, 0);
            const int n = __shfl_sync(0xffffffffu, sm.piece[slot].n, 0);
            const int tiles = __shfl_sync(0xffffffffu, sm.piece[slot].tiles, 0);
            if (lane == 0) mbar_arrive(smem_u32(&sm.piece_empty[slot]));
            __syncwarp();
            ++it;
            if (h < 0) break;
            const int nq = q_tiles(n);
            for (int j = 0; j < tiles && ok; ++j, ++f) {
                for (int qt = 0; qt < nq && ok; ++qt) {
                    const int gq = g + qt, w = MANY ? 0 : j & 1;
                    const int bf = (MANY ? 0 : 2 * w) + (cnt[w] & 1);
                    if (j == 0) {
                        const bool q_in = mbar_test_wait(smem_u32(&sm.q_land[gq % QB]), (gq / QB) & 1);
                        const bool l_in = mbar_test_wait(smem_u32(&sm.q_full[gq % QB]), (gq / QB) & 1);
                        if (!__all_sync(0xffffffffu, q_in) && !wait(sm.q_land[gq % QB], gq / QB)) break;
                        if (!__all_sync(0xffffffffu, l_in) && !wait(sm.q_full[gq % QB], gq / QB)) break;
                    }
                    // (a wait takes ~140 cycles even when nothing is missing: both are looked
                    // up at once first.  Each is at most a phase behind.)
                    const bool k_in = qt > 0 || mbar_test_wait(smem_u32(&sm.full[f % S]), (f / S) & 1);
                    const bool s_in = cnt[w] < 2 || mbar_test_wait(smem_u32(&sm.s_free[bf]), ((cnt[w] - 2) >> 1) & 1);
                    if (!__all_sync(0xffffffffu, k_in) && !wait(sm.full[f % S], f / S)) break;
                    if (!__all_sync(0xffffffffu, s_in) && !wait(sm.s_free[bf], (cnt[w] - 2) >> 1)) break;
                    tc_fence_after();
                    const uint64_t da = make_sdesc(smem_u32(sm.k[f % S]), 16, 1024);
                    const uint64_t db = make_sdesc(smem_u32(sm.q[gq % QB]), 16, 1024);
#pragma unroll
                    for (int kk = 0; kk < DR / 16; ++kk)
                        warp_mma_ss(lead, tmem + bf * C::kSCols,
                                    sdesc_add(da, (kk >> 2) * (kBN * 128) + (kk & 3) * 32),
                                    sdesc_add(db, (kk >> 2) * (NQ * 128) + (kk & 3) * 32), id, kk > 0);
                    warp_mma_commit(lead, smem_u32(&sm.s_full[bf]));
                    if (qt == nq - 1) warp_mma_commit(lead, smem_u32(&sm.empty[f % S]));
                    if (j == tiles - 1) warp_mma_commit(lead, smem_u32(&sm.q_empty[gq % QB]));
                    ++cnt[w];
                }
            }
            g += nq;
        }
        warp_mma_commit(lead, smem_u32(&sm.drain));
        mbar_wait(smem_u32(&sm.drain), 0, &sm.zero);
    } else if (warp >= 4) {
        // ------------------------------------------------------------ exponentials and sums
        const int w = (warp - 4) >> 2, q4 = warp & 3;
        const int row = q4 * 32 + lane;  // key of the tile
        const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
        // col / group is (col * per_group) >> 16: the product is less than 256 / 65536 of a
        // group too large
        const unsigned per_group = 65536u / p.group + 1;
        int it = 0, g = 0, cnt = 0, x_it = 0;  // x_it: key tiles whose halves have met
        bool ok = true;
        while (ok) {
            const int slot = it & 1;
            if (!(ok = warp_wait(smem_u32(&sm.piece_full[slot]), (it >> 1) & 1, stop, status))) break;
            const Piece x = sm.piece[slot];
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.piece_empty[slot]));
            ++it;
            if (x.h < 0) break;
            const int nq = q_tiles(x.n);
            float* out = p.weights + ((long long)x.slot * p.cache.heads + x.h) *
                                         ((long long)p.cache.max_pages * p.cache.page_size);
            const int c0 = MANY ? w * C::kSpan : 0;  // this warpgroup's first column
            for (int qt = 0; qt < nq && ok; ++qt)    // (the LSE that the scores go with)
                ok = warp_wait(smem_u32(&sm.q_full[(g + qt) % QB]), ((g + qt) / QB) & 1, stop, status);
            for (int j = MANY ? 0 : w; j < x.tiles && ok; j += MANY ? 1 : 2) {
                const int key0 = (x.k0 + j) * kBN, key = key0 + row;
                const bool own = key0 + kBN > x.ctx;  // some keys are the call's own tokens
                float sum = 0.f;
                for (int qt = 0; qt < nq; ++qt, ++cnt) {
                    const int qs = (g + qt) % QB, bf = (MANY ? 0 : 2 * w) + (cnt & 1);
                    if (!(ok = warp_wait(smem_u32(&sm.s_full[bf]), (cnt >> 1) & 1, stop, status))) break;
                    tc_fence_after();
                    const uint32_t s_at = tmem + lane_off + bf * C::kSCols;
                    const int tok0 = qt * p.tile_tokens;
                    const int ncols = min(min(p.tile_tokens, x.n - tok0) * p.group, c0 + C::kSpan);
                    const float* nl = sm.nl[qs];
                    // without a mask most Q tiles see all keys of the tile, or none
                    const int tok = x.first + tok0, k0 = key0 - x.ctx;  // first token, first key
                    const bool none = !p.mask && k0 >= tok + min(p.tile_tokens, x.n - tok0);
                    if (none) {
                    } else if (!own || (!p.mask && k0 + kBN - 1 <= tok)) {
                        sum += weigh<false>(s_at, nl, p.scale_log2, c0, ncols, [](int) { return true; });
                    } else {
                        const int k = key - x.ctx;  // among the sequence's new tokens; < 0: the context
                        if (!p.mask) {
                            const int from = (k - tok) * p.group;  // column that sees it
                            sum += weigh<true>(s_at, nl, p.scale_log2, c0, ncols,
                                               [&](int col) { return col >= from; });
                        } else {
                            const unsigned long long* words = static_cast<const unsigned long long*>(p.mask) +
                                                              (size_t)(x.tok0 + tok0) * p.words + max(k, 0) / 64;
                            const bool some = k < 64 * p.words;
                            sum += weigh<true>(s_at, nl, p.scale_log2, c0, ncols, [&](int col) {
                                if (k < 0) return true;
                                const int t = (int)(((unsigned)col * per_group) >> 16);
                                return some && ((words[(size_t)t * p.words] >> (k & 63)) & 1) != 0;
                            });
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sm.s_free[bf]));
                }
                if (!ok) break;
                if constexpr (MANY) {
                    const int xs = x_it & 3;
                    if (w == 1) {
                        sm.x[xs][row] = sum;
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_u32(&sm.x_full[xs]));
                    } else {
                        if (!(ok = warp_wait(smem_u32(&sm.x_full[xs]), (x_it >> 2) & 1, stop, status))) break;
                        sum += sm.x[xs][row];
                    }
                    ++x_it;
                    if (w == 1) continue;
                }
                if (key < x.len) atomicAdd(out + key, sum);
            }
            __syncwarp();
            if (ok && lane == 0)
                for (int qt = 0; qt < nq; ++qt) mbar_arrive(smem_u32(&sm.q_empty[(g + qt) % QB]));
            g += nq;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D, int DR, int NQ, bool MANY>
cudaError_t launch(const Params& p, int ctas, cudaStream_t stream) {
    auto kern = weights_kernel<D, DR, NQ, MANY>;
    constexpr size_t smem = sizeof(Smem<D, NQ, MANY>) + 1024;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(ctas), dim3(kThreads), smem, stream, p);
}

bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" fa_status fa_cache_weights(const fa_cache* cache, int layer, const int* slots, int B, int N,
                                      const int* cu_seqlens, int T, const void* q, int Hq,
                                      long long q_token_stride, long long q_head_stride,
                                      const float* lse, const void* mask, int mask_words,
                                      float* weights, float scale, fa_stream_t stream) {
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
    if (T == 0 || B == 0) return FA_OK;
    if (!slots || !q || !lse || !weights) return FA_ERR_INVALID_ARG;
    if (N == 0) N = 1;  // (a packed batch of empty sequences)
    if (!aligned(slots, 4) || !aligned(cu_seqlens, 4) || !aligned(q, 16) || !aligned(lse, 4) ||
        !aligned(mask, 8) || !aligned(weights, 4))
        return FA_ERR_INVALID_ARG;
    if (T == 1) q_token_stride = (long long)Hq * d;  // (a stride that is never taken)
    if (Hq == 1) q_head_stride = d;
    if (q_token_stride <= 0 || q_head_stride <= 0 || q_token_stride % 8 || q_head_stride % 8 ||
        q_token_stride >= (1LL << 38) || q_head_stride >= (1LL << 31))
        return FA_ERR_INVALID_ARG;
    const int group = Hq / Hkv, few = d > 128 && group <= 64 ? 64 : 128;  // rows of the only Q tile
    const bool many = (long long)N * group > few;
    const int nq = !many ? few : (d > 128 ? 128 : 256);
    const int tokens = nq / group < N ? nq / group : N;
    TreeParams maps;
    std::memset(&maps, 0, sizeof(maps));
    if (!make_tree_maps(maps, *cache, q, T, Hq, q_token_stride, q_head_stride, tokens, kBN))
        return FA_ERR_CUDA;
    Params p;
    std::memset(&p, 0, sizeof(p));
    p.tm_q = maps.tm_q;
    p.tm_k = maps.tm_k;
    p.cache = *cache;
    p.slots = slots;
    p.cu = cu_seqlens;
    p.mask = mask;
    p.words = mask_words;
    p.lse = lse;
    p.weights = weights;
    p.layer = layer;
    p.B = B; p.N = N; p.T = T; p.Hq = Hq;
    p.group = group;
    p.tile_tokens = tokens;
    p.page_shift = __builtin_ctz(cache->page_size);
    p.scale_log2 = scale * 1.4426950408889634f;
    const int ctas = device_sms();
    if (ctas <= 0) return FA_ERR_CUDA;
    cudaStream_t strm = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (many) {
        if (d == 64) e = launch<64, 64, 256, true>(p, ctas, strm);
        else if (d == 96) e = launch<128, 96, 256, true>(p, ctas, strm);
        else if (d == 128) e = launch<128, 128, 256, true>(p, ctas, strm);
        else if (d == 192) e = launch<192, 192, 128, true>(p, ctas, strm);
        else e = launch<256, 256, 128, true>(p, ctas, strm);
    } else if (d == 64) e = launch<64, 64, 128, false>(p, ctas, strm);
    else if (d == 96) e = launch<128, 96, 128, false>(p, ctas, strm);
    else if (d == 128) e = launch<128, 128, 128, false>(p, ctas, strm);
    else if (d == 192) e = few == 64 ? launch<192, 192, 64, false>(p, ctas, strm)
                                     : launch<192, 192, 128, false>(p, ctas, strm);
    else e = few == 64 ? launch<256, 256, 64, false>(p, ctas, strm)
                       : launch<256, 256, 128, false>(p, ctas, strm);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
