// rotary.cu -- rotary positions, forward and backward, and the same pass
// writing new keys and values into a paged cache.
//
// A head's first rot columns are rot / 2 pairs; pair i of a token at position
// p turns by the angle p * freq_i: (a, b) -> (a cos - b sin, b cos + a sin).
// A pair is columns (i, i + rot/2) (half layout) or (2i, 2i + 1)
// (interleaved).  The rotation is linear, so its backward pass is the
// transposed one: the same kernel with sin negated.  cos and sin come from a
// table [length, rot/2, 2] in fp32 that the caller keeps; products and sums
// are fp32, rounded once on the store.
//
// Bound: memory.  Each value is read and written once, and nothing is reused
// but the token's table row.  So a thread takes one 16-byte unit of a head's
// columns in kHeadsPerThread heads of one token: the cos and sin it loads serve
// all of them, and all its loads are in flight before the first use.  In the
// half layout the two halves of a pair lie in two lanes, which exchange them:
// a thread that loads both halves needs 91 registers instead of 56 and has too
// few warps beside it (bf16, 2 x 8192 tokens, 32 + 8 heads of 128: 91 us; now 55
// us, interleaved 50 us; fp32 with 16 + 16 heads of 192, 59 us; at the copy rate
// 50, 50 and 60 us).  bf16 is not far from the instruction limit either (60% of
// issue slots), which is why indexes are divided by multiplication.  Blocks of
// 64 threads, 4 heads a thread: 128 threads up to 3% slower; 32 threads or 2 heads
// 50% slower, since blocks start no faster than one in a nanosecond; 8 heads 3%
// faster in the half layout, 2% slower interleaved, 15% slower for few tokens.
// Head dimensions, strides or alignments that do not allow 16-byte accesses
// run the same code one element at a time (VW = 1: 2 x 8192 tokens, 32 + 8 heads of
// 80 with 20 or 40 columns turned in the half layout, 181 and 155 us for 31 us of
// bytes), and fp32 heads wider than a warp's lanes take both halves in a thread.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/fa.h"
#include "cache.cuh"
#include "common.cuh"
#include "internal.h"

namespace fa {
namespace {

constexpr int kRotThreads = 64;
constexpr int kHeadsPerThread = 4;
constexpr long long kMostThreads = 0x3FFFFF00LL;  // of a launch (idle lanes come on top)

// Division by a number known at the launch: a high product and a shift
// (x < 2^31; the multiplier is 2^(32 + s) / d rounded up, 2^s >= d).
struct Divider {
    unsigned d, mul, shift;
    void set(unsigned by) {
        d = by;
        shift = 0;
        while ((1u << shift) < by) ++shift;
        mul = (unsigned)(((1ull << 32) * ((1ull << shift) - by)) / by + 1);
    }
    __device__ __forceinline__ unsigned operator()(unsigned x) const {
        return (unsigned)(((unsigned long long)__umulhi(x, mul) + x) >> shift);
    }
};

struct RotParams {
    // segment 0: q, 1: k, 2: v (copied); heads 0 when absent
    const void* in[3];
    void* out[3];                // contiguous [T, heads, d]; 1 and 2 are unused for a paged call
    long long ts[3], hs[3];      // input strides in elements
    int heads[3], quads[3];      // quads: groups of kHeadsPerThread heads
    int T, d, rot, units;        // units per head
    Divider by_units, by_quads;  // quads: of a token, all segments
    int t_first;                 // first token of this launch
    unsigned n_items;            // (token, quad) pairs, times units where lanes are not grouped
    int lanes;                   // kShuffle: items of one warp
    const float2* table;         // [table_len, rot / 2]
    int table_len;
    const void* positions;       // int32 or int64 [T], or null
    int pos64;
    const int* cu;               // packed batch, or null
    int B, N;
    int backward;
    // paged call
    fa_cache cache;
    const int* slots;
    int layer, page_shift;
    unsigned bounds_block;       // one more block, which looks the boundaries over
};

template <typename E>
__device__ __forceinline__ float to_f(E x) { return (float)x; }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename E>
__device__ __forceinline__ E from_f(float x) { return (E)x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16_rn(x); }

template <typename E, int VW>
struct alignas(VW * sizeof(E)) Vec {
    E e[VW];
};

// Data is read and written once: lines that leave the caches first (2 x 8192
// tokens 61.6 -> 57.6 us, appended prompts 47.6 -> 46.8; as whole 16-byte values,
// not as elements, which takes 45 registers there instead of 62, 53.5 -> 47.6).
template <typename V>
__device__ __forceinline__ V load_once(const void* p) {
    if constexpr (sizeof(V) == 16) {
        const uint4 y = __ldcs(static_cast<const uint4*>(p));
        return *reinterpret_cast<const V*>(&y);
    } else {
        return *static_cast<const V*>(p);
    }
}
template <typename V>
__device__ __forceinline__ void store_once(void* p, const V& v) {
    if constexpr (sizeof(V) == 16) __stcs(static_cast<uint4*>(p), *reinterpret_cast<const uint4*>(&v));
    else *static_cast<V*>(p) = v;
}

// Where the two halves of a pair are: in one access (kInter: pairs (2i, 2i + 1)),
// in two accesses of the thread (kTwo), or in the accesses of two lanes of a
// warp, which exchange them (kShuffle: half layout, a head's row in one warp).
enum Layout { kInter, kTwo, kShuffle };

// E: element type; VW: elements of one access; PAGED: k and v go to the
// cache's pages.
template <typename E, int VW, Layout L, bool PAGED>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const __grid_constant__ RotParams p) {
    pdl_begin();
    constexpr bool INTER = L == kInter;
    using V = Vec<E, VW>;
    if (PAGED && blockIdx.x == p.bounds_block) {
        // Boundaries that decrease or leave the batch are reported here: the tokens'
        // search takes them as ascending and may not meet the sequence (as a block of
        // its own, it delays no token).
        bool bad = false;
        for (int i = threadIdx.x; i < p.B; i += kRotThreads)
            bad |= seq_range(p.cu, p.N, p.T, i).n < 0;
        if (bad) atomicOr(p.cache.scratch, kCacheBadLength);
        return;
    }
    const unsigned U = p.units;
    const unsigned quads = p.quads[0] + p.quads[1] + p.quads[2];
    unsigned item;  // token * quads + quad
    int u;
    bool idle = false;
    if (L == kShuffle) {  // whole heads to a warp; the lanes left over follow item 0
        const unsigned lane = threadIdx.x & 31, warp = (blockIdx.x * kRotThreads + threadIdx.x) >> 5;
        const unsigned g = p.by_units(lane);
        item = warp * p.lanes + g;
        u = (int)(lane - g * U);
        idle = g >= (unsigned)p.lanes || item >= p.n_items;
        if (idle) item = 0;
    } else {
        const unsigned idx = blockIdx.x * kRotThreads + threadIdx.x;
        if (idx >= p.n_items) return;
        item = p.by_units(idx);
        u = (int)(idx - item * U);
    }
    const unsigned tok_i = p.by_quads(item);
    const int tok = p.t_first + (int)tok_i;
    int quad = (int)(item - tok_i * quads);
    int seg = 0;
    if (quad >= p.quads[0]) {
        quad -= p.quads[0];
        seg = 1;
        if (quad >= p.quads[1]) {
            quad -= p.quads[1];
            seg = 2;
        }
    }
    const int h0 = quad * kHeadsPerThread;
    const int nh = idle ? 0 : min(kHeadsPerThread, p.heads[seg] - h0);

    // Columns of this unit: one access (c0) or, for the pairs of the half
    // layout, two (c0 and c1).  first_pair < 0: nothing turns here.
    const int half = p.rot >> 1;
    int c0, c1 = -1, first_pair = -1;
    if (INTER) {
        // VW = 1 takes whole pairs all the same: unit u < half is pair u
        if (VW == 1) {
            if (u < half) { c0 = 2 * u; c1 = 2 * u + 1; first_pair = u; }
            else c0 = p.rot + (u - half);
        } else {
            c0 = u * VW;
            if (c0 < p.rot) first_pair = c0 >> 1;
        }
    } else if (L == kShuffle) {
        c0 = u * VW;
        if (c0 < p.rot) first_pair = c0 < half ? c0 : c0 - half;
    } else {
        const int pair_units = half / VW;
        if (u < pair_units) { c0 = u * VW; c1 = c0 + half; first_pair = c0; }
        else c0 = p.rot + (u - pair_units) * VW;
    }

    // All of the thread's data loads first; the position follows while they fly.
    const E* src = static_cast<const E*>(p.in[seg]) + (long long)tok * p.ts[seg] +
                   (long long)h0 * p.hs[seg];
    V x0[kHeadsPerThread], x1[kHeadsPerThread];
#pragma unroll
    for (int h = 0; h < kHeadsPerThread; ++h) {
        if (h < nh) {
            x0[h] = load_once<V>(src + h * p.hs[seg] + c0);
            if (c1 >= 0) x1[h] = load_once<V>(src + h * p.hs[seg] + c1);
        }
    }

    // The token's sequence, place in the cache and position.
    bool owned = true, writable = true;
    long long pos = 0, place_off = 0;
    if (PAGED) {
        const int b = seq_of_token(p.cu, p.B, p.N, tok);
        owned = b >= 0;
        int place = -1;
        if (owned) {
            const SeqRange r = seq_range(p.cu, p.N, p.T, b);
            const int slot = p.slots[b];
            int bad = 0;
            if (r.n < 0) bad = kCacheBadLength;
            else if (slot < 0 || slot >= p.cache.slots) bad = kCacheBadSlot;
            else {
                // (a length is at most 2^30, and out-of-range ones wrap to no column)
                const int at = p.cache.lengths[slot] - r.n + (tok - r.t0);
                const unsigned col = (unsigned)at >> p.page_shift;
                if (at < 0 || col >= (unsigned)p.cache.max_pages) bad = kCacheBadLength;
                else {
                    place = at;
                    if (seg != 0) {  // (q stays out of the cache)
                        const int page = p.cache.table[(long long)slot * p.cache.max_pages + col];
                        if (page < 0 || page >= p.cache.pages) bad = kCacheBadSlot;
                        else if (p.cache.refs[page] > 1) bad = kCacheShared;  // (costs < 1%)
                        else
                            place_off = ((((long long)p.layer * p.cache.pages + page) *
                                              p.cache.heads + h0) * p.cache.page_size +
                                         (place & (p.cache.page_size - 1))) * p.d;
                    }
                }
            }
            if (bad) {
                if (!idle) atomicOr(p.cache.scratch, bad);
                writable = false;
            }
        }
        pos = place;
    } else if (!p.positions) {
        const int b = seq_of_token(p.cu, p.B, p.N, tok);
        owned = b >= 0;
        if (owned) pos = tok - (p.cu ? p.cu[b] : b * p.N);
    }
    if (p.positions)
        pos = p.pos64 ? static_cast<const long long*>(p.positions)[tok]
                      : (long long)static_cast<const int*>(p.positions)[tok];

    const bool turns = seg != 2 && first_pair >= 0;
    if (turns || L == kShuffle) {
        // A position outside the table reads nothing and makes the columns NaN.
        const bool known = pos >= 0 && pos < p.table_len;
        constexpr int NP = INTER && VW > 1 ? VW / 2 : VW;  // pairs of this unit
        float cs[NP], sn[NP];
        const float2* row = p.table + (known ? pos : 0) * half + first_pair;
        if (!turns) {
#pragma unroll
            for (int i = 0; i < NP; ++i) { cs[i] = 1.f; sn[i] = 0.f; }
        } else if (NP == 1) {
            const float2 t = *row;
            cs[0] = t.x;
            sn[0] = t.y;
        } else {
            // two pairs an access: the row begins at a multiple of 16 bytes (see vector_ok)
#pragma unroll
            for (int i = 0; i < NP / 2; ++i) {
                const float4 t = reinterpret_cast<const float4*>(row)[i];
                cs[2 * i] = t.x;
                sn[2 * i] = t.y;
                cs[2 * i + 1] = t.z;
                sn[2 * i + 1] = t.w;
            }
        }
        if (turns && !known) {
#pragma unroll
            for (int i = 0; i < NP; ++i) cs[i] = sn[i] = NAN;
        }
        // backward turns the other way; own * cos +- partner * sin for the lanes of a pair
        const float sign = (p.backward != 0) != (L == kShuffle && c0 < half) ? -1.f : 1.f;
#pragma unroll
        for (int i = 0; i < NP; ++i) sn[i] *= sign;
#pragma unroll
        for (int h = 0; h < kHeadsPerThread; ++h) {
            if (L == kShuffle) {
                // own * cos -+ partner * sin, the partner's columns from its lane
                const int step = turns ? (c0 < half ? half : -half) / VW : 0;
                V other;
                const unsigned* mine = reinterpret_cast<const unsigned*>(&x0[h]);
                unsigned* theirs = reinterpret_cast<unsigned*>(&other);
#pragma unroll
                for (int i = 0; i < (int)sizeof(V) / 4; ++i)
                    theirs[i] = __shfl_sync(0xffffffffu, mine[i], (int)(threadIdx.x & 31) + step);
                if (turns) {
#pragma unroll
                    for (int i = 0; i < VW; ++i)
                        x0[h].e[i] = from_f<E>(to_f(x0[h].e[i]) * cs[i % NP] + to_f(other.e[i]) * sn[i % NP]);
                }
                continue;
            }
            if (h >= nh) break;
            if (INTER && VW > 1) {
#pragma unroll
                for (int i = 0; i < VW / 2; ++i) {
                    const float a = to_f(x0[h].e[2 * i]), b = to_f(x0[h].e[2 * i + 1]);
                    x0[h].e[2 * i] = from_f<E>(a * cs[i] - b * sn[i]);
                    x0[h].e[2 * i + 1] = from_f<E>(b * cs[i] + a * sn[i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < VW; ++i) {
                    const float a = to_f(x0[h].e[i]), b = to_f(x1[h].e[i]);
                    x0[h].e[i] = from_f<E>(a * cs[i] - b * sn[i]);
                    x1[h].e[i] = from_f<E>(b * cs[i] + a * sn[i]);
                }
            }
        }
    }
    if (!owned) {  // a token behind the last sequence: zeros, and nothing in the cache
        writable = false;
#pragma unroll
        for (int h = 0; h < kHeadsPerThread; ++h)
#pragma unroll
            for (int i = 0; i < VW; ++i) x0[h].e[i] = x1[h].e[i] = from_f<E>(0.f);
    }

    E* dst;
    long long hs;
    if (PAGED && seg != 0) {
        if (!writable) return;
        dst = static_cast<E*>(seg == 1 ? p.cache.k : p.cache.v) + place_off;
        hs = (long long)p.cache.page_size * p.d;
    } else {
        dst = static_cast<E*>(p.out[seg]) + ((long long)tok * p.heads[seg] + h0) * p.d;
        hs = p.d;
    }
#pragma unroll
    for (int h = 0; h < kHeadsPerThread; ++h) {
        if (h < nh) {
            store_once(dst + h * hs + c0, x0[h]);
            if (c1 >= 0) store_once(dst + h * hs + c1, x1[h]);
        }
    }
}

template <typename E, int VW, Layout L, bool PAGED>
cudaError_t launch_t(RotParams p, cudaStream_t stream) {
    const int half = p.rot / 2;
    p.units = VW == 1 ? half + (p.d - p.rot)
                      : (L != kTwo ? p.d / VW : half / VW + (p.d - p.rot) / VW);
    for (int s = 0; s < 3; ++s) p.quads[s] = cdiv(p.heads[s], kHeadsPerThread);
    const long long per_token = (long long)(p.quads[0] + p.quads[1] + p.quads[2]) * p.units;
    if (per_token == 0) return cudaSuccess;
    p.lanes = 32 / p.units;
    p.by_units.set(p.units);
    p.by_quads.set(p.quads[0] + p.quads[1] + p.quads[2]);
    // item and thread indexes are 32 bits: more tokens than that go in several launches
    const long long most = kMostThreads / per_token;
    for (long long t = 0; t < p.T; t += most) {
        const long long n = p.T - t < most ? p.T - t : most;
        p.t_first = (int)t;
        long long threads = n * per_token;
        if (L == kShuffle) {
            p.n_items = (unsigned)(threads / p.units);
            threads = ((long long)p.n_items + p.lanes - 1) / p.lanes * 32;
        } else {
            p.n_items = (unsigned)threads;
        }
        dim3 grid((unsigned)((threads + kRotThreads - 1) / kRotThreads));
        p.bounds_block = ~0u;
        if (PAGED && p.cu && t == 0) p.bounds_block = grid.x++;
        const cudaError_t e = launch_pdl(rotary_kernel<E, VW, L, PAGED>, grid, dim3(kRotThreads), 0,
                                         stream, p);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// 16-byte accesses need every unit to begin on a 16-byte boundary, in memory
// and in the rotated columns, and the units' pairs to begin on an even pair.
template <typename E>
bool vector_ok(const RotParams& p, int interleaved, bool paged) {
    constexpr int VW = 16 / (int)sizeof(E);
    if (p.d % VW || p.rot % VW || (!interleaved && (p.rot / 2) % VW)) return false;
    uintptr_t bits = reinterpret_cast<uintptr_t>(p.table);
    if (paged)
        bits |= reinterpret_cast<uintptr_t>(p.cache.k) | reinterpret_cast<uintptr_t>(p.cache.v);
    for (int s = 0; s < 3; ++s) {
        if (!p.heads[s]) continue;
        bits |= reinterpret_cast<uintptr_t>(p.in[s]) | (uintptr_t)(p.ts[s] * (long long)sizeof(E)) |
                (uintptr_t)(p.hs[s] * (long long)sizeof(E));
        if (!paged || s == 0) bits |= reinterpret_cast<uintptr_t>(p.out[s]);
    }
    return (bits & 15u) == 0;
}

template <typename E, bool PAGED>
cudaError_t launch_any(const RotParams& p, int interleaved, cudaStream_t stream) {
    constexpr int VW = 16 / (int)sizeof(E);
    if (!vector_ok<E>(p, interleaved, PAGED))
        return interleaved ? launch_t<E, 1, kInter, PAGED>(p, stream)
                           : launch_t<E, 1, kTwo, PAGED>(p, stream);
    if (interleaved) return launch_t<E, VW, kInter, PAGED>(p, stream);
    return p.d <= 32 * VW ? launch_t<E, VW, kShuffle, PAGED>(p, stream)
                          : launch_t<E, VW, kTwo, PAGED>(p, stream);
}

// Table row of one position: angle p * freq in 64 bits, so that far positions
// keep their phase, rounded once to fp32.
__global__ void rotary_table_kernel(const double* freq, int half, long long n, double scale,
                                    float2* table) {
    pdl_begin();
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= n) return;
    const long long pos = i / half;
    double s, c;
    sincos((double)pos * freq[i - pos * half], &s, &c);
    table[i] = make_float2((float)(c * scale), (float)(s * scale));
}

bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// The arguments that both calls share.
fa_status check_rotary(const RotParams& p, const float* table, int pos_bytes) {
    if (p.T < 0 || p.d <= 0 || p.d > 65536 || p.rot < 0 || p.rot > p.d || (p.rot & 1))
        return FA_ERR_INVALID_ARG;
    for (int s = 0; s < 3; ++s)
        if (p.heads[s] < 0 || p.heads[s] > 65535 || p.ts[s] < 0 || p.hs[s] < 0)
            return FA_ERR_INVALID_ARG;
    if (p.B < 0 || p.N < 0 || p.table_len < 0) return FA_ERR_INVALID_ARG;
    if (pos_bytes != 0 && pos_bytes != 4 && pos_bytes != 8) return FA_ERR_INVALID_ARG;
    if ((pos_bytes != 0) != (p.positions != nullptr)) return FA_ERR_INVALID_ARG;
    if (!aligned(p.positions, pos_bytes ? pos_bytes : 1) || !aligned(p.cu, 4) || !aligned(table, 8))
        return FA_ERR_INVALID_ARG;
    if (!p.cu && (long long)p.B * p.N != p.T) return FA_ERR_INVALID_ARG;
    if (p.B > kMostSequences) return FA_ERR_UNSUPPORTED;
    // the most threads that one token takes must leave room for 32-bit indexes
    if (((long long)p.heads[0] + p.heads[1] + p.heads[2] + 12) / kHeadsPerThread * p.d > kMostThreads)
        return FA_ERR_UNSUPPORTED;
    return FA_OK;
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

fa_status fa_rotary_table(const double* freq, int half, long long length, double scale,
                          float* table, fa_stream_t stream) {
    if (half <= 0 || half > 32768 || length < 0 || length > 0x7FFFFFFFLL || !std::isfinite(scale))
        return FA_ERR_INVALID_ARG;
    if (length == 0) return FA_OK;
    if (!freq || !table || !aligned(freq, 8) || !aligned(table, 16)) return FA_ERR_INVALID_ARG;
    const long long n = length * half;
    if (n > 0x7FFFFFFFLL * 256) return FA_ERR_UNSUPPORTED;
    const cudaError_t e =
        launch_pdl(rotary_table_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0,
                   reinterpret_cast<cudaStream_t>(stream), freq, half, n, scale,
                   reinterpret_cast<float2*>(table));
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_rotary(const void* q, void* q_out, int Hq, long long q_token_stride,
                    long long q_head_stride, const void* k, void* k_out, int Hkv,
                    long long k_token_stride, long long k_head_stride, fa_dtype dtype, int T,
                    int d, int rot, const float* table, int table_len, const void* positions,
                    int pos_bytes, int B, int N, const int* cu_seqlens, int interleaved,
                    int backward, fa_stream_t stream) {
    RotParams p;
    std::memset(&p, 0, sizeof(p));
    p.in[0] = q; p.out[0] = q_out; p.heads[0] = Hq; p.ts[0] = q_token_stride; p.hs[0] = q_head_stride;
    p.in[1] = k; p.out[1] = k_out; p.heads[1] = Hkv; p.ts[1] = k_token_stride; p.hs[1] = k_head_stride;
    p.T = T; p.d = d; p.rot = rot;
    p.table = reinterpret_cast<const float2*>(table);
    p.table_len = table_len;
    p.positions = positions;
    p.pos64 = pos_bytes == 8;
    p.cu = cu_seqlens;
    p.B = B; p.N = N;
    p.backward = backward ? 1 : 0;
    if (dtype != FA_BF16 && dtype != FA_FP32) return FA_ERR_INVALID_ARG;
    const fa_status st = check_rotary(p, table, pos_bytes);
    if (st != FA_OK) return st;
    if (T == 0 || Hq + Hkv == 0) return FA_OK;
    if ((Hq > 0 && (!q || !q_out)) || (Hkv > 0 && (!k || !k_out)) || (rot > 0 && !table))
        return FA_ERR_INVALID_ARG;
    const unsigned e = dtype == FA_BF16 ? 2 : 4;
    if (!aligned(q, e) || !aligned(q_out, e) || !aligned(k, e) || !aligned(k_out, e))
        return FA_ERR_INVALID_ARG;
    if (rot > 0 && table_len == 0) return FA_ERR_INVALID_ARG;
    cudaStream_t strm = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t err = dtype == FA_BF16 ? launch_any<__nv_bfloat16, false>(p, interleaved, strm)
                                             : launch_any<float, false>(p, interleaved, strm);
    return err == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_cache_append(const fa_cache* cache, int layer, const int* slots, int B, int N,
                          const int* cu_seqlens, int T, const void* q, void* q_out, int Hq,
                          long long q_token_stride, long long q_head_stride, const void* k,
                          long long k_token_stride, long long k_head_stride, const void* v,
                          long long v_token_stride, long long v_head_stride, int rot,
                          const float* table, int table_len, const void* positions, int pos_bytes,
                          int interleaved, fa_stream_t stream) {
    const fa_status cs = check_cache(cache);
    if (cs != FA_OK) return cs;
    if (layer < 0 || layer >= cache->layers) return FA_ERR_INVALID_ARG;
    RotParams p;
    std::memset(&p, 0, sizeof(p));
    p.in[0] = q; p.out[0] = q_out; p.heads[0] = Hq; p.ts[0] = q_token_stride; p.hs[0] = q_head_stride;
    p.in[1] = k; p.heads[1] = cache->heads; p.ts[1] = k_token_stride; p.hs[1] = k_head_stride;
    p.in[2] = v; p.heads[2] = cache->heads; p.ts[2] = v_token_stride; p.hs[2] = v_head_stride;
    p.T = T; p.d = cache->d; p.rot = rot;
    p.table = reinterpret_cast<const float2*>(table);
    p.table_len = table_len;
    p.positions = positions;
    p.pos64 = pos_bytes == 8;
    p.cu = cu_seqlens;
    p.B = B; p.N = N;
    p.cache = *cache;
    p.slots = slots;
    p.layer = layer;
    p.page_shift = __builtin_ctz(cache->page_size);
    const fa_status st = check_rotary(p, table, pos_bytes);
    if (st != FA_OK) return st;
    if (T == 0) return FA_OK;
    if ((B > 0 && !slots) || !k || !v || (Hq > 0 && (!q || !q_out)) || (rot > 0 && (!table || !table_len)))
        return FA_ERR_INVALID_ARG;
    if (!aligned(slots, 4) || !aligned(q, 2) || !aligned(q_out, 2) || !aligned(k, 2) || !aligned(v, 2))
        return FA_ERR_INVALID_ARG;
    const cudaError_t err = launch_any<__nv_bfloat16, true>(p, interleaved,
                                                            reinterpret_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
