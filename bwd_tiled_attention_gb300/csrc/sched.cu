// sched.cu -- on-device tile scheduler metadata.
//
// "FlashAttention-4反向传播优化" section 3.3.2: for variable-length batches a
// preprocessing kernel sorts the sequences by their per-tile work, writes a
// virtual-to-actual index mapping, and the attention kernel walks the work in
// that order (longest processing time first).  Section 3.3.1: for the
// deterministic causal backward, key/value blocks are launched in descending
// order (shortest processing time first).  Section 5.2: query heads that share
// a key/value head are walked together.
//
// A CTA reads cu_seqlens (or the dense length N), ranks the sequences by
// tile count (descending, ties by index), and writes the ordered list of work
// units (sequence, tile, head) into the workspace, heads innermost.  The
// attention kernels take units from that list through an atomic counter that
// this kernel resets, so CTAs that finish early pick up the next unit.  The
// backward's units are key/value tiles while its dQ semaphores are per query
// tile, so it also passes the query boundaries, from which this kernel writes
// the per-sequence query-tile offsets; both sides' lengths are checked against
// their bounds.
#include <cuda_runtime.h>

#include "common.cuh"
#include "internal.h"
#include "window.cuh"

#ifndef FA_DYNAMIC_SHARED
#define FA_DYNAMIC_SHARED(type, name) extern __shared__ type name[]
#endif

namespace fa {

constexpr int kSchedThreads = 1024;

struct SchedArgs {
    const int* cu_seqlens;  // device int32[B+1] or null (dense): the unit tiles
    const int* cu_aux;      // the other side's boundaries (null when dense)
    int B, N, H, rows;      // rows per tile
    int T;                  // tokens on the unit side (cu_seqlens[B] must equal it)
    int N_aux, T_aux;       // bound on the other side's lengths, its tokens
    int order;              // SchedOrder
    int max_units;          // capacity of the unit list
    WsHeader* header;
    int2* units;
    int* tile_off;          // int[B+1] offsets of the other side's tiles (may be null)
    int far_chunk, window, sinks;  // far units of a windowed backward (sinks = 0: none)
};

// Number of sequences whose tile count exceeds m, given counts sorted descending.
__device__ __forceinline__ int count_above(const int* nt_sorted, int B, int m) {
    int lo = 0, hi = B;  // first index with nt <= m
    while (lo < hi) {
        int mid = (lo + hi) >> 1;
        if (nt_sorted[mid] > m) lo = mid + 1; else hi = mid;
    }
    return lo;
}

// Largest index i in [0, n) with prefix[i] <= u (prefix non-decreasing, prefix[0] = 0).
__device__ __forceinline__ int find_slot(const long long* prefix, int n, long long u) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= u) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// FAR: with far units.  (A kernel of its own: their arithmetic, although not run, made the
// forward's schedule of 1024 units 6 us longer.)
template <bool FAR>
__global__ void __launch_bounds__(kSchedThreads) sched_kernel(SchedArgs a) {
    pdl_begin();
    FA_DYNAMIC_SHARED(long long, sm64);
    unsigned char* sm = reinterpret_cast<unsigned char*>(sm64);
    const int tid = threadIdx.x;
    const int B = a.B, H = a.H;
    // Every CTA ranks the sequences and writes its share of the list, the first one the rest.
    const long long at = (long long)blockIdx.x * kSchedThreads + tid;
    const long long step = (long long)gridDim.x * kSchedThreads;
    __shared__ long long s_total;
    __shared__ int s_maxnt, s_bad, s_maxfar;
    __shared__ long long s_sums[kSchedThreads / 32 + 1];
    const int sink_tiles = FAR ? cdiv(a.sinks, kTile) : 0;
    // (far units come in descending tile of sinks, as a deterministic dQ tile takes them, then by
    // sequence and chunk, heads innermost; only those that have rows are listed)

    if (a.cu_seqlens == nullptr) {
        // Dense batch: every sequence has nt tiles; closed-form order.
        const int nt = cdiv(a.N, a.rows);
        const int nt_aux = cdiv(a.N_aux, a.rows);
        const long long per_level = (long long)B * H;
        const int all = FAR ? far_all(a.far_chunk, a.N_aux) : 0;  // chunks of one sequence
        long long far = 0;
        if constexpr (FAR)
            for (int j = 0; j < sink_tiles; ++j)
                far += per_level * (all - far_first(j, a.far_chunk, a.N_aux, a.N, a.window, a.sinks));
        const long long total = far + per_level * nt;
        if (at == 0) {
            a.header->n_units = (int)(total <= a.max_units ? total : 0);
            a.header->counter = 0;
            a.header->error = total <= a.max_units ? 0 : kErrSchedule;
            a.header->n_qtiles = B * nt_aux;
        }
        if (total > a.max_units) return;
        if constexpr (FAR) {
            int2* out = a.units;
            for (int j = sink_tiles - 1; j >= 0; --j) {
                const int first = far_first(j, a.far_chunk, a.N_aux, a.N, a.window, a.sinks);
                const int some = all - first;
                for (long long u = at; u < per_level * some; u += step) {
                    const int h = (int)(u % H), b = (int)(u / H / some), q = first + (int)(u / H % some);
                    out[u] = make_int2(b | kFarUnit, make_unit_y(q * sink_tiles + j, h));
                }
                out += per_level * some;
            }
        }
        for (long long u = at; u < total - far; u += step) {
            int b, tile, h;
            if (a.order == kOrderSeqDesc) {
                b = (int)(u / ((long long)nt * H));
                long long r = u % ((long long)nt * H);
                tile = (int)(r / H);
                h = (int)(r % H);
            } else {
                const int lvl = (int)(u / per_level);
                const long long r = u % per_level;
                b = (int)(r / H);
                h = (int)(r % H);
                tile = (a.order == kOrderLevelDesc) ? nt - 1 - lvl : lvl;
            }
            a.units[far + u] = make_int2(b, make_unit_y(tile, h));
        }
        if (a.tile_off)
            for (long long b = at; b <= B; b += step) a.tile_off[b] = (int)b * nt_aux;
        return;
    }

    // Variable-length batch.
    int* nt_of = reinterpret_cast<int*>(sm);           // [B] tile count per sequence
    int* sorted = nt_of + B;                           // [B] sequence at rank r
    int* nt_sorted = sorted + B;                       // [B] tile count at rank r
    long long* prefix = reinterpret_cast<long long*>(  // [max(B, maxnt) + 1]
        sm + align_up((size_t)3 * B * sizeof(int), 16));
    if (tid == 0) {
        s_maxnt = s_maxfar = 0;
        // the boundaries must span exactly the tokens the buffers hold
        s_bad = a.cu_seqlens[0] != 0 || a.cu_seqlens[B] != a.T ||
                (a.cu_aux && (a.cu_aux[0] != 0 || a.cu_aux[B] != a.T_aux));
    }
    __syncthreads();
    for (int b = tid; b < B; b += kSchedThreads) {
        const int L = a.cu_seqlens[b + 1] - a.cu_seqlens[b];
        if (L < 0 || L > a.N) atomicOr(&s_bad, 1);  // N bounds every length
        if (a.cu_aux) {
            const int La = a.cu_aux[b + 1] - a.cu_aux[b];
            if (La < 0 || La > a.N_aux) atomicOr(&s_bad, 1);
            if (FAR && La > 0) atomicMax(&s_maxfar, far_rows(L, a.window, a.sinks));
        }
        const int nt = L > 0 ? cdiv(L, a.rows) : 0;
        nt_of[b] = nt;
        atomicMax(&s_maxnt, nt);
    }
    __syncthreads();
    if (s_bad) {
        if (at == 0) {
            a.header->n_units = 0;
            a.header->counter = 0;
            a.header->error = kErrSchedule;
            a.header->n_qtiles = 0;
        }
        return;
    }
    // rank by tile count descending, ties by index
    for (int b = tid; b < B; b += kSchedThreads) {
        const int nb = nt_of[b];
        int rank = 0;
        for (int o = 0; o < B; ++o) {
            const int no = nt_of[o];
            rank += (no > nb) || (no == nb && o < b);
        }
        sorted[rank] = b;
        nt_sorted[rank] = nb;
    }
    __syncthreads();
    const int maxnt = s_maxnt;
    long long far = 0;  // far units
    if constexpr (FAR) {
        const int each = cdiv(B, kSchedThreads);
        const int b0 = min(B, tid * each), b1 = min(B, b0 + each);
        for (int j = cdiv(s_maxfar, kTile) - 1; j >= 0; --j) {
            // chunks of sequence b with rows for tile j
            auto first = [&](int b, int& all) {
                const int L = a.cu_aux[b + 1] - a.cu_aux[b], Lk = a.cu_seqlens[b + 1] - a.cu_seqlens[b];
                all = far_all(a.far_chunk, L);
                return far_first(j, a.far_chunk, L, Lk, a.window, a.sinks);
            };
            long long mine = 0, total;
            int all;
            for (int b = b0; b < b1; ++b) {
                prefix[b] = mine;
                const int q0 = first(b, all);
                mine += all - q0;
            }
            const long long before = block_scan(mine, s_sums, total);
            for (int b = b0; b < b1; ++b) prefix[b] += before;
            __syncthreads();
            if (far + total * H <= a.max_units)
                for (long long u = at; u < total * H; u += step) {
                    const int b = find_slot(prefix, B, u / H);
                    const int q = first(b, all) + (int)(u / H - prefix[b]);
                    a.units[far + u] = make_int2(b | kFarUnit, make_unit_y(q * sink_tiles + j, (int)(u % H)));
                }
            far += total * H;
            __syncthreads();  // (prefix has been read)
        }
    }
    int nslots;
    if (a.order == kOrderSeqDesc) {
        nslots = B;
        if (tid == 0) {
            long long acc = 0;
            for (int r = 0; r < B; ++r) { prefix[r] = acc; acc += (long long)nt_sorted[r] * H; }
            prefix[B] = acc;
            s_total = acc;
        }
    } else {
        nslots = maxnt;
        if (tid == 0) {
            long long acc = 0;
            for (int l = 0; l < maxnt; ++l) {
                prefix[l] = acc;
                acc += (long long)count_above(nt_sorted, B, maxnt - 1 - l) * H;
            }
            prefix[maxnt] = acc;
            s_total = acc;
        }
    }
    __syncthreads();
    const long long total = far + s_total;
    if (at == 0) {
        a.header->n_units = (int)(total <= a.max_units ? total : 0);
        a.header->counter = 0;
        a.header->error = total <= a.max_units ? 0 : kErrSchedule;
    }
    if (a.tile_off && at == 0) {
        int acc = 0;
        for (int b = 0; b < B; ++b) {
            a.tile_off[b] = acc;
            acc += cdiv(a.cu_aux[b + 1] - a.cu_aux[b], a.rows);
        }
        a.tile_off[B] = acc;
        a.header->n_qtiles = acc;
    } else if (at == 0) {
        a.header->n_qtiles = 0;
    }
    if (total > a.max_units || nslots == 0) return;
    for (long long u = at; u < total - far; u += step) {
        const int slot = find_slot(prefix, nslots, u);
        const long long r = u - prefix[slot];
        int b, tile;
        const int h = (int)(r % H);
        if (a.order == kOrderSeqDesc) {
            b = sorted[slot];
            tile = (int)(r / H);
        } else {
            const int rank = (int)(r / H);
            b = sorted[rank];
            const int m = maxnt - 1 - slot;   // sequences of this level have nt > m
            tile = (a.order == kOrderLevelDesc) ? m : nt_of[b] - 1 - m;
        }
        a.units[far + u] = make_int2(b, make_unit_y(tile, h));
    }
}

size_t sched_smem_bytes(int B, int maxnt_bound) {
    const int slots = (B > maxnt_bound ? B : maxnt_bound) + 1;
    return align_up((size_t)3 * B * sizeof(int), 16) + (size_t)slots * sizeof(long long);
}

cudaError_t launch_sched(const int* cu_seqlens, int B, int N, int T, int H, int rows, int order,
                         long long max_units, void* workspace, size_t units_off,
                         size_t tile_off_off, bool want_tile_off, const int* cu_tiles_seqlens,
                         int N_tiles, int T_tiles, cudaStream_t stream, int far_chunk,
                         int window, int sinks) {
    SchedArgs a;
    a.far_chunk = far_chunk;
    a.window = window;
    a.sinks = sinks;
    a.cu_seqlens = cu_seqlens;
    a.cu_aux = cu_tiles_seqlens;
    a.T = T;
    a.N_aux = N_tiles;
    a.T_aux = T_tiles;
    a.B = B;
    a.N = N;
    a.H = H;
    a.rows = rows;
    a.order = order;
    a.max_units = (int)(max_units > 0x7FFFFFFF ? 0x7FFFFFFF : max_units);
    a.header = reinterpret_cast<WsHeader*>(workspace);
    a.units = reinterpret_cast<int2*>(static_cast<char*>(workspace) + units_off);
    a.tile_off = want_tile_off ? reinterpret_cast<int*>(static_cast<char*>(workspace) + tile_off_off)
                               : nullptr;
    size_t smem = 0;
    auto kern = sinks ? sched_kernel<true> : sched_kernel<false>;
    if (cu_seqlens) {
        smem = sched_smem_bytes(B, cdiv(N, rows));
        cudaError_t e = cudaFuncSetAttribute(kern,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)smem);
        if (e != cudaSuccess) return e;
    }
    // (16 packed sequences of 256-8192 tokens, 16 heads: one CTA -> up to 16, forward 1289.5 ->
    // 1286.8 us, the backward's preparation 179.3 -> 175.0)
    const int ctas = max_units <= 2 * kSchedThreads ? 1 : (int)(max_units < 16 * kSchedThreads
                                                                    ? cdiv((int)max_units, kSchedThreads) : 16);
    return launch_pdl(kern, dim3(ctas), dim3(kSchedThreads), smem, stream, a);
}

}  // namespace fa
