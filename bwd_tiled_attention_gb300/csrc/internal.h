// internal.h -- host-side interfaces between the C ABI layer and the kernel
// launchers (not part of the public ABI).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>

#include "../../include/fa.h"

namespace fa {

// Forward kernel arguments (device pointers, tensor maps built on the host).
struct FwdParams {
    CUtensorMap tm_q, tm_k, tm_v;  // 3-D maps over [T, H, d], box {64, 1, 128}
    void* o;
    float* lse;
    const int* cu_seqlens;         // query sequences; null for dense
    void* workspace;               // header + unit list
    size_t units_off;
    int B, Hq, Hkv, N, T, d;       // N, T: query length bound and tokens
    float scale_log2;              // scale * log2(e)
    int causal;
    int o_fp32;
    const int* cu_seqlens_k;       // key/value sequences; null for dense
    int Nk, Tk;                    // key/value length bound and tokens
    int kv;                        // key boundaries differ from the query ones
    int window, sinks;             // window > 0: p sees c <= p with p - c < window or c < sinks
};

struct BwdParams {
    CUtensorMap tm_q, tm_k, tm_v, tm_do;
    CUtensorMap tm_dq_acc;         // fp32 map over the dQ accumulator, box {32, 1, 128}
    const float* lse;
    const float* D;
    void* dk;                      // final dK (MHA) -- bf16 or fp32
    void* dv;
    const int* cu_seqlens;         // query sequences; null for dense
    void* workspace;
    size_t units_off, tile_off_off, sems_off, dq_acc_off, dk_acc_off, dv_acc_off;
    int B, Hq, Hkv, N, T, d;       // N, T: query length bound and tokens
    float scale;                   // softmax scale (dK and dQ factor)
    float scale_log2;              // scale * log2(e)
    int causal;
    int deterministic;
    int grad_fp32;
    int hchunk;                    // query heads one unit walks (bwd_head_run)
    int nchunks;                   // runs of heads per key/value head: (Hq / Hkv) / hchunk
    const int* cu_seqlens_k;       // key/value sequences; null for dense
    int Nk, Tk;                    // key/value length bound and tokens
    int kv;                        // key boundaries differ from the query ones
    int window, sinks;             // window > 0: p sees c <= p with p - c < window or c < sinks
    int far_chunk, sink_tiles;     // query tiles of a far unit, tiles that hold sinks (0: none)
    size_t sink_off;               // fp32 partials of the sinks' dK and dV (window.cuh)
    long long near_rows;           // of them, near units' rows
};

// Writes the unit list over the tiles of `cu_seqlens` / N (T tokens) and,
// when want_tile_off, the per-sequence offsets of the query tiles that
// cu_tiles_seqlens / N_tiles (T_tiles tokens) define (the backward's units
// are key/value tiles, its semaphores query tiles).  Every length is checked
// against its bound and both boundary arrays against their token counts; on a
// mismatch no unit is written and the error word is set.  With sink_tiles > 0
// the far units of a windowed backward come before the others (queries of the other side).
cudaError_t launch_sched(const int* cu_seqlens, int B, int N, int T, int H, int rows, int order,
                         long long max_units, void* workspace, size_t units_off,
                         size_t tile_off_off, bool want_tile_off, const int* cu_tiles_seqlens,
                         int N_tiles, int T_tiles, cudaStream_t stream, int far_chunk = 0,
                         int window = 0, int sinks = 0);

// Dynamic shared memory the scheduler needs for a packed batch of B sequences
// whose longest spans at most maxnt_bound tiles (each of its CTAs ranks them all).
size_t sched_smem_bytes(int B, int maxnt_bound);

cudaError_t launch_fwd(const FwdParams& p, int num_sms, cudaStream_t stream);
cudaError_t launch_fwd_window(const FwdParams& p, int num_sms, cudaStream_t stream);

cudaError_t launch_bwd_preprocess(const void* o, int o_fp32, const void* dout, float* D,
                                  float* dq_acc, int* sems, long long n_sems, int T, int Hq,
                                  int d, int num_sms, cudaStream_t stream);

cudaError_t launch_bwd(const BwdParams& p, int num_sms, cudaStream_t stream);
cudaError_t launch_bwd_window(const BwdParams& p, int num_sms, cudaStream_t stream);

// dK and dV of the sinks from their partials, behind launch_bwd_postprocess.
cudaError_t launch_fold_sinks(const BwdParams& p, int num_sms, cudaStream_t stream);

// dk_acc/dv_acc: fp32 partials [Tk, Hkv * nruns, d] to sum per key/value head,
// or null when each unit wrote final dK/dV.
cudaError_t launch_bwd_postprocess(const float* dq_acc, void* dq, const float* dk_acc,
                                   const float* dv_acc, void* dk, void* dv, int Tq, int Tk,
                                   int Hq, int Hkv, int nruns, int d, float scale, int grad_fp32,
                                   int num_sms, cudaStream_t stream);

// ---- paged cache (cache.cu, rotary.cu, tree.cu)

// Validates a cache descriptor (host side).
fa_status check_cache(const fa_cache* c);

// SMs of the current device (cached), 0 on error.
int device_sms();

constexpr int kTreeMaxCtas = 160;  // CTAs that the attention over the cache runs at most

struct TreeParams {
    CUtensorMap tm_q;              // 4-D {d, group, Hkv, T}, box {64, group, 1, tile_tokens}
    CUtensorMap tm_k, tm_v;        // 3-D {d, page_size, layers * pages * Hkv}, box of one page's keys
    fa_cache cache;
    const int* slots;
    const int* cu;                 // null for a dense batch
    const void* mask;              // int64 [T, words], or null: causal
    void* o;                       // bf16 [T, Hq, d]
    float* lse;                    // [Hq, T]
    int4* meta;                    // per CTA: the item that its first piece ends (not fused)
    unsigned long long* arrived;   // fused: per CTA, partials of the item that ends there
    unsigned long long call;       // fused: this call's number (56 bits)
    int fused;                     // the last CTA of an item joins its partials
    float* part_stats;             // [2 * CTAs, part_rows, 2]: m and l
    float* part_o;                 // not normalised: [2 * CTAs, part_rows, d] if fused,
                                   // else [2 * CTAs, d / 4, part_rows, 4]
    int part_rows;
    int layer, B, N, T, Hq, group;
    int words, page_shift;         // page_size = 1 << page_shift
    int tile_tokens;               // tokens of one 128-row tile
    int min_tiles;                 // least key tiles of a CTA
    int zero_rest;                 // write zeros for tokens that no sequence owns
    int clear_odd;                 // one more slice of the join kernel does so between odd boundaries
    float scale_log2;
    int window, sinks;             // window > 0: p sees key j when p - j < window or j < sinks
    const int* depth;              // tokens' places behind the context, or null: as the mask says
};

// The attention over the cache with a window (tree_window.cu).
cudaError_t launch_tree_window(const TreeParams& p, bool pair, int ctas, cudaStream_t stream);

// The tensor maps of p (api.cu); bn: keys of a tile.
bool make_tree_maps(TreeParams& p, const fa_cache& c, const void* q, int T, int Hq,
                    long long token_stride, long long head_stride, int tile_tokens, int bn);

}  // namespace fa
