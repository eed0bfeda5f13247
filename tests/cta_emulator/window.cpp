// The window's geometry and the scheduler's source as the host runs them.
#include "cuda_runtime.h"

struct int2 { int x, y; };
inline int2 make_int2(int x, int y) { return {x, y}; }
inline int atomicMax(int* p, int v) { const int old = *p; *p = max(old, v); return old; }
enum { cudaFuncAttributeMaxDynamicSharedMemorySize = 8 };
template <typename K>
cudaError_t cudaFuncSetAttribute(K, int, int) { return cudaSuccess; }

#define FA_DYNAMIC_SHARED(type, name) static type name[32768]
#include "../../bwd_tiled_attention_gb300/csrc/sched.cu"

namespace fa {
template <int D>
struct FwdCfg {
    static constexpr int kQTiles = D > 128 ? 1 : 2, kUnitRows = kQTiles * kTile;
};
#include "fwd_units.inc"  // UnitGeom and decode_unit, as they stand in fwd.cu
}  // namespace fa

using namespace fa;

extern "C" {
void order_threads(int order, unsigned long long seed) { emu_order(order, seed); }

// out: chunk, sink tiles, far units at most, near rows, rows, offset of the partials, offset of
// the unit list, bytes, units in all at most.
void far_layout(int B, int Hq, int Hkv, int Tq, int Tk, int d, int W, int S, long long* out) {
    const BwdWs lay = bwd_ws_layout(B, Hq, Hkv, Tq, Tk, d);
    const FarWs f = far_ws_layout(lay, B, Hkv, Tq, Tk, d, W, S);
    const long long all[] = {f.chunk, f.tiles, f.max_units, f.near_rows, f.rows, (long long)f.sinks,
                             (long long)f.units, (long long)f.bytes, f.max_units + lay.max_units};
    std::memcpy(out, all, sizeof(all));
}
// The backward's unit list, as its preprocessing writes it; returns the units, or -1 with an error.
int schedule(const int* cu_q, int Nq, int Tq, const int* cu_k, int Nk, int Tk, int B, int H, int d, int det, int W,
             int S, void* ws, int* units, int* tile_off) {
    const BwdWs lay = bwd_ws_layout(B, H, H, Tq, Tk, d);
    FarWs far = {};
    if (S) far = far_ws_layout(lay, B, H, Tq, Tk, d, W, S);
    const size_t at = S ? far.units : lay.units;
    launch_sched(cu_k, B, Nk, Tk, H, kTile, det ? kOrderLevelDesc : kOrderWorkDesc, lay.max_units + far.max_units,
                 ws, at, lay.tile_off, true, cu_q, Nq, Tq, nullptr, far.chunk, W, S);
    const WsHeader* h = static_cast<const WsHeader*>(ws);
    if (h->error) return -1;
    std::memcpy(units, static_cast<char*>(ws) + at, (size_t)h->n_units * 8);
    std::memcpy(tile_off, static_cast<char*>(ws) + lay.tile_off, (size_t)(B + 1) * 4);
    return h->n_units;
}
// Unit (x, y) of the list: sequence, tile, 1 + chunk (0: near), head.
void unit(int x, int y, int sink_tiles, int* out) {
    const int far = x & kFarUnit ? 1 + unit_tile(y) / sink_tiles : 0;
    const int all[] = {x & ~kFarUnit, far ? unit_tile(y) % sink_tiles : unit_tile(y), far, unit_head(y)};
    std::memcpy(out, all, sizeof(all));
}
void span(int j, int far, int C, int L, int Lk, int W, int S, int* out) {
    const WindowSpan s = far ? far_span(j, far - 1, C, L, Lk, W, S) : near_span(j, L, Lk, W);
    out[0] = s.i0;
    out[1] = s.ni;
}
// lo, hi of the 128 keys of a tile within query tile i.
void cols(int j, int far, int i, int L, int Lk, int W, int S, int* lo, int* hi) {
    for (int c = 0; c < kTile; ++c) window_cols(far != 0, j * kTile + c, i, L, Lk, W, S, lo[c], hi[c]);
}
int rank_of(int j, int far, int i, int L, int Lk, int W, int S) { return window_rank(far != 0, j, i, L, Lk, W, S); }
int far_rows_of(int Lk, int W, int S) { return far_rows(Lk, W, S); }
int far_first_of(int j, int C, int L, int Lk, int W, int S) { return far_first(j, C, L, Lk, W, S); }
long long near_place_of(int b, int tk0, int W, int S) { return near_place(b, tk0, W, S); }
long long far_place_of(int b, int t0, int tk0, int C, int W, int S) { return far_place(b, t0, tk0, C, W, S); }
// Forward unit m: n of both tiles, nkv; the walk, who takes part (bits), and the tiles' own walks.
}
template <int D>
void walk_of(const FwdParams& p, int m, int* n, int* steps, int* parts, int* own) {
    const UnitGeom x = decode_unit<D, true, true>(make_int2(0, make_unit_y(m, 0)), p);
    n[0] = x.n[0]; n[1] = x.n[1]; n[2] = x.nkv;
    for (int j = 0; j < x.nkv; ++j) {
        steps[j] = x.template tile<true>(j);
        parts[j] = (x.template active<true>(0, j) ? 1 : 0) | (x.template active<true>(1, j) ? 2 : 0);
    }
    for (int t = 0; t < 2; ++t)
        for (int j = 0; j < x.n[t]; ++j) own[t * 4096 + j] = x.template tile_of<true>(t, j);
}
extern "C" void walk(int m, int qtiles, int L, int Lk, int W, int S, int* n, int* steps, int* parts, int* own) {
    FwdParams p = {};
    p.Hq = p.Hkv = p.B = p.causal = p.kv = 1;
    p.N = p.T = L;
    p.Nk = p.Tk = Lk;
    p.window = W;
    p.sinks = S;
    if (qtiles == 2) walk_of<128>(p, m, n, steps, parts, own);
    else walk_of<256>(p, m, n, steps, parts, own);
}
