// window.cuh -- geometry of the backward within a sliding window of W keys and S first ones
// (sinks): its units, masks, ranks and partials.  Whole numbers only, and callable from the
// host.  (The forward's is in fwd.cu: calls out of here cost it 1% at 32768 tokens, W = 4096.)
//
// The query at row r of a sequence with L queries and Lk keys stands at p = r + Lk - L and
// sees key c <= p when p - c < W or c < S.
#pragma once
#include "common.cuh"

namespace fa {

#define FA_HD __host__ __device__ __forceinline__

// A unit of key/value tile j (near) walks the query tiles whose window reaches it, under
// the window's mask alone.  The pairs of sinks and rows further on are far units, of a tile
// of sinks and a chunk of C query tiles.  Sinks [0, far_rows) have such pairs.
FA_HD int far_rows(int Lk, int W, int S) { return max(0, min(S, Lk - W)); }

struct WindowSpan {
    int i0, ni;  // query tiles [i0, i0 + ni)
};
// Rows r with c - off <= r < c - off + W for a key c of tile j.
FA_HD WindowSpan near_span(int j, int L, int Lk, int W) {
    const int c0 = j * kTile, off = Lk - L;
    const int i0 = max(0, floor_div(c0 - off, kTile));
    const int i1 = min(cdiv(L, kTile), floor_div(min(c0 + kTile, Lk) - 2 + W - off, kTile) + 1);
    return {i0, max(0, i1 - i0)};
}
// Rows r >= c - off + W, of chunk q, for a sink c of tile j.
FA_HD WindowSpan far_span(int j, int q, int C, int L, int Lk, int W, int S) {
    const int c0 = j * kTile;
    const int i0 = max(q * C, floor_div(c0 + W - (Lk - L), kTile));
    const int i1 = c0 < far_rows(Lk, W, S) ? min(cdiv(L, kTile), (q + 1) * C) : i0;
    return {i0, max(0, i1 - i0)};
}

// Chunks [first, all) of a sequence have far rows for the sinks of tile j (none: first = all).
FA_HD int far_all(int C, int L) { return cdiv(cdiv(L, kTile), C); }
FA_HD int far_first(int j, int C, int L, int Lk, int W, int S) {
    if (j * kTile >= far_rows(Lk, W, S)) return far_all(C, L);
    return min(far_all(C, L), max(0, floor_div(j * kTile + W - (Lk - L), kTile)) / C);
}

// Visible query columns [lo, hi), within query tile i, of key c of a near or far unit.
FA_HD void window_cols(bool far, int c, int i, int L, int Lk, int W, int S, int& lo, int& hi) {
    const int r = c - (Lk - L);  // the key's own row
    const int from = far ? r + W : r;
    const int to = far ? (c < min(S, Lk) ? L : 0) : (c < Lk ? min(L, r + W) : 0);
    lo = max(0, from - i * kTile);
    hi = min(kTile, to - i * kTile);
}

// Rank of a unit's contribution to dQ tile i: the far units' come first, and of either kind in
// descending tile.  Sink tiles [0, before) have far rows in query tile i.
FA_HD int window_rank(bool far, int j, int i, int L, int Lk, int W, int S) {
    const int off = Lk - L;
    const int last = min((i + 1) * kTile, L) - 1 + off;  // the tile's last position
    const int before = max(0, min(cdiv(min(S, Lk), kTile), floor_div(last - W, kTile) + 1));
    if (far) return before - 1 - j;
    return before + min(cdiv(Lk, kTile) - 1, floor_div((i + 1) * kTile + off - 1, kTile)) - j;
}

// Both kinds leave fp32 partials of dK and dV of the sinks that have far rows, R = far_rows of a
// sequence: R rows of its near units, and R of each chunk.  Where they begin must keep
// sequences apart without a sum over those before, and within what they hold: a place that
// grows from a sequence to the next by what the sequence needs at least.
//   near: min(b S, tk0, tk0 / (W + 1) S) does, as R <= S, R <= Lk, and R = 0 where Lk <= W;
//   far: ceil(L / (128 C)) R rows <= floor(L / (128 C)) S + R, so t0 / (128 C) S + the former.
// t0, tk0: the sequence's first query and key.
FA_HD long long near_place(int b, int tk0, int W, int S) {
    long long x = (long long)b * S;
    const long long y = tk0 / (W + 1) * (long long)S;
    if (tk0 < x) x = tk0;
    return y < x ? y : x;
}
FA_HD long long far_place(int b, int t0, int tk0, int C, int W, int S) {
    return (long long)(t0 / (kTile * C)) * S + near_place(b, tk0, W, S);
}

// Chunks that far units of one tile of sinks have, at most, over all sequences.
FA_HD long long far_chunks(int B, int Tq, int Tk, int C, int W) {
    return Tq / (kTile * C) + min(B, Tk / (W + 1));
}

// Backward workspace of a window with sinks: that of the plain call (w), the partials [rows, 2,
// Hkv * runs, d], and a longer unit list, whose far units -- x carries kFarUnit, the tile field is
// chunk * sink tiles + sink tile -- come first.  C is 16 tiles, so that a far unit is about as
// long as one of a window of 2000 keys, or as many as there are sink tiles.  So there are
// at most Tq + 2 Tk rows of partials, however the batch is cut, and far fewer where few are sinks.
constexpr int kFarUnit = 1 << 30;
constexpr int kFarChunk = 16;

struct FarWs {
    int chunk, tiles;      // query tiles of a far unit, sink tiles
    long long max_units;   // far units, at most
    long long near_rows, rows;   // of partials: near units', and in all
    size_t sinks, units, bytes;  // offsets of the partials and of the unit list, workspace in all
};

__host__ __device__ inline FarWs far_ws_layout(const BwdWs& w, int B, int Hkv, int Tq, int Tk, int d, int W,
                                               int S) {
    FarWs f;
    f.tiles = cdiv(S, kTile);
    f.chunk = f.tiles > kFarChunk ? f.tiles : kFarChunk;
    f.max_units = far_chunks(B, Tq, Tk, f.chunk, W) * f.tiles * Hkv * w.nruns;
    f.near_rows = near_place(B, Tk, W, S);
    f.rows = f.near_rows + far_place(B, Tq, Tk, f.chunk, W, S);
    f.sinks = w.bytes;
    f.units = align_up(f.sinks + (size_t)f.rows * 2 * Hkv * w.nruns * (size_t)d * 4, kAlign);
    f.bytes = align_up(f.units + (size_t)(w.max_units + f.max_units) * 8, kAlign);
    return f;
}

}  // namespace fa
