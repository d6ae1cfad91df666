// paged_q8_list.cuh -- what the kernels of the 8-bit cache's attention share: the requests'
// rows and tiles, and the drafted rows' share of an output.
#pragma once

#include "paged.cuh"
#include "paged_q8.cuh"

namespace vtmu {

// One request: packed rows [row0, row0 + T) are computed, n of them exist (their
// last one is the last row of the cache without a tree), len rows are cached.
struct Q8Req {
    int row0, T, len, n;
};
__device__ __forceinline__ Q8Req q8_load_req(const PagedDesc& a, int b) {
    const PackedRows pr = packed_rows(a.cu_rows, b, a.B, a.rows);
    Q8Req r;
    r.row0 = (int)pr.row0;
    r.n = (int)pr.n;
    r.T = min(r.n, a.max_rows);
    r.len = (int)clamp64(__ldg(a.lens + b), 0, (int64_t)a.max_pages * a.page_size);
    return r;
}

// Its tiles of kt cached keys: those of sinks before the window's range, then the range's.
// Drafted rows have a kernel of their own.
// The range is the request's, from its first row's window to its last row, and counts in full for every row
// block; tiles that causality hides from a whole block are skipped when a CTA gets to them
// (q8_seen_tiles), those before its window are computed for nothing.  So the CTAs' shares are even for trees
// and for a few rows behind a long cache.  A prompt of 4096 rows (32 heads over 8) gives the busiest CTA
// 213 live tiles of 128 keys where an even share is 111, and takes 1.39 ms; one of 8192 with a window of 1024
// walks 66 560 tiles where 17 280 hold a key that is seen, 5.27 ms (2048 rows: 0.38 ms, 4096: 1.41).
struct Q8Units {
    int lo_tile, n_sink, nt;
};
__device__ __forceinline__ Q8Units q8_units(const PagedDesc& a, const Q8Req& r, int kt) {
    Q8Units t;
    int64_t lo = 0;
    if (a.window > 0) lo = clamp64((a.tree ? (int64_t)r.len : (int64_t)r.len - r.n) - a.window + 1, 0, r.len);
    t.lo_tile = (int)(lo / kt);
    const int n_main = lo < r.len ? (int)(((int64_t)r.len + kt - 1) / kt) - t.lo_tile : 0;
    // Where the window leaves nothing of the cache, no main tile holds the sinks of the last one.
    const int64_t sink_tiles = (min(a.sinks, (int64_t)r.len) + kt - 1) / kt;
    t.n_sink = (int)(n_main > 0 ? min(sink_tiles, (int64_t)t.lo_tile) : sink_tiles);
    t.nt = t.n_sink + n_main;
    if (r.T == 0) t.nt = 0;
    else if (t.nt == 0 && !a.tree) t.nt = 1;  // so that the rows are written; a tree's are by then
    return t;
}

// Tiles of a unit whose last row sits at t_last that it sees (no tree: causality hides the others).
__device__ __forceinline__ int q8_seen_tiles(const Q8Req& r, const Q8Units& w, int t_last, int kt) {
    const int p_last = r.len - r.n + t_last;
    const int seen = p_last < 0 ? 0 : p_last / kt + 1 - w.lo_tile;
    return max(w.n_sink + max(seen, 0), 1);
}

// A row's drafted part: its output stands in `out`, its maximum and sum in `ml` [rows][H].
// The weights of a part (m, l, divided by l) beside it, both divided by their sum.
// A part that saw nothing has none (-0, not to be used: its output may be anything); one that
// comes to +0 counts (0 x inf is NaN).
struct Q8Share {
    float own, draft;
};
__device__ __forceinline__ Q8Share q8_share(float m, float l, float2 d) {
    const float top = fmaxf(m, d.x);
    const float a = l != 0.f ? exp2f(m - top) * l : 0.f, b = d.y != 0.f ? exp2f(d.x - top) * d.y : 0.f;
    const float sum = a + b, inv = sum != 0.f ? 1.f / sum : 0.f;
    Q8Share s;
    s.own = l != 0.f ? a * inv : -0.f;
    s.draft = d.y != 0.f ? b * inv : -0.f;
    return s;
}
__device__ __forceinline__ bool q8_nothing(float weight) { return __float_as_uint(weight) == 0x80000000u; }

}  // namespace vtmu
