// paged_q8_mma.cu -- attention of a few query rows per request over an 8-bit paged
// cache: the step of a serving batch.  headDim 64 or 128.
//
// Mathematics.  For request b and KV head hk the T rows x G heads of the group are
// virtual rows v = t G + g, 8 NT of them a row block.  With codes c and scales s:
//   x2[v, j] = log2 e softcap(scale q_v . ck_j sk_j),  m = running max of x2,
//   l = sum 2^(x2 - m),  o = sum 2^(x2 - m) sv_j cv_j,  out = o / l.
// A code is exact in f16, so q and the weights 2^(x2 - m) sv_j are f16 pairs hi + lo
// (22 bits) and each product takes two f16 MMAs with f32 sums, lo first.  The sums of
// a tile of 32 keys start at zero and are added to the running output outside the tensor
// cores, which round towards zero at every step.
// The weight carries the value's scale, and a large scale may weigh nothing, so the
// output has a reference of its own: o is kept times 2^-(m + r), r an integer per virtual
// row that the largest product 2^(x2 - m) sv sets, and l times 2^-m.  A tile whose scales
// are at most 4 2^r takes one exponential a score; another one takes the exponents of the
// scales into a second exponential and moves r where a product is larger (the first
// tile, and rows of very different size: rare).  m moves when it is beaten by 2^3, so
// a weight is at most 2^5, and has 2^10 as a factor in f16: kept to 2^-35 of the
// largest product.
//
// Work.  A worker is a warp; Hk neighbouring ones (a team) walk the same keys for
// their KV heads, so that a pool row is read whole by warps that run side by side.
// Lengths are known to the device alone: the teams of one wave of CTAs divide the tiles
// of all (request, row block) units evenly.  A unit cut by a team's end leaves
// partials (m, l, o / l) that q8_merge_kernel joins in a fixed order.  Nothing is
// shared between warps but the request table: no barrier after it.
//
// Memory.  A warp keeps kStages tiles of K and V codes and scales in flight by 16-byte
// asynchronous copies, a row index per lane looked up a tile ahead.  Fragments come from
// shared memory 16 bytes a lane: the order of the contraction is free, so a lane takes
// 16 neighbouring channels of a K row (its channels of four k-steps), and of V rows the
// channels that are its rows of the transposed product: O^T = V^T P^T, S^T = K q^T, keys
// and channels fill the 16-row side, 8 virtual rows the other.  P^T changes layout by
// movmatrix.
#include <cstring>

#include "attn_common.cuh"
#include "launch_cache.h"
#include "paged.cuh"
#include "paged_q8.cuh"
#include "paged_q8_mma.cuh"
#include "pdl.cuh"

namespace vtmu {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int kKT = 32;  // keys per tile
constexpr float kLazy = 3.f;     // log2 by which a maximum is beaten before it moves
constexpr float kSlack = 4.f;    // a scale may be this times 2^r
constexpr float kShift = 10.f;   // weights in f16: times 2^10
constexpr float kLeastRef = -116.f;
enum : int { kFirst = 1, kLast = 2, kSlotShift = 2 };  // of a tile; slot + 1 above them

struct MmaArgs {
    PagedDesc a;
    Q8Pools p;
    int32_t page_shift;  // log2 page_size, or -1
    float* part_m;       // [2 teams][Hk][NV]: slot 0 goes on with a unit, slot 1 starts one
    float* part_l;
    float* part_o;       // [2 teams][Hk][NV][D], divided by l
    int4* head;          // [teams]: last team, row block and request of the unit a team starts
};

template <int D, int NT>
struct Cfg {
    static constexpr int kWarps = 8, kStages = 3;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kTileBytes = kKT * D;                      // of K or V
    static constexpr int kStage = 2 * kTileBytes + 2 * kKT * 4 + 16;  // and scales, and what the tile is
    static constexpr size_t smem(int requests) {
        return (size_t)kWarps * kStages * kStage + (size_t)(requests + 1) * 8;
    }
    static_assert(kStage % 16 == 0, "16-byte copies");
};

// ---- the list of tiles: as in the f32 kernel, with 32 keys a tile and the drafted rows'
// tiles behind the cache's ----
struct Req {
    int row0, T, len, n;
};
struct Units {
    int lo_tile, n_sink, n_ctx, nt;
};
__device__ __forceinline__ Req load_req(const PagedDesc& a, int b) {
    const PackedRows pr = packed_rows(a.cu_rows, b, a.B, a.rows);
    Req r;
    r.row0 = (int)pr.row0;
    r.n = (int)pr.n;
    r.T = min(r.n, a.max_rows);
    r.len = (int)clamp64(__ldg(a.lens + b), 0, (int64_t)a.max_pages * a.page_size);
    return r;
}
__device__ __forceinline__ Units units_of(const PagedDesc& a, const Req& r) {
    Units t;
    int64_t lo = 0;
    if (a.window > 0) lo = clamp64((a.tree ? (int64_t)r.len : (int64_t)r.len - r.n) - a.window + 1, 0, r.len);
    t.lo_tile = (int)(lo / kKT);
    const int n_main = lo < r.len ? (int)(((int64_t)r.len + kKT - 1) / kKT) - t.lo_tile : 0;
    const int64_t sink_tiles = (min(a.sinks, (int64_t)r.len) + kKT - 1) / kKT;
    t.n_sink = (int)(n_main > 0 ? min(sink_tiles, (int64_t)t.lo_tile) : sink_tiles);
    t.n_ctx = t.n_sink + n_main;
    t.nt = t.n_ctx + (a.tree ? (r.T + kKT - 1) / kKT : 0);
    if (r.T == 0) t.nt = 0;
    else if (t.nt == 0) t.nt = 1;
    return t;
}

// A tile: first key, or -1 - i for the i-th tile of drafted rows.
struct Tile {
    int b, rb, key, flags;
};

// A team's place in the list; the same in every lane.
template <int NV>
struct Walk {
    long long pos, end, total, teams;
    int b, rb, u, u1, len, lo_tile, n_sink, n_ctx, slot;
    bool first;
    int4 starts;  // the cut unit that this team starts (x < 0: none)

    __device__ void start(const PagedDesc& a, const long long* prefix, int team, int most) {
        total = prefix[a.B];
        teams = max(min((long long)most, total), 1ll);
        pos = team < teams ? total * team / teams : 0;
        end = team < teams ? total * (team + 1) / teams : 0;
        int hi = a.B;
        b = 0;  // the last request whose prefix is at most pos
        while (hi - b > 1) {
            const int mid = (b + hi) >> 1;
            if (prefix[mid] <= pos) b = mid; else hi = mid;
        }
        u = u1 = 0;
        starts = make_int4(-1, 0, 0, 0);
    }
    // The next tile; `empty(slot)` for a piece that causality leaves without one.
    template <class Empty>
    __device__ bool next(const PagedDesc& a, const long long* prefix, Tile& t, Empty empty) {
        while (u >= u1) {
            if (pos >= end) return false;
            while (prefix[b + 1] <= pos) ++b;
            const Req r = load_req(a, b);
            const Units w = units_of(a, r);
            const long long rel = pos - prefix[b], unit = rel / w.nt;
            rb = (int)unit;
            u = (int)(rel - unit * w.nt);
            u1 = (int)min((long long)w.nt, u + (end - pos));
            const long long from = pos - u;
            pos += u1 - u;
            slot = u > 0 ? 0 : u1 < w.nt ? 1 : -1;
            if (slot == 1) starts = make_int4((int)(((from + w.nt) * teams - 1) / total), rb, b, 0);
            if (!a.tree) {  // tiles past the block's last row's position
                const int t_last = (min((rb + 1) * NV, r.T * a.G) - 1) / a.G;
                const int p_last = r.len - r.n + t_last;
                const int seen = p_last < 0 ? 0 : p_last / kKT + 1 - w.lo_tile;
                u1 = min(u1, max(w.n_sink + max(seen, 0), 1));  // a unit has a first tile, so that its rows are written
            }
            len = r.len;
            lo_tile = w.lo_tile;
            n_sink = w.n_sink;
            n_ctx = w.n_ctx;
            first = true;
            if (u >= u1) empty(slot);
        }
        t.b = b;
        t.rb = rb;
        t.key = u < n_ctx ? (u < n_sink ? u : lo_tile + u - n_sink) * kKT : a.tree ? -1 - (u - n_ctx) : 0;
        t.flags = (first ? kFirst : 0) | (u + 1 == u1 ? kLast : 0) | (slot + 1) << kSlotShift;
        first = false;
        ++u;
        return true;
    }
};

// 16-byte chunk c of row `row` of a tile in shared memory.  K: lanes read rows g, g + 1
// side by side, 64 bytes of each; V: rows 2 t, the same two chunks of each.  The order
// makes both free of bank conflicts at headDim 128.
template <int D>
__device__ __forceinline__ int k_chunk(int row, int c) {
    return D == 128 ? c ^ ((row & 1) << 2) : c;
}
template <int D>
__device__ __forceinline__ int v_chunk(int row, int c) {
    return D == 128 ? c ^ (((row >> 1) & 3) << 1) : c ^ ((row >> 1) & 3);
}

template <int D, int NT, int FORM>
__global__ void __launch_bounds__((Cfg<D, NT>::kThreads), 1) q8_mma_kernel(const __grid_constant__ MmaArgs g) {
    using C = Cfg<D, NT>;
    constexpr int NV = 8 * NT, S = C::kStages, CH = D / 16, KC = D / 64, MT = D / 16;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ long long scan_s[C::kWarps];
    const PagedDesc& a = g.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, t4 = lane & 3;
    unsigned char* mine = smem + (size_t)warp * S * C::kStage;
    long long* prefix = reinterpret_cast<long long*>(smem + (size_t)C::kWarps * S * C::kStage);

    pdl_launch_dependents();
    // The requests' tiles and their running sum.
    long long carry = 0;
    for (int b0 = 0; b0 < a.B; b0 += C::kThreads) {
        const int b = b0 + threadIdx.x;
        long long v = 0;
        if (b < a.B) {
            const Req r = load_req(a, b);
            v = ((long long)r.T * a.G + NV - 1) / NV * units_of(a, r).nt;
        }
        long long s = v;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long u = __shfl_up_sync(FULL, s, off);
            if (lane >= off) s += u;
        }
        if (lane == 31) scan_s[warp] = s;
        __syncthreads();
        long long before = carry, all = carry;
        for (int w = 0; w < C::kWarps; ++w) {
            if (w < warp) before += scan_s[w];
            all += scan_s[w];
        }
        if (b < a.B) prefix[b] = before + s - v;
        carry = all;
        __syncthreads();
    }
    if (threadIdx.x == 0) prefix[a.B] = carry;
    __syncthreads();

    const int worker = blockIdx.x * C::kWarps + warp, most = gridDim.x * C::kWarps / a.Hk;
    const int team = worker / a.Hk, hk = worker - team * a.Hk;
    if (team >= most) return;
    Walk<NV> walk;
    walk.start(a, prefix, team, most);
    auto part_row = [&](int slot, int i) -> int64_t { return (((int64_t)2 * team + slot) * a.Hk + hk) * NV + i; };
    auto empty = [&](int slot) {
        if (slot >= 0 && lane < NV) {
            g.part_m[part_row(slot, lane)] = -INFINITY;
            g.part_l[part_row(slot, lane)] = 0.f;
        }
    };

    // ---- loads: a tile's rows are looked up one tile before its copies are issued ----
    Tile ahead;
    bool have = walk.next(a, prefix, ahead, empty);
    int row_ahead = -1;  // pool row of key `lane` of that tile; -1: zeros
    auto look_up = [&]() {
        row_ahead = -1;
        if (!have || ahead.key < 0) return;
        const int key = ahead.key + lane;
        if (key >= walk.len) return;
        const int col = g.page_shift >= 0 ? key >> g.page_shift : key / a.page_size;
        const int page = __ldg(a.block_table + (int64_t)ahead.b * a.max_pages + col);
        if (page >= 0 && page < a.pages) row_ahead = page * a.page_size + (key - col * a.page_size);
    };
    look_up();
    auto issue = [&](int st) {  // the copies of `ahead`, which moves on; one commit in any case
        unsigned char* to = mine + st * C::kStage;
        if (have) {
            const int row = row_ahead;
            if (lane == 0) *reinterpret_cast<Tile*>(to + 2 * C::kTileBytes + 2 * kKT * 4) = ahead;
            if (ahead.key >= 0) {
                constexpr int kLanes = CH, kRows = 32 / CH;  // lanes a row, rows a round
#pragma unroll
                for (int i = 0; i < kKT / kRows; ++i) {
                    const int r = i * kRows + lane / kLanes, c = lane % kLanes;
                    const int from = __shfl_sync(FULL, row, r);
                    const int64_t at = ((int64_t)max(from, 0) * a.Hk + hk) * D + 16 * c;
                    cp_async16(to + r * D + 16 * k_chunk<D>(r, c), g.p.k + at, from >= 0 ? 16 : 0);
                    cp_async16(to + C::kTileBytes + r * D + 16 * v_chunk<D>(r, c), g.p.v + at, from >= 0 ? 16 : 0);
                }
                const int64_t at = (int64_t)max(row, 0) * a.Hk + hk;
                cp_async4(to + 2 * C::kTileBytes + 4 * lane, g.p.k_scale + at, row >= 0 ? 4 : 0);
                cp_async4(to + 2 * C::kTileBytes + 4 * kKT + 4 * lane, g.p.v_scale + at, row >= 0 ? 4 : 0);
            }
            have = walk.next(a, prefix, ahead, empty);
            look_up();
        }
        cp_async_commit();
    };
    int issued = 0;
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
        issued += have;
        issue(i);
    }

    // ---- state of a piece: this lane's virtual rows are 2 t4, 2 t4 + 1 of each eight ----
    uint32_t qf[KC][4][NT][4];  // hi and lo, two registers each, of k-step s of chunk c
    float o[MT][NT][4], m[NT][2], l[NT][2], r[NT][2], unit[NT][2], rf[NT][2];
    int hi[NT][2], lo[NT][2];
    float limit = -1.f;  // a tile whose scales are at most this takes the fast way
    Req rq{};
    int sinks = 0;
    int st = 0, nx = S - 1;
    for (int n = 0; n < issued; ++n, st = st + 1 < S ? st + 1 : 0, nx = nx + 1 < S ? nx + 1 : 0) {
        issued += have;
        issue(nx);
        cp_async_wait<S - 1>();
        __syncwarp();
        const unsigned char* from = mine + st * C::kStage;
        const Tile tile = *reinterpret_cast<const Tile*>(from + 2 * C::kTileBytes + 2 * kKT * 4);
        const float* sks = reinterpret_cast<const float*>(from + 2 * C::kTileBytes);
        const float* svs = sks + kKT;

        if (tile.flags & kFirst) {
            rq = load_req(a, tile.b);
            sinks = (int)min(a.sinks, (int64_t)rq.len);
            limit = -1.f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                // Queries: lane row gr is the virtual row, times qk_mul and a power of two that
                // brings its largest element to [2^13, 2^14).
                const int v = tile.rb * NV + 8 * nt + gr, t = v / a.G;
                const bool alive = v < rq.T * a.G;
                const float* q = a.q + (((int64_t)rq.row0 + t) * a.H + (int64_t)hk * a.G + (v - t * a.G)) * D;
                float top = 0.f;
                float4 y[KC][4];
#pragma unroll
                for (int c = 0; c < KC; ++c)
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (alive) x = __ldg(reinterpret_cast<const float4*>(q + 64 * c + 16 * t4 + 4 * s));
                        x = make_float4(x.x * a.qk_mul, x.y * a.qk_mul, x.z * a.qk_mul, x.w * a.qk_mul);
                        top = fmaxf(fmaxf(fmaxf(top, fabsf(x.x)), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w)));
                        y[c][s] = x;
                    }
                top = fmaxf(top, __shfl_xor_sync(FULL, top, 1));
                top = fmaxf(top, __shfl_xor_sync(FULL, top, 2));
                const float sc = mma_row_scale(top, 13);
#pragma unroll
                for (int c = 0; c < KC; ++c)
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const float4 x = y[c][s];
                        mma_split(x.x * sc, x.y * sc, qf[c][s][nt][0], qf[c][s][nt][2]);
                        mma_split(x.z * sc, x.w * sc, qf[c][s][nt][1], qf[c][s][nt][3]);
                    }
                const float back = 1.f / sc;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    rf[nt][e] = __shfl_sync(FULL, back, 4 * (2 * t4 + e));
                    const int w = tile.rb * NV + 8 * nt + 2 * t4 + e, tw = w / a.G;
                    const bool on = w < rq.T * a.G;
                    int p = a.tree ? rq.len : rq.len - rq.n + tw;
                    if (a.tree && a.window > 0 && on) p = __ldg(a.positions + rq.row0 + tw);
                    // A row of no request sees everything and is not stored.
                    hi[nt][e] = !on ? INT32_MAX : a.tree ? rq.len - 1 : min(p, rq.len - 1);
                    lo[nt][e] = on && a.window > 0 ? (int)max((int64_t)p - a.window + 1, (int64_t)0) : 0;
                    m[nt][e] = -INFINITY;
                    l[nt][e] = 0.f;
                    r[nt][e] = kLeastRef;
                    unit[nt][e] = exp2f(kShift - kLeastRef);
                }
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i][nt][e] = 0.f;
            }
        }

        // ---- scores: x[block of 16 keys][nt]: keys gr (0, 1) and gr + 8 (2, 3), rows 2 t4 and + 1 ----
        float x[2][NT][4];
        float vs[2][2];  // value scales of keys gr, gr + 8
        const float* vrow[2][4];  // drafted value rows
        float vinv[2][4];
        if (tile.key >= 0) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[b][nt][e] = 0.f;
                const int r0 = 16 * b + gr, r1 = r0 + 8;
#pragma unroll
                for (int c = 0; c < KC; ++c) {
                    const uint4 w0 = *reinterpret_cast<const uint4*>(from + r0 * D + 16 * k_chunk<D>(r0, 4 * c + t4));
                    const uint4 w1 = *reinterpret_cast<const uint4*>(from + r1 * D + 16 * k_chunk<D>(r1, 4 * c + t4));
                    const uint32_t a0[4] = {w0.x, w0.y, w0.z, w0.w}, a1[4] = {w1.x, w1.y, w1.z, w1.w};
                    uint32_t f[4][4];
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        q8_halves<FORM>(a0[s], f[s][0], f[s][2]);
                        q8_halves<FORM>(a1[s], f[s][1], f[s][3]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma_16816(x[b][nt], f[s], qf[c][s][nt][2], qf[c][s][nt][3]);
                    }
#pragma unroll
                    for (int s = 0; s < 4; ++s)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma_16816(x[b][nt], f[s], qf[c][s][nt][0], qf[c][s][nt][1]);
                }
                const float ks[2] = {sks[r0], sks[r1]};
                vs[b][0] = svs[r0];
                vs[b][1] = svs[r1];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[b][nt][e] *= ks[e >> 1] * rf[nt][e & 1];
            }
        } else {
            // Drafted rows: f32, as f16 hi + lo after a power of two per row, straight from memory.
            const int d0 = kKT * (-1 - tile.key);
#pragma unroll 1
            for (int b = 0; b < 2; ++b) {
                float xx[NT][4], inv[2], vsc[2], ksc[2];
                const float* kr[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int j = d0 + 16 * b + gr + 8 * h;
                    const int64_t at = ((int64_t)(rq.row0 + min(j, rq.T - 1)) * a.Hk + hk) * D;
                    float top[2];
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        const float* row = (kv ? a.v_new : a.k_new) + at;
                        float tp = 0.f;
                        for (int d = 4 * t4; d < D; d += 16) tp = q8_abs_top(tp, __ldg(reinterpret_cast<const float4*>(row + d)));
                        tp = q8_nan_max(tp, __shfl_xor_sync(FULL, tp, 1));
                        top[kv] = q8_nan_max(tp, __shfl_xor_sync(FULL, tp, 2));
                    }
                    kr[h] = a.k_new + at;
                    const bool kfine = top[0] < INFINITY, vfine = top[1] < INFINITY;
                    inv[h] = kfine ? mma_row_scale(top[0], 8) : 0.f;
                    ksc[h] = kfine ? 1.f / inv[h] : __int_as_float(0x7fc00000);
                    const float vi = vfine ? mma_row_scale(top[1], 8) : 0.f;
                    vsc[h] = vfine ? 1.f / vi : __int_as_float(0x7fc00000);
                    // value rows 2 t4 + e + 8 h, whose scales rows gr = 2 t4 + e know
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float w = __shfl_sync(FULL, vi, 4 * (2 * t4 + e));
                        const int jv = min(d0 + 16 * b + 2 * t4 + e + 8 * h, rq.T - 1);
                        const float* pv = a.v_new + ((int64_t)(rq.row0 + jv) * a.Hk + hk) * D;
                        if (b == 0) {
                            vinv[0][2 * h + e] = w;
                            vrow[0][2 * h + e] = pv;
                        } else {
                            vinv[1][2 * h + e] = w;
                            vrow[1][2 * h + e] = pv;
                        }
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) xx[nt][e] = 0.f;
#pragma unroll
                for (int c = 0; c < KC; ++c)
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        uint32_t fh[4], fl[4];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float4 y = __ldg(reinterpret_cast<const float4*>(kr[h] + 64 * c + 16 * t4 + 4 * s));
                            if (inv[h] == 0.f) y = make_float4(0.f, 0.f, 0.f, 0.f);
                            mma_split(y.x * inv[h], y.y * inv[h], fh[h], fl[h]);
                            mma_split(y.z * inv[h], y.w * inv[h], fh[2 + h], fl[2 + h]);
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma_16816(xx[nt], fh, qf[c][s][nt][2], qf[c][s][nt][3]);
                            mma_16816(xx[nt], fl, qf[c][s][nt][0], qf[c][s][nt][1]);
                            mma_16816(xx[nt], fh, qf[c][s][nt][0], qf[c][s][nt][1]);
                        }
                    }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float y = xx[nt][e] * (ksc[e >> 1] * rf[nt][e & 1]);
                        if (b == 0) x[0][nt][e] = y; else x[1][nt][e] = y;
                    }
                if (b == 0) vs[0][0] = vsc[0], vs[0][1] = vsc[1];
                else vs[1][0] = vsc[0], vs[1][1] = vsc[1];
            }
        }
        if (a.softcap_on) {
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[b][nt][e] = a.cap_log2 * softcap_tanh(x[b][nt][e]);
        }
        // ---- mask: bit (b, nt, e) of `see` ----
        uint32_t see = FULL;
        bool whole = tile.key >= 0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) whole = whole && hi[nt][e] - tile.key >= kKT - 1 && lo[nt][e] <= tile.key;
        if (!__all_sync(FULL, whole)) {
            see = 0;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    uint64_t mask = 0;
                    int p = 0;
                    if (tile.key < 0) {
                        const int w = tile.rb * NV + 8 * nt + 2 * t4 + e, tw = w / a.G;
                        if (w < rq.T * a.G) {
                            mask = __ldg(reinterpret_cast<const unsigned long long*>(a.masks) + rq.row0 + tw);
                            if (a.window > 0) p = __ldg(a.positions + rq.row0 + tw);
                        }
                    }
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int k = 16 * b + gr + 8 * h;
                            bool on;
                            if (tile.key >= 0) {
                                const int key = tile.key + k;
                                on = key <= hi[nt][e] && (key >= lo[nt][e] || key < sinks);
                            } else {
                                const int j = kKT * (-1 - tile.key) + k;
                                on = j < rq.T && ((mask >> (j & 63)) & 1);
                                if (on && a.window > 0) on = (int64_t)__ldg(a.positions + rq.row0 + j) > (int64_t)p - a.window;
                            }
                            if (on) see |= 1u << ((b * NT + nt) * 4 + 2 * h + e);
                        }
                }
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (!((see >> ((b * NT + nt) * 4 + e)) & 1)) x[b][nt][e] = -INFINITY;
        }
        // ---- running maximum ----
        float mt[NT][2];
        bool beaten = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                mt[nt][e] = fmaxf(fmaxf(x[0][nt][e], x[0][nt][2 + e]), fmaxf(x[1][nt][e], x[1][nt][2 + e]));
                beaten = beaten || mt[nt][e] > m[nt][e] + kLazy;
            }
        if (__any_sync(FULL, beaten)) {
            limit = -1.f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float top = mt[nt][e];
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, off));
                    if (top > m[nt][e]) {
                        // m + r, the output's reference, stays: r takes the whole part of the way.
                        const float by = top - m[nt][e];
                        float ref = kLeastRef, alpha = 0.f;
                        if (m[nt][e] != -INFINITY) {
                            ref = fmaxf(r[nt][e] - floorf(by), kLeastRef);
                            alpha = exp2f(-(by - (r[nt][e] - ref)));
                        }
                        l[nt][e] *= exp2f(-by);
                        r[nt][e] = ref;
                        unit[nt][e] = exp2f(kShift - ref);
                        m[nt][e] = top;
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            o[i][nt][e] *= alpha;
                            o[i][nt][2 + e] *= alpha;
                        }
                    }
                }
        }
        // ---- weights, as B fragments: P^T ----
        float tile_top;  // the largest scale: as bits, so that a NaN is the largest
        {
            uint32_t bits = 0;
            if (tile.key >= 0)
                bits = __float_as_uint(svs[lane]) & 0x7fffffffu;
            else
                bits = 0x7fc00000u;  // drafted rows take the slow way
            tile_top = __uint_as_float(__reduce_max_sync(FULL, bits));
        }
        uint32_t ph[2][NT][2], pl[2][NT][2];
        const bool fast = tile_top <= limit;
        float w[2][NT][4];
        if (fast) {
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float mu = m[nt][e & 1] == -INFINITY ? 0.f : m[nt][e & 1];
                        const float p = fast_exp2(x[b][nt][e] - mu);
                        l[nt][e & 1] += p;
                        w[b][nt][e] = p * (vs[b][e >> 1] * unit[nt][e & 1]);
                    }
        } else {
            float lim = INFINITY;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float mu = m[nt][e] == -INFINITY ? 0.f : m[nt][e];
                    auto power = [&](int b, int h) { return (float)((int)((__float_as_uint(vs[b][h]) >> 23) & 255u) - 127); };
                    float top = -INFINITY;
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int h = 0; h < 2; ++h) top = fmaxf(top, (x[b][nt][2 * h + e] - mu) + power(b, h));
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, off));
                    // Products up to 2^(top + 1): r from there, at most the largest exponent.
                    if (top > r[nt][e]) {
                        const float ref = fminf(ceilf(top), 127.f), alpha = exp2f(r[nt][e] - ref);
                        r[nt][e] = ref;
                        unit[nt][e] = exp2f(kShift - ref);
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            o[i][nt][e] *= alpha;
                            o[i][nt][2 + e] *= alpha;
                        }
                    }
                    lim = fminf(lim, kSlack * exp2f(r[nt][e]));
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float y = x[b][nt][2 * h + e] - mu, ex = power(b, h);
                            // The mantissa of the scale (0 stays 0), its exponent in the power.
                            const float f = vs[b][h] * (ex > 0.f ? exp2f(-ex) : exp2f(-ex - 1.f) * 2.f);
                            l[nt][e] += fast_exp2(y);
                            w[b][nt][2 * h + e] = fast_exp2(y + (ex - r[nt][e])) * f * exp2f(kShift);
                        }
                }
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) lim = fminf(lim, __shfl_xor_sync(FULL, lim, off));
            limit = lim;
        }
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    // A scale of a key that is not seen may be anything.
                    const int at = (b * NT + nt) * 4 + 2 * h;
                    const float u = (see >> at) & 1 ? w[b][nt][2 * h] : 0.f, v = (see >> (at + 1)) & 1 ? w[b][nt][2 * h + 1] : 0.f;
                    mma_split(u, v, ph[b][nt][h], pl[b][nt][h]);
                    ph[b][nt][h] = mma_transpose(ph[b][nt][h]);
                    pl[b][nt][h] = mma_transpose(pl[b][nt][h]);
                }
        // ---- O^T += V^T P^T: row gr of product i is channel (D / 8) gr + 2 i, row gr + 8 the next ----
        if (tile.key >= 0) {
            constexpr int W = D / 32;  // words of a lane's channels of one key
            uint32_t vw[2][4][W];
            const unsigned char* vt = from + C::kTileBytes;
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int row = 16 * b + 2 * t4 + (j & 1) + 8 * (j >> 1);
                    if constexpr (D == 128) {
                        const uint4 y = *reinterpret_cast<const uint4*>(vt + row * D + 16 * v_chunk<D>(row, gr));
                        vw[b][j][0] = y.x; vw[b][j][1] = y.y; vw[b][j][2] = y.z; vw[b][j][3] = y.w;
                    } else {
                        const uint2 y = *reinterpret_cast<const uint2*>(vt + row * D + 16 * v_chunk<D>(row, gr >> 1) + 8 * (gr & 1));
                        vw[b][j][0] = y.x; vw[b][j][1] = y.y;
                    }
                }
#pragma unroll
            for (int k = 0; k < W; ++k) {
                uint32_t f[2][2][4];  // product 2 k + i, keys of block b
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    q8_halves2<FORM>(vw[b][0][k], vw[b][1][k], f[0][b][0], f[0][b][1], f[1][b][0], f[1][b][1]);
                    q8_halves2<FORM>(vw[b][2][k], vw[b][3][k], f[0][b][2], f[0][b][3], f[1][b][2], f[1][b][3]);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float acc[4] = {0.f, 0.f, 0.f, 0.f};
                        mma_16816(acc, f[i][0], pl[0][nt][0], pl[0][nt][1]);
                        mma_16816(acc, f[i][1], pl[1][nt][0], pl[1][nt][1]);
                        mma_16816(acc, f[i][0], ph[0][nt][0], ph[0][nt][1]);
                        mma_16816(acc, f[i][1], ph[1][nt][0], ph[1][nt][1]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[2 * k + i][nt][e] += acc[e];
                    }
            }
        } else {
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                float acc[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[nt][e] = 0.f;
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    uint32_t fh[4], fl[4];
                    float2 y[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        y[j] = __ldg(reinterpret_cast<const float2*>(vrow[b][j] + (D / 8) * gr + 2 * i));
                        y[j] = vinv[b][j] == 0.f ? make_float2(0.f, 0.f) : make_float2(y[j].x * vinv[b][j], y[j].y * vinv[b][j]);
                    }
                    mma_split(y[0].x, y[1].x, fh[0], fl[0]);
                    mma_split(y[0].y, y[1].y, fh[1], fl[1]);
                    mma_split(y[2].x, y[3].x, fh[2], fl[2]);
                    mma_split(y[2].y, y[3].y, fh[3], fl[3]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma_16816(acc[nt], fh, pl[b][nt][0], pl[b][nt][1]);
                        mma_16816(acc[nt], fl, ph[b][nt][0], ph[b][nt][1]);
                        mma_16816(acc[nt], fh, ph[b][nt][0], ph[b][nt][1]);
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i][nt][e] += acc[nt][e];
            }
        }
        __syncwarp();  // the stage may be filled again
        // ---- the end of a piece ----
        if (tile.flags & kLast) {
            const int slot = (tile.flags >> kSlotShift) - 1;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float sum = l[nt][e];
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(FULL, sum, off);
                    const float inv = sum != 0.f ? 1.f / sum : 0.f, back = exp2f(r[nt][e] - kShift);
                    const int i = 8 * nt + 2 * t4 + e, v = tile.rb * NV + i, t = v / a.G;
                    float* to;
                    if (slot < 0) {
                        if (v >= rq.T * a.G) continue;
                        to = a.out + (((int64_t)rq.row0 + t) * a.H + (int64_t)hk * a.G + (v - t * a.G)) * D;
                    } else {
                        to = g.part_o + part_row(slot, i) * D;
                        if (gr == 0) {
                            g.part_m[part_row(slot, i)] = m[nt][e];
                            g.part_l[part_row(slot, i)] = sum;
                        }
                    }
                    to += (D / 8) * gr;
#pragma unroll
                    for (int k = 0; k < MT; k += 2)
                        *reinterpret_cast<float4*>(to + 2 * k) =
                            make_float4(o[k][nt][e] * inv * back, o[k][nt][2 + e] * inv * back, o[k + 1][nt][e] * inv * back,
                                        o[k + 1][nt][2 + e] * inv * back);
                }
        }
    }
    cp_async_wait<0>();
    if (hk == 0 && lane == 0) g.head[team] = walk.starts;
}

// Joins the partials of the unit that team blockIdx.x starts: as the f32 kernel's merge.  A
// warp per virtual row of KV head blockIdx.y.
template <int D, int NT>
__global__ void __launch_bounds__(256) q8_merge_kernel(const __grid_constant__ MmaArgs g) {
    constexpr int NV = 8 * NT, kPer = D / 32;
    pdl_wait();
    const PagedDesc& a = g.a;
    const int4 h = __ldcg(&g.head[blockIdx.x]);
    if (h.x < 0) return;
    const int first = blockIdx.x, hk = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rb = h.y, count = h.x - first + 1;
    const Req r = load_req(a, h.z);
    for (int i = warp; i < NV; i += 8) {
        const int v = rb * NV + i;
        if (v >= r.T * a.G) return;
        auto row = [&](int k) -> int64_t {
            return (((int64_t)2 * (first + k) + (k == 0 ? 1 : 0)) * a.Hk + hk) * NV + i;
        };
        auto load = [&](int k) -> float2 {
            return k < count ? make_float2(__ldcg(g.part_m + row(k)), __ldcg(g.part_l + row(k))) : make_float2(-INFINITY, 0.f);
        };
        const float2 own = load(lane);
        float m = own.x;
        for (int k = lane + 32; k < count; k += 32) m = fmaxf(m, __ldcg(g.part_m + row(k)));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, off));
        // -0 where a piece saw nothing and left no output; +0 counts (0 x inf is NaN).
        auto weight = [&](float2 p) -> float { return p.y != 0.f ? fast_exp2(p.x - m) * p.y : -0.f; };
        float den = weight(own);
        for (int k = lane + 32; k < count; k += 32) den += weight(load(k));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) den += __shfl_xor_sync(FULL, den, off);
        const float inv = den != 0.f ? 1.f / den : 0.f;
        float acc[kPer];
#pragma unroll
        for (int c = 0; c < kPer; ++c) acc[c] = 0.f;
        for (int k0 = 0; k0 < count; k0 += 32) {
            const float wgt = weight(k0 == 0 ? own : load(k0 + lane)) * inv;
            const int here = min(count - k0, 32);
            for (int k = 0; k < here; ++k) {
                const float f = __shfl_sync(FULL, wgt, k);
                if (__float_as_uint(f) == 0x80000000u) continue;
                const float* src = g.part_o + row(k0 + k) * D;
#pragma unroll
                for (int c = 0; c < kPer; ++c) acc[c] = fmaf(f, __ldcg(src + lane + 32 * c), acc[c]);
            }
        }
        float* out = a.out + (((int64_t)r.row0 + v / a.G) * a.H + (int64_t)hk * a.G + v % a.G) * D;
#pragma unroll
        for (int c = 0; c < kPer; ++c) out[lane + 32 * c] = acc[c];
    }
}

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

// Row blocks of 8 virtual rows where they hold a request's, else 16.
int blocks_of(const PagedDesc& a) { return (int64_t)a.max_rows * a.G <= 8 ? 1 : 2; }
constexpr int kMmaWarps = 8;

struct Scratch {
    size_t m, l, o, head, total;
};
int ctas_of(int sms, int Hk) {
    const int need = (Hk + kMmaWarps - 1) / kMmaWarps, n = sms < kPagedMaxCtas ? sms : kPagedMaxCtas;
    return n < need ? need : n;
}
Scratch scratch_of(int ctas, int Hk, int NV, int D) {
    const size_t teams = (size_t)ctas * kMmaWarps / Hk, rows = 2 * teams * Hk * NV;
    Scratch s;
    s.m = kWorkspaceHeader;
    s.l = s.m + up256(rows * 4);
    s.o = s.l + up256(rows * 4);
    s.head = s.o + up256(rows * D * 4);
    s.total = s.head + up256(teams * sizeof(int4));
    return s;
}

template <int D, int NT, int FORM>
cudaError_t launch_form(const MmaArgs& g, int ctas, cudaStream_t stream) {
    using C = Cfg<D, NT>;
    static_assert(C::kWarps == kMmaWarps, "the workspace counts them");
    auto kern = q8_mma_kernel<D, NT, FORM>;
    cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kern), (int)C::smem(kPagedMaxRequests));
    if (e != cudaSuccess) return e;
    kern<<<ctas, C::kThreads, C::smem(g.a.B), stream>>>(g);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_pdl(q8_merge_kernel<D, NT>, dim3((unsigned)(ctas * C::kWarps / g.a.Hk), (unsigned)g.a.Hk), dim3(256), 0,
                      stream, g);
}
template <int D, int NT>
cudaError_t launch_nt(const MmaArgs& g, int ctas, cudaStream_t stream) {
    return g.p.form == kFormInt8 ? launch_form<D, NT, kFormInt8>(g, ctas, stream)
                                 : launch_form<D, NT, kFormE4m3>(g, ctas, stream);
}

}  // namespace

bool paged_q8_mma_supported(const PagedDesc& a) {
    return (a.D == 64 || a.D == 128) && a.pages > 0 && (int64_t)a.max_rows * a.G < ((int64_t)1 << 30);
}

size_t paged_q8_mma_workspace(const PagedDesc& a) {
    return scratch_of(ctas_of(kPagedMaxCtas, a.Hk), a.Hk, 8 * blocks_of(a), a.D).total;
}

cudaError_t launch_paged_q8_mma(const PagedDesc& a, const Q8Pools& p, int num_sms, void* workspace, cudaStream_t stream) {
    MmaArgs g;
    std::memset(&g, 0, sizeof(g));
    g.a = a;
    g.p = p;
    g.page_shift = -1;
    for (int i = 0; i < 31; ++i)
        if (a.page_size == 1 << i) g.page_shift = i;
    const int ctas = ctas_of(num_sms, a.Hk), nt = blocks_of(a);
    const Scratch s = scratch_of(ctas, a.Hk, 8 * nt, a.D);
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    g.part_m = reinterpret_cast<float*>(ws + s.m);
    g.part_l = reinterpret_cast<float*>(ws + s.l);
    g.part_o = reinterpret_cast<float*>(ws + s.o);
    g.head = reinterpret_cast<int4*>(ws + s.head);
    if (a.D == 128) return nt == 1 ? launch_nt<128, 1>(g, ctas, stream) : launch_nt<128, 2>(g, ctas, stream);
    return nt == 1 ? launch_nt<64, 1>(g, ctas, stream) : launch_nt<64, 2>(g, ctas, stream);
}

}  // namespace vtmu
