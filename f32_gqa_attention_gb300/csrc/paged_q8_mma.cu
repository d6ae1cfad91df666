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
// Work.  Lengths are known to the device alone, so the launch is one persistent CTA per
// SM, and the CTAs divide the tiles of all (request, head block, row block) units
// evenly (each unit counted with its request's whole range: paged_q8_list.cuh).  A tile is
// 32 keys for each of kg key groups, hb KV heads wide (all of them up to eight), hb kg <= 8: a
// consumer warp per head and key group, which shares nothing with the others until the piece ends.  A CTA so reads whole rows of the pool; with a worker
// per head that loaded its own 128 bytes of each row, the heads drifted apart and HBM
// gave 3.2 TB/s.  Key groups are joined inside the CTA; a unit cut by a CTA's end leaves
// partials (m, l, o / l) that q8_merge_kernel joins in a fixed order: no atomics.
//
// Memory.  Producer warps look up pages and copy rows and scales kStages tiles ahead, in
// 16-byte asynchronous copies: 6.2 TB/s with nothing else to do, where bulk copies of a row
// (1 KB) gave 4.5 TB/s, of a head (128 bytes) 0.7, and only whole pages 6.3.  Consumers
// read fragments 16 bytes a lane: the order of the contraction is free, so a lane takes
// 16 neighbouring channels of a K row (its channels of four k-steps), and of V rows the
// channels that are its rows of the transposed product: S^T = K q^T, O^T = V^T P^T, keys and
// channels fill the 16-row side, 8 virtual rows the other.  P^T changes layout by movmatrix.
// Every wait is bounded; one that gives up sets a bit of the device flag.
//
// Measured (a replayed graph): 24 requests of 8192 to 32704 rows, 32 heads over 8 of 128, e4m3
// (1.08 GB) 177 us, 91 % of the copy rate; 32 of 517 to 8111, int8 (304 MB) 71 us, 64 %: of 24 us
// above the copy's the launches, the scan of the requests, the first loads and the join take most.
#include <cstring>

#include "attn_common.cuh"
#include "launch_cache.h"
#include "paged_q8_list.cuh"
#include "paged_q8_mma.cuh"
#include "pdl.cuh"
#include "softcap.cuh"
#include "tma_sync.cuh"

namespace vtmu {

__device__ unsigned int g_q8_device_error;

namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int kKT = 32;  // keys of a warp's tile
constexpr float kLazy = 3.f;     // log2 by which a maximum is beaten before it moves
constexpr float kSlack = 4.f;    // a scale may be this times 2^r
constexpr float kShift = 10.f;   // weights in f16: times 2^10
constexpr float kLeastRef = -116.f;

struct MmaArgs {
    PagedDesc a;
    Q8Pools p;
    int32_t page_shift;  // log2 page_size, or -1
    int32_t hb, blocks;  // heads of a block, head blocks
    int32_t kg;          // key groups
    int32_t wide;        // four scales of a row may be one copy
    int32_t stage;       // bytes of one
    float* part_m;       // [3 CTAs][8 warps][NV]: slot 0 goes on with a unit, slot 1 starts one, 2: key groups
    float* part_l;
    float* part_o;       // [3 CTAs][8 warps][NV][D], divided by l
    const float2* draft; // [rows][H]: maximum and sum over the drafted rows, whose output is in a.out
    int4* head;          // [2 CTAs]: the unit a CTA starts: last CTA, virtual rows [y, z), first packed row; first head
};

// A tile in shared memory: K rows, V rows, scales [row][head] of K and of V, what it is.
constexpr int kConsumers = 8;  // at most
constexpr int kProducers = 4;
constexpr int kStages = 3, kThreads = 32 * (kConsumers + kProducers);
constexpr size_t kSmemMost = 232448 - 1024;  // less the static part

enum : unsigned int {
    kErrQ8Load = 1u << 3,  // the paged kernels' bits: a tile that did not come,
    kErrQ8Free = 1u << 4,  // a stage that was not given back
};

// A tile: its first key.
struct Tile {
    int b, rb, key, flags;
};
enum : int { kFirst = 1, kLast = 2, kStop = 4, kSlotShift = 3, kBlockShift = 5 };  // flags; slot + 1, head block above them

// A CTA's place in the list; the same in every lane of the producer.
template <int NV>
struct Walk {
    long long pos, end, total, ctas;
    int kt;  // keys of a tile
    int b, rb, hblock, u, u1, len, lo_tile, n_sink, slot;
    bool first;
    int4 starts;  // the cut unit that this CTA starts (x < 0: none)
    int starts_block;

    __device__ void start(const MmaArgs& g, const long long* prefix) {
        const PagedDesc& a = g.a;
        kt = 32 * g.kg;
        total = prefix[a.B];
        ctas = max(min((long long)gridDim.x, total), 1ll);
        const int c = blockIdx.x;
        pos = c < ctas ? total * c / ctas : 0;
        end = c < ctas ? total * (c + 1) / ctas : 0;
        int hi = a.B;
        b = 0;  // the last request whose prefix is at most pos
        while (hi - b > 1) {
            const int mid = (b + hi) >> 1;
            if (prefix[mid] <= pos) b = mid; else hi = mid;
        }
        u = u1 = 0;
        starts = make_int4(-1, 0, 0, 0);
        starts_block = 0;
    }
    // The next tile; `empty(slot)` for a piece that causality leaves without one.
    template <class Empty>
    __device__ bool next(const MmaArgs& g, const long long* prefix, Tile& t, Empty empty) {
        const PagedDesc& a = g.a;
        while (u >= u1) {
            if (pos >= end) return false;
            while (prefix[b + 1] <= pos) ++b;
            const Q8Req r = q8_load_req(a, b);
            const Q8Units w = q8_units(a, r, kt);
            const long long rel = pos - prefix[b], unit = rel / w.nt;
            const int rows = (r.T * a.G + NV - 1) / NV;  // row blocks
            hblock = (int)(unit / rows);
            rb = (int)(unit - (long long)hblock * rows);
            u = (int)(rel - unit * w.nt);
            u1 = (int)min((long long)w.nt, u + (end - pos));
            const long long from = pos - u;
            pos += u1 - u;
            slot = u > 0 ? 0 : u1 < w.nt ? 1 : -1;
            if (slot == 1) {
                starts = make_int4((int)(((from + w.nt) * ctas - 1) / total), rb * NV, r.T * a.G, r.row0);
                starts_block = hblock;
            }
            if (!a.tree) {  // tiles past the block's last row's position
                const int t_last = (min((rb + 1) * NV, r.T * a.G) - 1) / a.G;
                u1 = min(u1, q8_seen_tiles(r, w, t_last, kt));
            }
            len = r.len;
            lo_tile = w.lo_tile;
            n_sink = w.n_sink;
            first = true;
            if (u >= u1) empty(slot);
        }
        t.b = b;
        t.rb = rb;
        t.key = (u < n_sink ? u : lo_tile + u - n_sink) * kt;
        t.flags = (first ? kFirst : 0) | (u + 1 == u1 ? kLast : 0) | (slot + 1) << kSlotShift | hblock << kBlockShift;
        first = false;
        ++u;
        return true;
    }
};

// Chunk c (16 bytes) of a row of hb D bytes in shared memory.  A K fragment's load takes 64
// bytes of each of two neighbouring rows, a V fragment's 32 (16 at headDim 64) of every other
// row; in this order they meet no bank twice (V at headDim 64: twice).
template <int D>
__device__ __forceinline__ int k_chunk(int row, int c, int hb) {
    return D == 128 || (hb & 1) == 0 ? c ^ ((row & 1) << 2) : c;
}
template <int D>
__device__ __forceinline__ int v_chunk(int row, int c) {
    return c ^ (D == 128 ? ((row >> 1) & 3) << 1 : (row >> 1) & 3);
}

// GROUPS: more than one key group (fewer than five KV heads).  Without their join in it the kernel
// takes 80.8 us instead of 83.3 for 32 requests of 517 to 8111 rows over 8 heads, 193 instead of 196
// for 24 of 8192 to 32704 (replayed graphs, caches flushed).
template <int D, int NT, int FORM, bool GROUPS>
__global__ void __launch_bounds__(kThreads, 1) q8_mma_kernel(const __grid_constant__ MmaArgs g) {
    constexpr int NV = 8 * NT, S = kStages, KC = D / 64, MT = D / 16;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ long long scan_s[kConsumers + kProducers];
    __shared__ __align__(8) uint64_t known[S], full[S], freed[S], x_put, x_got;
    __shared__ __align__(16) Tile tile_s[S];
    const PagedDesc& a = g.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, t4 = lane & 3;
    constexpr int warps = kConsumers + kProducers;
    const int consumers = g.hb * g.kg;  // that work
    long long* prefix = reinterpret_cast<long long*>(smem + (size_t)S * g.stage);

    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&known[i], 1);                // what the tile is
            mbar_init(&full[i], 32 * kProducers);  // every producer lane's copies
            mbar_init(&freed[i], consumers);
        }
        mbar_init(&x_put, consumers - g.hb > 0 ? consumers - g.hb : 1);
        mbar_init(&x_got, g.hb);
        fence_barrier_init();
    }
    // The requests' tiles and their running sum.
    long long carry = 0;
    for (int b0 = 0; b0 < a.B; b0 += blockDim.x) {
        const int b = b0 + threadIdx.x;
        long long v = 0;
        if (b < a.B) {
            const Q8Req r = q8_load_req(a, b);
            v = ((long long)r.T * a.G + NV - 1) / NV * g.blocks * q8_units(a, r, 32 * g.kg).nt;
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
        for (int w = 0; w < warps; ++w) {
            if (w < warp) before += scan_s[w];
            all += scan_s[w];
        }
        if (b < a.B) prefix[b] = before + s - v;
        carry = all;
        __syncthreads();
    }
    if (threadIdx.x == 0) prefix[a.B] = carry;
    __syncthreads();

    const int rows_stage = 32 * g.kg;
    const int width = g.hb * D;  // of a row
    const int scales_k = 2 * rows_stage * width, scales_v = scales_k + rows_stage * g.hb * 4;
    auto part_row = [&](int slot, int w, int i) -> int64_t { return ((int64_t)(3 * blockIdx.x + slot) * kConsumers + w) * NV + i; };

    if (warp >= kConsumers) {
        // ---- producers: each a quarter of a tile's rows, 8 of every 32 ----------------------
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        const int pw = warp - kConsumers;
        Walk<NV> walk;
        walk.start(g, prefix);
        auto empty = [&](int slot) {
            if (slot < 0 || pw > 0) return;
            for (int i = lane; i < g.hb * NV; i += 32) {  // key group 0's warps have the piece's partials
                g.part_m[part_row(slot, 0, i)] = -INFINITY;
                g.part_l[part_row(slot, 0, i)] = 0.f;
            }
        };
        // Lane i looks up row i of this warp's 8 kg of a tile: row 32 (i / 8) + 8 pw + i % 8 (kg of
        // more than 4: lane i row i + 32 too).  A tile ahead of its copies.
        Tile t, ahead;
        int len = 0, len_ahead = 0, h0 = 0, h0_ahead = 0, page[2], page_ahead[2];
        bool more = true;
        auto place = [&](int i) { return 32 * (i >> 3) + 8 * pw + (i & 7); };
        auto look = [&]() {
            more = walk.next(g, prefix, ahead, empty);
            if (!more) ahead.flags = kStop, ahead.key = -1;
            len_ahead = walk.len;
            h0_ahead = walk.hblock * g.hb;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                page_ahead[j] = -1;
                const int i = lane + 32 * j, key = ahead.key + place(i);
                if (ahead.key >= 0 && i < 8 * g.kg && key < len_ahead)
                    page_ahead[j] = __ldg(a.block_table + (int64_t)ahead.b * a.max_pages +
                                          (g.page_shift >= 0 ? key >> g.page_shift : key / a.page_size));
            }
        };
        look();
        int n = 0;
        for (;; ++n) {
            t = ahead;
            len = len_ahead;
            h0 = h0_ahead;
            page[0] = page_ahead[0];
            page[1] = page_ahead[1];
            if (more) look();
            const int st = n % S;
            if (n >= S && !__all_sync(FULL, mbar_wait(&freed[st], (uint32_t)((n / S - 1) & 1)))) {
                raise_device_error(&g_q8_device_error, kErrQ8Free);
                break;
            }
            unsigned char* to = smem + (size_t)st * g.stage;
            if (pw == 0 && lane == 0) {
                tile_s[st] = t;
                mbar_arrive(&known[st]);
            }
            if (t.key >= 0) {
                const int hb = min(g.hb, a.Hk - h0), chunks = hb * (D / 16);  // of a row
                int row[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int key = t.key + place(lane + 32 * j);
                    row[j] = (unsigned)page[j] < (unsigned)a.pages
                                 ? page[j] * a.page_size + (g.page_shift >= 0 ? key & (a.page_size - 1) : key % a.page_size)
                                 : -1;
                }
                const uint8_t* ks = g.p.k + (int64_t)h0 * D;
                const uint8_t* vs = g.p.v + (int64_t)h0 * D;
                const int64_t pitch = (int64_t)a.Hk * D;
                // 8 kg rows of `chunks` chunks each.
                // Rows of 1024 bytes (8 heads of 128) have a loop without divisions.  32 requests of 517 to 8112 rows:
                // 292 MB of such rows 76 us; by the other loop 146 MB of 4 heads of 128 66, 150 MB of 8 of 64 72, 182 MB of
                // 5 of 128 86.
                if (chunks == 64) {  // two accesses a row
#pragma unroll 8
                    for (int i = 0; i < 8; ++i) {
                        const int from = __shfl_sync(FULL, row[0], i), r = 8 * pw + i, bytes = from >= 0 ? 16 : 0;
                        const int64_t at = max(from, 0) * pitch + 16 * lane;
                        unsigned char* tk = to + r * 1024 + 16 * k_chunk<D>(r, lane, 8);
                        unsigned char* tv = to + 32768 + r * 1024 + 16 * v_chunk<D>(r, lane);
                        cp_async16(tk, ks + at, bytes);
                        cp_async16(tk + 512, ks + at + 512, bytes);
                        cp_async16(tv, vs + at, bytes);
                        cp_async16(tv + 512, vs + at + 512, bytes);
                    }
                } else {
                    for (int e = lane; e < 8 * g.kg * chunks; e += 32) {  // a multiple of 32
                        const int i = e / chunks, c = e - i * chunks, r = place(i);
                        const int from0 = __shfl_sync(FULL, row[0], i & 31), from1 = __shfl_sync(FULL, row[1], i & 31);
                        const int from = i < 32 ? from0 : from1, bytes = from >= 0 ? 16 : 0;
                        const int64_t at = max(from, 0) * pitch + 16 * c;
                        cp_async16(to + r * width + 16 * k_chunk<D>(r, c, g.hb), ks + at, bytes);
                        cp_async16(to + rows_stage * width + r * width + 16 * v_chunk<D>(r, c), vs + at, bytes);
                    }
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int i = lane + 32 * j;
                    if (i >= 8 * g.kg) break;
                    const int r = place(i);
                    const int64_t at = (int64_t)max(row[j], 0) * a.Hk + h0;
                    float* sk = reinterpret_cast<float*>(to + scales_k) + r * g.hb;
                    float* sv = reinterpret_cast<float*>(to + scales_v) + r * g.hb;
                    if (g.wide && (hb & 3) == 0) {
                        for (int h = 0; h < hb; h += 4) {
                            cp_async16(sk + h, g.p.k_scale + at + h, row[j] >= 0 ? 16 : 0);
                            cp_async16(sv + h, g.p.v_scale + at + h, row[j] >= 0 ? 16 : 0);
                        }
                    } else {
                        for (int h = 0; h < hb; ++h) {
                            cp_async4(sk + h, g.p.k_scale + at + h, row[j] >= 0 ? 4 : 0);
                            cp_async4(sv + h, g.p.v_scale + at + h, row[j] >= 0 ? 4 : 0);
                        }
                    }
                }
            }
            __syncwarp();
            cp_async_arrive(&full[st]);
            if (t.flags & kStop) break;
        }
        if (pw == 0 && lane == 0) {
            g.head[2 * blockIdx.x] = walk.starts;
            g.head[2 * blockIdx.x + 1] = make_int4(walk.starts_block * g.hb, 0, 0, 0);
        }
        cp_async_wait_all();  // no copy may be in flight when the CTA exits
        pdl_wait();           // nor this grid be done before the one that it overlaps
        return;
    }

    // ---- consumers: head `hi_warp` of the block, key group `group`; this lane's virtual rows are 2 t4,
    // 2 t4 + 1 of each eight ----
    // Shares of the launch's registers: 8 x 224 + 4 x 56 = 12 x 168 a lane.
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    if (warp >= consumers) return;
    const int group = GROUPS ? warp / g.hb : 0, head_w = warp - group * g.hb;
    uint32_t qf[KC][4][NT][4];  // hi and lo, two registers each, of k-step s of chunk c
    // What the queries' power of two takes back, as a factor of at most 1 for the keys' scales and one of at
    // least 1 for the scores: neither a scale's product nor a score then leaves f32 where x2 does
    // not, and a score of 0 stays 0.
    float rf[NT][2], up[NT][2];
    float o[MT][NT][4], m[NT][2], l[NT][2], r[NT][2], unit[NT][2];
    int hi[NT][2], lo[NT][2];
    float limit = -1.f;  // a tile whose scales are at most this takes the fast way
    Q8Req rq{};
    int sinks = 0, pieces = 0;
    for (int n = 0;; ++n) {
        const int st = n % S;
        auto wait = [&](uint64_t* bar) -> bool {
            if (__all_sync(FULL, mbar_wait(bar, (uint32_t)((n / S) & 1)))) return true;
            raise_device_error(&g_q8_device_error, kErrQ8Load);
            return false;
        };
        if (!wait(&known[st])) break;
        Tile tile = tile_s[st];
        if (tile.flags & kStop) break;
        const int hk = (tile.flags >> kBlockShift) * g.hb + head_w;
        const unsigned char* from = smem + (size_t)st * g.stage;
        const unsigned char* kt = from + group * 32 * width;
        const unsigned char* vt = from + (rows_stage + group * 32) * width;
        const float* sks = reinterpret_cast<const float*>(from + scales_k) + group * 32 * g.hb + head_w;
        const float* svs = reinterpret_cast<const float*>(from + scales_v) + group * 32 * g.hb + head_w;
        auto give_back = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(&freed[st]);
        };
        if (hk >= a.Hk) {  // the last block's missing heads
            give_back();
            continue;
        }
        tile.key += 32 * group;  // this warp's keys

        if (tile.flags & kFirst) {
            rq = q8_load_req(a, tile.b);
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
                    up[nt][e] = fmaxf(rf[nt][e], 1.f);
                    rf[nt][e] = fminf(rf[nt][e], 1.f);
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

        if (!wait(&full[st])) break;  // a piece's queries are asked for beside its first keys
        // ---- scores: x[block of 16 keys][nt]: keys gr (0, 1) and gr + 8 (2, 3), rows 2 t4 and + 1 ----
        float x[2][NT][4];
        float vs[2][2];  // value scales of keys gr, gr + 8
        {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[b][nt][e] = 0.f;
                const int r0 = 16 * b + gr, r1 = r0 + 8;
#pragma unroll
                for (int c = 0; c < KC; ++c) {
                    const uint4 w0 = *reinterpret_cast<const uint4*>(kt + r0 * width + 16 * k_chunk<D>(gr, head_w * (D / 16) + 4 * c + t4, g.hb));
                    const uint4 w1 = *reinterpret_cast<const uint4*>(kt + r1 * width + 16 * k_chunk<D>(gr, head_w * (D / 16) + 4 * c + t4, g.hb));
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
                const float ks[2] = {sks[r0 * g.hb], sks[r1 * g.hb]};
                vs[b][0] = svs[r0 * g.hb];
                vs[b][1] = svs[r1 * g.hb];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[b][nt][e] *= ks[e >> 1] * rf[nt][e & 1];
            }
        }
        if (a.softcap_on) {
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float f = up[nt][e & 1];
                        x[b][nt][e] = a.cap_log2 * softcap_tanh(x[b][nt][e] * f) * (1.f / f);
                    }
        }
        // ---- mask: bit (b, nt, e) of `see` ----
        uint32_t see = FULL;
        bool whole = true;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) whole = whole && hi[nt][e] - tile.key >= kKT - 1 && lo[nt][e] <= tile.key;
        whole = __all_sync(FULL, whole);
        if (!whole) {
            see = 0;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int key = tile.key + 16 * b + gr + 8 * h;
                            const bool on = key <= hi[nt][e] && (key >= lo[nt][e] || key < sinks);
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
                mt[nt][e] = fmaxf(fmaxf(x[0][nt][e], x[0][nt][2 + e]), fmaxf(x[1][nt][e], x[1][nt][2 + e])) * up[nt][e];
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
        // The largest scale, as bits, so that a NaN is the largest.
        const float tile_top = __uint_as_float(__reduce_max_sync(FULL, __float_as_uint(svs[lane * g.hb]) & 0x7fffffffu));
        uint32_t ph[2][NT][2], pl[2][NT][2];  // hi, lo
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
                        const float p = fast_exp2(fmaf(x[b][nt][e], up[nt][e & 1], -mu));
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
                        for (int h = 0; h < 2; ++h) top = fmaxf(top, fmaf(x[b][nt][2 * h + e], up[nt][e], -mu) + power(b, h));
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
                            const float y = fmaf(x[b][nt][2 * h + e], up[nt][e], -mu), ex = power(b, h);
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
        if (!whole) {  // the scale of a key that is not seen may be anything
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (!((see >> ((b * NT + nt) * 4 + e)) & 1)) w[b][nt][e] = 0.f;
        }
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    mma_split(w[b][nt][2 * h], w[b][nt][2 * h + 1], ph[b][nt][h], pl[b][nt][h]);
                    ph[b][nt][h] = mma_transpose(ph[b][nt][h]);
                    pl[b][nt][h] = mma_transpose(pl[b][nt][h]);
                }
        // ---- O^T += V^T P^T: row gr of product i is channel (D / 8) gr + 2 i, row gr + 8 the next ----
        {
            constexpr int W = D / 32;  // words of a lane's channels of one key
            uint32_t vw[2][4][W];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int row = 16 * b + 2 * t4 + (j & 1) + 8 * (j >> 1);
                    if constexpr (D == 128) {
                        const uint4 y = *reinterpret_cast<const uint4*>(vt + row * width + 16 * v_chunk<D>(2 * t4, head_w * (D / 16) + gr));
                        vw[b][j][0] = y.x; vw[b][j][1] = y.y; vw[b][j][2] = y.z; vw[b][j][3] = y.w;
                    } else {
                        const uint2 y = *reinterpret_cast<const uint2*>(vt + row * width + 16 * v_chunk<D>(2 * t4, head_w * (D / 16) + (gr >> 1)) + 8 * (gr & 1));
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
                        for (int e = 0; e < 4; e += 2)
                            f2_unpack(f2_add(f2_pack(o[2 * k + i][nt][e], o[2 * k + i][nt][e + 1]), f2_pack(acc[e], acc[e + 1])),
                                      o[2 * k + i][nt][e], o[2 * k + i][nt][e + 1]);
                    }
            }
        }
        give_back();
        // ---- the end of a piece ----
        if (tile.flags & kLast) {
            if (a.tree) pdl_wait();  // the drafted rows' part
            const int slot = ((tile.flags >> kSlotShift) & 3) - 1;
            // Key groups: the others leave theirs as partials in slot 2, group 0 takes them in.
            const uint32_t turn = (uint32_t)(pieces++ & 1);
            if (GROUPS) {
                uint64_t* bar = group ? &x_got : &x_put;
                if ((group == 0 || pieces > 1) && !__all_sync(FULL, mbar_wait(bar, group ? turn ^ 1 : turn))) {
                    raise_device_error(&g_q8_device_error, kErrQ8Load);
                    break;
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float sum = l[nt][e], top = m[nt][e];
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(FULL, sum, off);
                    const int i = 8 * nt + 2 * t4 + e, v = tile.rb * NV + i, t = v / a.G;
                    float y[D / 8];
                    {
                        const float inv = sum != 0.f ? 1.f / sum : 0.f, back = exp2f(r[nt][e] - kShift);
#pragma unroll
                        for (int k = 0; k < MT; ++k) {
                            y[2 * k] = o[k][nt][e] * inv * back;
                            y[2 * k + 1] = o[k][nt][2 + e] * inv * back;
                        }
                    }
                    if (GROUPS && group == 0) {  // by the log-sum-exp rule: the row's lane gr has group gr's part
                        float all = top, share = sum;
                        if (gr > 0) {
                            const int64_t at = part_row(2, gr * g.hb + head_w, i);
                            all = gr < g.kg ? __ldcg(g.part_m + at) : -INFINITY;
                            share = gr < g.kg ? __ldcg(g.part_l + at) : 0.f;
                        }
                        const float mine = all;
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1) all = fmaxf(all, __shfl_xor_sync(FULL, all, off));
                        // A part that saw nothing has no weight (-0); one that comes to 0 counts (0 x inf is NaN).
                        share = share != 0.f ? fast_exp2(mine - all) * share : -0.f;
                        float den = share;
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1) den += __shfl_xor_sync(FULL, den, off);
                        // Shares of the whole sum, so that what is added up stays below the largest value.
                        share *= den != 0.f ? 1.f / den : 0.f;
                        const float own = __shfl_sync(FULL, share, t4);
#pragma unroll
                        for (int k = 0; k < D / 8; ++k) y[k] = q8_nothing(own) ? 0.f : y[k] * own;
                        for (int k = 1; k < g.kg; ++k) {
                            const float w = __shfl_sync(FULL, share, 4 * k + t4);
                            if (q8_nothing(w)) continue;
                            const int64_t at = part_row(2, k * g.hb + head_w, i);
#pragma unroll
                            for (int d = 0; d < D / 8; d += 4) {
                                const float4 z = __ldcg(reinterpret_cast<const float4*>(g.part_o + at * D + (D / 8) * gr + d));
                                y[d] = fmaf(w, z.x, y[d]);
                                y[d + 1] = fmaf(w, z.y, y[d + 1]);
                                y[d + 2] = fmaf(w, z.z, y[d + 2]);
                                y[d + 3] = fmaf(w, z.w, y[d + 3]);
                            }
                        }
                        sum = den;
                        top = all;
                    }
                    float* to = nullptr;
                    const int where = GROUPS && group ? 2 : slot;
                    if (where < 0) {
                        if (v < rq.T * a.G) {
                            const int64_t row = ((int64_t)rq.row0 + t) * a.H + (int64_t)hk * a.G + (v - t * a.G);
                            to = a.out + row * D;
                            if (a.tree) {
                                const Q8Share w = q8_share(top, sum, __ldcg(g.draft + row));
#pragma unroll
                                for (int d = 0; d < D / 8; d += 4) {
                                    float4 z = __ldcg(reinterpret_cast<const float4*>(to + (D / 8) * gr + d));
                                    if (q8_nothing(w.draft)) z = make_float4(0.f, 0.f, 0.f, 0.f);
                                    y[d] = fmaf(w.own, y[d], w.draft * z.x);
                                    y[d + 1] = fmaf(w.own, y[d + 1], w.draft * z.y);
                                    y[d + 2] = fmaf(w.own, y[d + 2], w.draft * z.z);
                                    y[d + 3] = fmaf(w.own, y[d + 3], w.draft * z.w);
                                }
                            }
                        }
                    } else {
                        const int64_t at = part_row(where, warp, i);
                        to = g.part_o + at * D;
                        if (gr == 0) {
                            g.part_m[at] = top;
                            g.part_l[at] = sum;
                        }
                    }
                    if (to) {
                        to += (D / 8) * gr;
#pragma unroll
                        for (int d = 0; d < D / 8; d += 4)
                            *reinterpret_cast<float4*>(to + d) = make_float4(y[d], y[d + 1], y[d + 2], y[d + 3]);
                    }
                }
            if (GROUPS) {
                __syncwarp();
                if (lane == 0) mbar_arrive(group ? &x_put : &x_got);
            }
        }
    }
}

// Joins the partials of the unit that CTA blockIdx.x starts by the log-sum-exp rule, always in
// the same order: a warp per (head, virtual row).
template <int D, int NT>
__global__ void __launch_bounds__(256) q8_merge_kernel(const __grid_constant__ MmaArgs g, int rows) {
    constexpr int NV = 8 * NT, kPer = D / 32;
    pdl_wait();
    const PagedDesc& a = g.a;
    const int4 h = __ldcg(&g.head[2 * blockIdx.x]);
    const int h0 = __ldcg(&g.head[2 * blockIdx.x + 1].x);
    const int lane = threadIdx.x & 31, job = blockIdx.y * 8 + (threadIdx.x >> 5), head = job / rows, i = job - head * rows;
    const int v = h.y + i, hk = h0 + head;
    if (h.x < 0 || head >= g.hb || hk >= a.Hk || v >= h.z) return;
    const int count = h.x - blockIdx.x + 1;
    auto row = [&](int k) -> int64_t {
        return ((int64_t)(3 * (blockIdx.x + k) + (k == 0 ? 1 : 0)) * kConsumers + head) * NV + i;
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
#pragma unroll 4
        for (int k = 0; k < here; ++k) {
            const float f = __shfl_sync(FULL, wgt, k);
            if (__float_as_uint(f) == 0x80000000u) continue;
            const float* src = g.part_o + row(k0 + k) * D;
#pragma unroll
            for (int c = 0; c < kPer; ++c) acc[c] = fmaf(f, __ldcg(src + lane + 32 * c), acc[c]);
        }
    }
    const int t = v / a.G;
    const int64_t at = ((int64_t)h.w + t) * a.H + (int64_t)hk * a.G + (v - t * a.G);
    float* out = a.out + at * D;
    if (a.tree) {
        const Q8Share w = q8_share(m, den, __ldcg(g.draft + at));
#pragma unroll
        for (int c = 0; c < kPer; ++c) {
            const float z = q8_nothing(w.draft) ? 0.f : __ldcg(out + lane + 32 * c);
            acc[c] = fmaf(w.own, acc[c], w.draft * z);
        }
    }
#pragma unroll
    for (int c = 0; c < kPer; ++c) out[lane + 32 * c] = acc[c];
}

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

// Row blocks of 8 virtual rows where they hold a request's, else 16.
int blocks_of(const PagedDesc& a) { return (int64_t)a.max_rows * a.G <= 8 ? 1 : 2; }

struct Scratch {
    size_t m, l, o, head, draft, total;
};
Scratch scratch_of(int NV, int D, int64_t draft_rows) {
    const size_t rows = (size_t)3 * kPagedMaxCtas * kConsumers * NV;
    Scratch s;
    s.m = kWorkspaceHeader;
    s.l = s.m + up256(rows * 4);
    s.o = s.l + up256(rows * 4);
    s.head = s.o + up256(rows * D * 4);
    s.draft = s.head + up256((size_t)2 * kPagedMaxCtas * sizeof(int4));
    s.total = s.draft + up256((size_t)draft_rows * sizeof(float2));
    return s;
}

template <int D, int NT, int FORM>
cudaError_t launch_form(MmaArgs& g, int num_sms, void* workspace, cudaStream_t stream) {
    const PagedDesc& a = g.a;
    g.blocks = (a.Hk + kConsumers - 1) / kConsumers;
    g.hb = (a.Hk + g.blocks - 1) / g.blocks;
    g.kg = kConsumers / g.hb;
    if (g.kg == 3) g.kg = 2;  // tiles of a power of two
    g.wide = (a.Hk | g.hb) % 4 == 0 &&
             ((reinterpret_cast<uintptr_t>(g.p.k_scale) | reinterpret_cast<uintptr_t>(g.p.v_scale)) & 15u) == 0;
    g.stage = 32 * g.kg * g.hb * (2 * D + 8);
    const int ctas = num_sms < kPagedMaxCtas ? num_sms : kPagedMaxCtas;
    const Scratch s = scratch_of(8 * NT, D, 0);
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    g.part_m = reinterpret_cast<float*>(ws + s.m);
    g.part_l = reinterpret_cast<float*>(ws + s.l);
    g.part_o = reinterpret_cast<float*>(ws + s.o);
    g.head = reinterpret_cast<int4*>(ws + s.head);
    float2* draft = reinterpret_cast<float2*>(ws + s.draft);
    g.draft = draft;
    auto kern = g.kg > 1 ? q8_mma_kernel<D, NT, FORM, true> : q8_mma_kernel<D, NT, FORM, false>;
    cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kern), (int)kSmemMost);
    if (e != cudaSuccess) return e;
    const size_t smem = (size_t)kStages * g.stage + (size_t)(a.B + 1) * 8;
    if (smem > kSmemMost) return cudaErrorInvalidConfiguration;
    if (a.tree) {  // the cached part runs beside the drafted one and waits for it at the end
        e = launch_paged_q8_draft(a, draft, stream);
        if (e == cudaSuccess) e = launch_pdl(kern, dim3(ctas), dim3(kThreads), smem, stream, g);
    } else {
        kern<<<ctas, kThreads, smem, stream>>>(g);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) return e;
    const int64_t most = (int64_t)a.max_rows * a.G;
    const int live = most < 8 * NT ? (int)most : 8 * NT;
    return launch_pdl(q8_merge_kernel<D, NT>, dim3((unsigned)ctas, (unsigned)(g.hb * live + 7) / 8), dim3(256), 0, stream, g,
                      live);
}
template <int D, int NT>
cudaError_t launch_nt(MmaArgs& g, int num_sms, void* ws, cudaStream_t stream) {
    return g.p.form == kFormInt8 ? launch_form<D, NT, kFormInt8>(g, num_sms, ws, stream)
                                 : launch_form<D, NT, kFormE4m3>(g, num_sms, ws, stream);
}

}  // namespace

bool paged_q8_mma_supported(const PagedDesc& a) {
    return (a.D == 64 || a.D == 128) && a.pages > 0 && (int64_t)a.max_rows * a.G < ((int64_t)1 << 30);
}

size_t paged_q8_mma_workspace(const PagedDesc& a) {
    return scratch_of(8 * blocks_of(a), a.D, a.tree ? a.rows * a.H : 0).total;
}

cudaError_t launch_paged_q8_mma(const PagedDesc& a, const Q8Pools& p, int num_sms, void* workspace, cudaStream_t stream) {
    MmaArgs g;
    std::memset(&g, 0, sizeof(g));
    g.a = a;
    g.p = p;
    g.page_shift = -1;
    for (int i = 0; i < 31; ++i)
        if (a.page_size == 1 << i) g.page_shift = i;
    const int nt = blocks_of(a);
    if (a.D == 128)
        return nt == 1 ? launch_nt<128, 1>(g, num_sms, workspace, stream) : launch_nt<128, 2>(g, num_sms, workspace, stream);
    return nt == 1 ? launch_nt<64, 1>(g, num_sms, workspace, stream) : launch_nt<64, 2>(g, num_sms, workspace, stream);
}

unsigned int paged_q8_take_device_error() {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_q8_device_error, sizeof(v)) != cudaSuccess) return 0;
    if (v) {
        const unsigned int zero = 0;
        cudaMemcpyToSymbol(g_q8_device_error, &zero, sizeof(zero));
    }
    return v;
}

}  // namespace vtmu
