// paged_tc.cu -- attention of a ragged batch over a paged cache on the tcgen05
// tensor cores, headDim 64 or 128: single tokens, short runs, prompt chunks
// and trees of drafted tokens through one kernel.
//
// Mathematics.  For request b and KV head hk the T rows x G heads of the group
// are virtual rows v = t G + g; up to 128 of them (a row block) meet the same
// keys:   x2[v, s] = log2 e * softcap(scale q_v.k_s),  m = running max,
//         p = 2^(x2 - m),  l = sum p,  o = sum p v_s,  out = o / l.
// Both products run on f16 operands that carry 22 bits of an f32: a row x of Q,
// K or V is brought to |x| < 2 by a power of two e_x of its own (exact), then
// x = hi + lo with hi, lo in f16, and x.y = hi.hi + hi.lo + lo.hi, each summed
// in f32.  What is dropped or rounded is at most 2^-22 of the row's largest
// element.  Three f16 products cost 1.5 passes of a tf32 one, so this is twice
// as fast as splitting into tf32 halves, at the same precision, and halves
// the bytes that the MMAs read from shared memory.  Key scales multiply the
// scores, value scales the probabilities: p'_s = p_s 2^(e_s - e_max + 14) with
// e_max over the keys that the row sees in the tile, so that p' fills f16's
// range, and the tile's output is multiplied by 2^(e_max - 14).
//
// Split of the work.  The lengths are on the device, so the launch is one
// persistent CTA per SM and the CTAs divide the 64-key tiles of all (request,
// KV head, row block) units evenly among themselves: CTA c takes tiles
// [total c / n, total (c + 1) / n) of their concatenation.  A unit inside one
// CTA is finished there; a unit cut by a boundary leaves partials (m, l, o) that
// paged_merge_kernel joins by the log-sum-exp rule, always in the same order.
// With more than 128 virtual rows per KV head, teams of R CTAs walk the same
// tiles for R row blocks at the same time, so the tiles come from HBM once.
//
// Tiles of 64 keys, M = 128 virtual rows (padded: a wave of MMAs takes less
// time than the tile's bytes take from HBM, so padding costs nothing).  Warps:
//   0       page ids (32 at a time, one per lane) and TMA loads of raw f32 K and
//           V tiles, one box per page; drafted rows come as one tile of their
//           own from k_new / v_new; rows of no page are read out of bounds, as
//           zeros;
//   1       lane 0 issues the MMAs: S(n) = Q.K^T, then O(n - 1) = P.V;
//   4 - 7   softmax, thread = virtual row: no exchange between threads; P goes
//           back to TMEM over S as the A operand of P.V;
//   8 - 15  split: raw f32 rows to hi and lo in the 128-byte swizzled layout
//           (K K-major, V MN-major: the same bytes), the unit's Q to TMEM, and
//           the fold o = o alpha + O of the tile before last, 64 columns a thread
//           (a fresh accumulator per tile: no sum runs long inside the pipe).
// TMEM: Q hi, lo (D columns), S / P two buffers (128), O two buffers (2 D).
// Every wait is bounded; a wait that gives up sets a bit of the device flag.
#include <cstring>
#include <mutex>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_fp16.h>

#include "attn_common.cuh"
#include "kernels.h"
#include "launch_cache.h"
#include "paged.cuh"
#include "pdl.cuh"
#include "tcgen05_ops.cuh"
#include "tma_sync.cuh"

namespace vtmu {

__device__ unsigned int g_paged_device_error;

namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int kKT = 64;        // keys per tile
constexpr int kM = 128;        // virtual rows per row block
constexpr int kThreads = 512;
constexpr int kSplitWarps = 8;
constexpr int kPShift = 14;    // probabilities are scaled to at most 2^14 in f16

enum : unsigned int {
    kErrPgLoad = 1u << 3,   // the splitters gave up on a loaded tile
    kErrPgFree = 1u << 4,   // the producer gave up on a free stage, or on its copies at the end
    kErrPgMma = 1u << 5,    // a wait around the MMAs gave up
};

struct PgArgs {
    PagedDesc a;
    int32_t team;        // CTAs that walk the same tiles for different row blocks
    int32_t sub;         // rows per TMA box: min(page_size, 64)
    float* part_m;       // [2 CTAs][128]
    float* part_l;
    float* part_o;       // [2 CTAs][128][D]
    int4* head;          // [CTAs]: the unit that a CTA starts and others go on with
};

template <int D>
struct Cfg {
    static constexpr int kStages = D == 128 ? 3 : 6;             // raw tiles in flight
    static constexpr uint32_t kRaw = kKT * D * 4;
    static constexpr uint32_t kHalf = kKT * D * 2;               // hi (or lo) of a tile
    static constexpr uint32_t kBlock = kKT * 128;                // [64 rows x 64 elements]
    static constexpr uint32_t kColQhi = 0, kColQlo = D / 2, kColS = D, kColO = D + 2 * kKT;
    static constexpr uint32_t kTmemCols = 512;
    static constexpr size_t kSmemTiles = (size_t)kStages * kRaw + 2 * kHalf + 4 * kHalf;
    static constexpr size_t kSmem = 1024 + kSmemTiles + (kPagedMaxRequests + 1) * 8;
    static_assert(kColO + 2 * D <= kTmemCols, "TMEM budget");
    static_assert(kSmem + 20 * 1024 <= 232448, "shared memory budget");
};

// ---- the list of tiles --------------------------------------------------------------
// One request: packed rows [row0, row0 + T) are computed, n of them exist (their
// last one is the last row of the cache without a tree), len rows are cached.
struct Req {
    int row0, T, len, n;
};
struct Tiles {
    int lo_tile;  // first tile of the window's range
    int n_sink;   // tiles of sinks before it
    int n_main;
    int nt;       // with the drafted rows' tile; at least 1 when there are rows
};

__device__ __forceinline__ Req load_req(const PagedDesc& a, int b) {
    const PackedRows pr = packed_rows(a.cu_rows, b, a.rows);
    Req r;
    r.row0 = (int)pr.row0;
    r.n = (int)pr.n;
    r.T = min(r.n, a.max_rows);
    r.len = (int)clamp64(__ldg(a.lens + b), 0, (int64_t)a.max_pages * a.page_size);
    return r;
}
__device__ __forceinline__ Tiles tiles_of(const PagedDesc& a, const Req& r) {
    Tiles t;
    int64_t lo = 0;
    if (a.window > 0) lo = clamp64((a.tree ? (int64_t)r.len : (int64_t)r.len - r.n) - a.window + 1, 0, r.len);
    t.lo_tile = (int)(lo / kKT);
    t.n_sink = (int)min((min(a.sinks, (int64_t)r.len) + kKT - 1) / kKT, (int64_t)t.lo_tile);
    t.n_main = lo < r.len ? (r.len + kKT - 1) / kKT - t.lo_tile : 0;
    t.nt = t.n_sink + t.n_main + a.tree;
    if (r.T == 0) t.nt = 0;
    else if (t.nt == 0) t.nt = 1;
    return t;
}

struct Seg {
    Req r;
    Tiles t;
    int b, hk, rb;
    int u0, u1;       // tiles of the unit, this CTA's
    int slot;         // partial slot: 0 continues a unit, 1 starts one; -1: the whole unit
    int last_team;    // slot 1: the team that ends the unit
};

struct Walk {
    const PagedDesc& a;
    const long long* prefix;
    long long pos, end, total;
    int b, team, member, teams;
    __device__ __forceinline__ Walk(const PgArgs& g, const long long* prefix_) : a(g.a), prefix(prefix_) {
        team = g.team;
        member = blockIdx.x % team;
        const int c = blockIdx.x / team;
        total = prefix[a.B];
        teams = (int)min((long long)(gridDim.x / team), total);
        if (teams < 1) teams = 1;
        pos = c < teams ? total * c / teams : 0;
        end = c < teams ? total * (c + 1) / teams : 0;
        b = 0;
        int hi = a.B;  // the request of tile pos: the last one with prefix <= pos
        while (hi - b > 1) {
            const int mid = (b + hi) >> 1;
            if (prefix[mid] <= pos) b = mid; else hi = mid;
        }
    }
    // The next piece of a unit that this CTA has rows of; false at the end.  A
    // piece may be empty (u1 <= u0) where causality leaves its tiles unseen.
    __device__ __forceinline__ bool next(Seg& s) {
        while (pos < end) {
            while (prefix[b + 1] <= pos) ++b;
            s.r = load_req(a, b);
            s.t = tiles_of(a, s.r);
            const int blocks = (s.r.T * a.G + kM - 1) / kM, groups = (blocks + team - 1) / team;
            const long long rel = pos - prefix[b];
            const long long unit = rel / s.t.nt;
            s.u0 = (int)(rel - unit * s.t.nt);
            s.u1 = (int)min((long long)s.t.nt, s.u0 + (end - pos));
            const long long first = pos - s.u0;
            pos += s.u1 - s.u0;
            s.b = b;
            s.hk = (int)(unit / groups);
            s.rb = (int)(unit % groups) * team + member;
            if (s.rb >= blocks) continue;
            s.slot = s.u0 > 0 ? 0 : s.u1 < s.t.nt ? 1 : -1;
            s.last_team = (int)(((first + s.t.nt) * teams - 1) / total);
            if (!a.tree) {  // tiles past the block's last row's position
                const int t_last = (min((s.rb + 1) * kM, s.r.T * a.G) - 1) / a.G;
                const int p_last = s.r.len - s.r.n + t_last;
                const int seen = p_last < 0 ? 0 : p_last / kKT + 1 - s.t.lo_tile;
                int cap = s.t.n_sink + max(seen, 0);
                if (cap < 1) cap = 1;  // a unit always has a first tile, so that its rows are written
                s.u1 = min(s.u1, cap);
            }
            return true;
        }
        return false;
    }
};

// First key of tile u, or -1 for the drafted rows' tile.
__device__ __forceinline__ int tile_key(const Tiles& t, int tree, int u) {
    if (u < t.n_sink) return u * kKT;
    if (u < t.n_sink + t.n_main) return (t.lo_tile + u - t.n_sink) * kKT;
    return tree ? -1 : 0;  // 0: a unit without keys
}
// Rows of the tile that hold keys.
__device__ __forceinline__ int tile_rows(const Req& r, int key) {
    return key < 0 ? min(r.T, kKT) : max(min(r.len - key, kKT), 0);
}

// ---- f16 operands ---------------------------------------------------------------------
// Descriptor of an f16 kind MMA: f32 accumulator, A K-major, B K-major or (mn) MN-major.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool mn) {
    return (1u << 4) | (mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// Shared-memory descriptor of MN-major blocks of 64 elements (128 bytes, the
// 128-byte swizzle): rows are K; 8-row atoms 1024 bytes apart, blocks of 64
// elements `block` bytes apart.
__device__ __forceinline__ uint64_t smem_desc_mn(const void* tile, uint32_t block) {
    const uint64_t addr = smem_u32(tile);
    uint64_t d = (addr >> 4) & 0x3FFFull;
    d |= (uint64_t)(block >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// The power of two of a row whose largest |element| has the bits `top`: its
// exponent, kept where both the scale and its inverse are normal and sums of
// scaled probabilities stay finite.
__device__ __forceinline__ uint32_t row_exponent(uint32_t top) {
    const uint32_t e = top >> 23;
    return e < 27u ? 27u : e > 253u ? 253u : e;
}
__device__ __forceinline__ float pow2_of(uint32_t biased) { return __uint_as_float(biased << 23); }

// x0, x1 as f16 hi and lo pairs.
__device__ __forceinline__ void split2(float x0, float x1, uint32_t& hi, uint32_t& lo) {
    const __half2 h = __floats2half2_rn(x0, x1);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(x0 - f.x, x1 - f.y);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = *reinterpret_cast<const uint32_t*>(&l);
}

__device__ __forceinline__ float finite_or_zero(float x) {
    return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u ? 0.f : x;
}

// One raw tile (rows of D floats) to hi and lo tiles by the eight split warps,
// eight rows each; the rows' inverse scales to `scale`.  Rows past `rows` are
// zeros.  In value tiles elements that are not finite become zeros here, and
// `bad` gets a bit for each row that had one (they are added in the fold, to
// the rows that see them only); in key tiles they make their own scores
// not finite, which the mask discards.
template <int D, bool VALUES>
__device__ __forceinline__ void split_tile(const unsigned char* raw, unsigned char* hi, unsigned char* lo,
                                           float* scale, uint8_t* bad, int rows, int w, int lane) {
    constexpr int kLanes = D / 4;        // lanes per row
    constexpr int kRows = 32 / kLanes;   // rows per step
    const int l = lane % kLanes, sub = lane / kLanes;
    uint32_t bad_bits = 0;
#pragma unroll
    for (int i0 = 0; i0 < 8; i0 += 4) {
        float4 x[4 / kRows];
#pragma unroll
        for (int i = 0; i < 4 / kRows; ++i)
            x[i] = *reinterpret_cast<const float4*>(raw + (size_t)(8 * w + i0 + i * kRows + sub) * D * 4 + l * 16);
#pragma unroll
        for (int i = 0; i < 4 / kRows; ++i) {
            const int r = 8 * w + i0 + i * kRows + sub;
            float4 v = x[i];
            if (r >= rows) v = make_float4(0.f, 0.f, 0.f, 0.f);
            auto top_of = [](const float4& y) {
                return max(max(__float_as_uint(y.x) & 0x7fffffffu, __float_as_uint(y.y) & 0x7fffffffu),
                           max(__float_as_uint(y.z) & 0x7fffffffu, __float_as_uint(y.w) & 0x7fffffffu));
            };
            auto row_max = [&](uint32_t t) {
                if constexpr (kLanes == 32) {
                    return __reduce_max_sync(FULL, t);
                } else {
#pragma unroll
                    for (int off = kLanes / 2; off > 0; off >>= 1) t = max(t, __shfl_xor_sync(FULL, t, off));
                    return t;
                }
            };
            uint32_t top = row_max(top_of(v));
            if (__any_sync(FULL, top >= 0x7f800000u)) {  // rare
                if (VALUES) {
                    const bool b = top >= 0x7f800000u;
                    v = make_float4(finite_or_zero(v.x), finite_or_zero(v.y), finite_or_zero(v.z), finite_or_zero(v.w));
                    top = row_max(top_of(v));
                    const unsigned votes = __ballot_sync(FULL, b);
#pragma unroll
                    for (int k = 0; k < kRows; ++k)
                        if ((votes >> (k * kLanes)) & 1u) bad_bits |= 1u << (i0 + i * kRows + k);
                } else if (top >= 0x7f800000u) {
                    top = 0x3f800000u;
                }
            }
            const uint32_t e = row_exponent(top);
            const float s = pow2_of(254u - e);
            uint32_t h0, h1, l0, l1;
            split2(v.x * s, v.y * s, h0, l0);
            split2(v.z * s, v.w * s, h1, l1);
            // Element 4 l of row r: block l / 16, 16-byte chunk (l % 16) / 2 of the
            // row's 128 bytes, swizzled by r % 8.
            const uint32_t off = (l >> 4) * (kKT * 128) + r * 128 + ((((l & 15) >> 1) ^ (r & 7)) << 4) + (l & 1) * 8;
            *reinterpret_cast<uint2*>(hi + off) = make_uint2(h0, h1);
            *reinterpret_cast<uint2*>(lo + off) = make_uint2(l0, l1);
            if (l == 0) scale[r] = pow2_of(e);
        }
    }
    if (VALUES && lane == 0) bad[w] = (uint8_t)bad_bits;
}

// ---- the kernel -------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ CUtensorMap tm_kn, const __grid_constant__ CUtensorMap tm_vn,
                    const PgArgs g) {
    using C = Cfg<D>;
    constexpr int ST = C::kStages;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                           ~uintptr_t(1023));
    unsigned char* raw = base;                                   // ST raw tiles
    unsigned char* kt = raw + (size_t)ST * C::kRaw;              // K hi, lo
    unsigned char* vt = kt + 2 * C::kHalf;                       // V hi, lo, two buffers
    long long* prefix = reinterpret_cast<long long*>(vt + 4 * C::kHalf);
    __shared__ __align__(8) uint64_t raw_full[ST], raw_empty[ST], k_ready, k_free, v_ready[2], s_full[2], p_full[2],
        o_full[2], o_free[2];
    __shared__ uint32_t tmem_base_s;
    __shared__ long long scan_s[kThreads / 32];
    // What tile n leaves for the roles that come later, at n % 4 (each is read
    // before the splitters can reach tile n + 4).
    __shared__ __align__(16) float k_scale[4][kKT], v_scale[4][kKT];
    __shared__ __align__(8) uint8_t v_bad[4][8];
    __shared__ float q_scale[4][kM];             // by piece % 4
    __shared__ float2 fold_f[4][kM];             // alpha, output scale
    __shared__ uint64_t row_bad[4][kM];          // values to add that are not finite
    __shared__ int4 tile_at[4];                  // last tile of its piece, request, first key, KV head
    __shared__ float* row_out[4][kM];            // last tile of a piece: where the row goes
    __shared__ float row_inv[4][kM];
    __shared__ __align__(16) float v_norm[4][kKT];  // per softmax warp: value scales of a tile all rows see

    const PagedDesc& a = g.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(&raw_full[i], 1);
            mbar_init(&raw_empty[i], kSplitWarps);
        }
        mbar_init(&k_ready, kSplitWarps);
        mbar_init(&k_free, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&v_ready[i], kSplitWarps);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&o_full[i], 1);
            mbar_init(&o_free[i], kSplitWarps);
        }
        fence_barrier_init();
    }
    if (warp == 1) tmem_alloc(&tmem_base_s, C::kTmemCols);
    if (threadIdx.x == 32) g.head[blockIdx.x] = make_int4(-1, 0, 0, 0);

    // The requests' tiles and their running sum.
    long long carry = 0;
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        long long v = 0;
        if (b < a.B) {
            const Req r = load_req(a, b);
            const long long blocks = ((long long)r.T * a.G + kM - 1) / kM;
            v = (blocks + g.team - 1) / g.team * a.Hk * tiles_of(a, r).nt;
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
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before += scan_s[w];
            all += scan_s[w];
        }
        if (b < a.B) prefix[b] = before + s - v;
        carry = all;
        __syncthreads();
    }
    if (threadIdx.x == 0) prefix[a.B] = carry;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_s;

    Walk walk(g, prefix);
    Seg s;

    if (warp == 0) {
        // ---- producer: raw K and V tiles --------------------------------------------
        if (lane == 0) {
            prefetch_tensormap(&tm_k);
            prefetch_tensormap(&tm_v);
        }
        const int nsub = kKT / g.sub;
        const int nowhere = (int)(a.pages * a.page_size);  // a row out of bounds: zeros
        int it = 0;
        bool ok = true;
        while (ok && walk.next(s)) {
            int batch = -1, y_cur = nowhere;
            const int subs = (s.r.len + g.sub - 1) / g.sub;
            for (int u = s.u0; ok && u < s.u1; ++u) {
                const int key = tile_key(s.t, a.tree, u);
                int y = nowhere;
                if (key >= 0) {
                    const int q0 = key / g.sub;
                    if ((q0 >> 5) != batch) {
                        batch = q0 >> 5;
                        const int q = (batch << 5) + lane;
                        y_cur = nowhere;
                        if (q < subs) {
                            const int row = q * g.sub;
                            const int page = __ldg(a.block_table + (int64_t)s.b * a.max_pages + row / a.page_size);
                            if (page >= 0 && page < a.pages) y_cur = page * a.page_size + row % a.page_size;
                        }
                    }
                    y = __shfl_sync(FULL, y_cur, (q0 & 31) + (lane < nsub ? lane : 0));
                }
#pragma unroll
                for (int kv = 0; kv < 2; ++kv, ++it) {
                    const int st = it % ST;
                    if (it >= ST && !__all_sync(FULL, mbar_wait(&raw_empty[st], (uint32_t)((it / ST - 1) & 1)))) {
                        raise_device_error(&g_paged_device_error, kErrPgFree);
                        ok = false;
                        break;
                    }
                    if (lane == 0) mbar_arrive_expect_tx(&raw_full[st], C::kRaw);
                    __syncwarp();
                    unsigned char* dst = raw + (size_t)st * C::kRaw;
                    if (key < 0) {
                        if (lane == 0) tma_load_2d(dst, kv ? &tm_vn : &tm_kn, s.hk * D, s.r.row0, &raw_full[st]);
                    } else if (lane < nsub) {
                        tma_load_2d(dst + (size_t)lane * g.sub * D * 4, kv ? &tm_v : &tm_k, s.hk * D, y, &raw_full[st]);
                    }
                }
            }
        }
        // No copy may be in flight when the CTA exits.
        for (int j = it < ST ? 0 : it - ST; j < it; ++j)
            if (!mbar_wait(&raw_full[j % ST], (uint32_t)((j / ST) & 1)))
                raise_device_error(&g_paged_device_error, kErrPgFree);
    } else if (warp == 1) {
        // ---- MMAs ------------------------------------------------------------------------
        if (lane == 0) {
            constexpr uint32_t id_s = idesc_f16(kM, kKT, false), id_o = idesc_f16(kM, D, true);
            int n = 0;
            bool ok = true;
            auto pv = [&](int j) -> bool {  // O(j) = P(j).V(j)
                const int bf = j & 1;
                const uint32_t ph = (uint32_t)((j >> 1) & 1);
                if (!mbar_wait(&p_full[bf], ph) || !mbar_wait(&v_ready[bf], ph) ||
                    (j >= 2 && !mbar_wait(&o_free[bf], ph ^ 1u))) {
                    raise_device_error(&g_paged_device_error, kErrPgMma);
                    return false;
                }
                tc_fence_after();
                const uint32_t d = tmem + C::kColO + bf * D;
                const uint32_t phi = tmem + C::kColS + bf * kKT, plo = phi + kKT / 2;
                const uint64_t vhi = smem_desc_mn(vt + bf * 2 * C::kHalf, C::kBlock);
                const uint64_t vlo = smem_desc_mn(vt + bf * 2 * C::kHalf + C::kHalf, C::kBlock);
#pragma unroll
                for (int k = 0; k < kKT / 16; ++k) {  // 16 keys: 8 columns of P, 16 rows (2048 bytes) of V
                    mma_f16_ts(d, phi + 8 * k, vhi + 128 * k, id_o, k > 0 ? 1u : 0u);
                    mma_f16_ts(d, plo + 8 * k, vhi + 128 * k, id_o, 1u);
                    mma_f16_ts(d, phi + 8 * k, vlo + 128 * k, id_o, 1u);
                }
                mma_commit(&o_full[bf]);
                return true;
            };
            while (ok && walk.next(s)) {
                for (int u = s.u0; ok && u < s.u1; ++u, ++n) {
                    if (!mbar_wait(&k_ready, (uint32_t)(n & 1))) {
                        raise_device_error(&g_paged_device_error, kErrPgMma);
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d = tmem + C::kColS + (n & 1) * kKT;
                    const uint64_t khi = smem_desc_sw128(kt), klo = smem_desc_sw128(kt + C::kHalf);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {  // 16 dims: 8 columns of Q, 32 bytes of a K row
                        const uint64_t off = (uint64_t)(k >> 2) * (C::kBlock >> 4) + 2 * (k & 3);
                        mma_f16_ts(d, tmem + C::kColQhi + 8 * k, khi + off, id_s, k > 0 ? 1u : 0u);
                        mma_f16_ts(d, tmem + C::kColQlo + 8 * k, khi + off, id_s, 1u);
                        mma_f16_ts(d, tmem + C::kColQhi + 8 * k, klo + off, id_s, 1u);
                    }
                    mma_commit(&k_free);
                    mma_commit(&s_full[n & 1]);
                    if (n > 0 && !pv(n - 1)) ok = false;
                }
            }
            if (ok && n > 0) pv(n - 1);
        }
    } else if (warp >= 4 && warp < 8) {
        // ---- softmax: thread = virtual row -------------------------------------------
        const int i = threadIdx.x - 128;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        int n = 0, piece = 0;
        bool ok = true;
        while (ok && walk.next(s)) {
            const int v = s.rb * kM + i, t = v / a.G;
            const bool alive = v < s.r.T * a.G;
            const int64_t row = (int64_t)s.r.row0 + (alive ? t : 0);
            const int64_t prow = (int64_t)(2 * blockIdx.x + (s.slot > 0 ? 1 : 0)) * kM + i;  // of the partials
            if (s.slot > 0 && i == 0)
                g.head[blockIdx.x] = make_int4(s.last_team, s.hk, s.rb, s.b);
            if (s.u1 <= s.u0) {  // nothing to see in this piece
                if (s.slot >= 0) {
                    g.part_m[prow] = -INFINITY;
                    g.part_l[prow] = 0.f;
                }
                continue;
            }
            // Keys of the cache that the row sees: [lo, hi], and those before `sinks`.
            int64_t p = a.tree ? (int64_t)s.r.len : (int64_t)s.r.len - s.r.n + t;
            if (a.tree && a.window > 0 && alive) p = __ldg(a.positions + row);
            const int64_t hi = a.tree ? s.r.len - 1 : min(p, (int64_t)s.r.len - 1);
            const int64_t lo = a.window > 0 ? max(p - a.window + 1, (int64_t)0) : 0;
            float m = -INFINITY, l = 0.f;
            const bool idle = !__any_sync(FULL, alive);  // a warp without rows only keeps step
            for (int u = s.u0; u < s.u1; ++u, ++n) {
                const int key = tile_key(s.t, a.tree, u), nb = n & 3, bf = n & 1;
                if (!__all_sync(FULL, mbar_wait(&s_full[bf], (uint32_t)((n >> 1) & 1)) &&
                                          mbar_wait(&v_ready[bf], (uint32_t)((n >> 1) & 1)))) {
                    raise_device_error(&g_paged_device_error, kErrPgMma);
                    ok = false;
                    break;
                }
                if (idle) {
                    row_out[nb][i] = nullptr;
                    row_bad[nb][i] = 0;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_full[bf]);
                    continue;
                }
                uint64_t see = ~0ull;  // rows of no request: anything
                if (alive) {
                    auto below = [](int64_t c) -> uint64_t { return c <= 0 ? 0ull : c >= 64 ? ~0ull : (1ull << c) - 1; };
                    if (key >= 0) {
                        see = below(hi - key + 1) & (~below(lo - key) | below(a.sinks - key));
                    } else {
                        see = __ldg(reinterpret_cast<const unsigned long long*>(a.masks) + row) & below(s.r.T);
                        if (a.window > 0)
                            for (int j = 0; j < s.r.T; ++j)
                                if (__ldg(a.positions + s.r.row0 + j) <= p - a.window) see &= ~(1ull << j);
                    }
                }
                tc_fence_after();
                float x[kKT];
                tmem_ld32(tmem + lanes + C::kColS + bf * kKT, x);
                tmem_ld32(tmem + lanes + C::kColS + bf * kKT + 32, x + 32);
                tmem_wait_ld();
                const float qs = q_scale[piece & 3][i];
                const bool whole = __all_sync(FULL, see == ~0ull);
#pragma unroll
                for (int k = 0; k < kKT; k += 4) {
                    const float4 ks = *reinterpret_cast<const float4*>(&k_scale[nb][k]);
                    x[k] *= ks.x;
                    x[k + 1] *= ks.y;
                    x[k + 2] *= ks.z;
                    x[k + 3] *= ks.w;
                }
                float mul = qs;  // x * mul is the score in base-2 units
                if (a.softcap_on) {
#pragma unroll
                    for (int k = 0; k < kKT; ++k) x[k] = softcap_tanh(x[k] * qs);
                    mul = a.cap_log2;
                }
                // The largest value scale among the keys seen.
                uint32_t vtop;
                if (whole) {
                    const float2 v2 = make_float2(v_scale[nb][lane], v_scale[nb][lane + 32]);
                    vtop = __reduce_max_sync(FULL, max(__float_as_uint(v2.x), __float_as_uint(v2.y)));
                } else {
                    float vm = pow2_of(27u);
#pragma unroll
                    for (int k = 0; k < kKT; ++k) {
                        const bool vis = (see >> k) & 1;
                        x[k] = vis ? x[k] : -INFINITY;
                        vm = fmaxf(vm, vis ? v_scale[nb][k] : 0.f);
                    }
                    vtop = __float_as_uint(vm);
                }
                const float c = pow2_of(254u + kPShift - (vtop >> 23));  // 2^kPShift / the largest scale
                if (whole) {
                    v_norm[warp & 3][lane] = v_scale[nb][lane] * c;
                    v_norm[warp & 3][lane + 32] = v_scale[nb][lane + 32] * c;
                    __syncwarp();
                }
                float mt = -INFINITY;
#pragma unroll
                for (int k = 0; k < kKT; ++k) mt = fmaxf(mt, x[k]);
                const float mn = fmaxf(m, mt * mul), mu = mn == -INFINITY ? 0.f : mn;
                const float alpha = fast_exp2(m - mu);
                m = mn;
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
                const float* vs = whole ? v_norm[warp & 3] : v_scale[nb];
                const float cc = whole ? 1.f : c;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float phi[16], plo[16];
#pragma unroll
                    for (int k = 0; k < 32; k += 4) {
                        const float4 w = *reinterpret_cast<const float4*>(&vs[32 * h + k]);
                        const float e0 = fast_exp2(fmaf(x[32 * h + k], mul, -mu)), e1 = fast_exp2(fmaf(x[32 * h + k + 1], mul, -mu)),
                                    e2 = fast_exp2(fmaf(x[32 * h + k + 2], mul, -mu)), e3 = fast_exp2(fmaf(x[32 * h + k + 3], mul, -mu));
                        sum[0] += e0;
                        sum[1] += e1;
                        sum[2] += e2;
                        sum[3] += e3;
                        uint32_t h0, l0, h1, l1;
                        split2(e0 * w.x * cc, e1 * w.y * cc, h0, l0);
                        split2(e2 * w.z * cc, e3 * w.w * cc, h1, l1);
                        phi[k / 2] = __uint_as_float(h0);
                        phi[k / 2 + 1] = __uint_as_float(h1);
                        plo[k / 2] = __uint_as_float(l0);
                        plo[k / 2 + 1] = __uint_as_float(l1);
                    }
                    tmem_st16(tmem + lanes + C::kColS + bf * kKT + 16 * h, phi);
                    tmem_st16(tmem + lanes + C::kColS + bf * kKT + kKT / 2 + 16 * h, plo);
                }
                l = fmaf(l, alpha, (sum[0] + sum[1]) + (sum[2] + sum[3]));
                fold_f[nb][i] = make_float2(alpha, pow2_of((vtop >> 23) - kPShift));
                const uint64_t bad = *reinterpret_cast<const uint64_t*>(v_bad[nb]);
                if (bad) row_bad[nb][i] = alive ? bad & see : 0ull;
                if (u == s.u1 - 1) {
                    float* to = nullptr;
                    float inv = 1.f;
                    if (s.slot < 0) {
                        if (alive) to = a.out + (row * a.H + (int64_t)s.hk * a.G + (v - t * a.G)) * D;
                        inv = l != 0.f ? 1.f / l : 0.f;
                    } else {
                        if (alive) to = g.part_o + prow * D;
                        g.part_m[prow] = m;
                        g.part_l[prow] = l;
                    }
                    row_out[nb][i] = to;
                    row_inv[nb][i] = inv;
                }
                if (i == 0) tile_at[nb] = make_int4(u == s.u1 - 1, s.b, key, s.hk);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[bf]);
            }
            ++piece;
        }
    } else if (warp >= 8) {
        // ---- split, queries and fold --------------------------------------------------
        const int w = warp - 8, quarter = warp & 3, side = w >> 2;  // columns side * D / 2 ..
        const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
        const int i = 32 * quarter + lane;
        float o[D / 2];
#pragma unroll
        for (int d = 0; d < D / 2; ++d) o[d] = 0.f;
        int n = 0, piece = 0, it = 0;
        bool ok = true;
        auto fold = [&](int j) -> bool {
            const int nb = j & 3, bf = j & 1;
            if (!__all_sync(FULL, mbar_wait(&o_full[bf], (uint32_t)((j >> 1) & 1)))) {
                raise_device_error(&g_paged_device_error, kErrPgMma);
                return false;
            }
            tc_fence_after();
            const float2 f = fold_f[nb][i];
            const uint32_t at = tmem + lanes + C::kColO + bf * D + side * (D / 2);
#pragma unroll
            for (int c0 = 0; c0 < D / 2; c0 += 16) {
                float acc[16];
                tmem_ld16(at + c0, acc);
                tmem_wait_ld();
#pragma unroll
                for (int d = 0; d < 16; ++d) o[c0 + d] = fmaf(acc[d], f.y, o[c0 + d] * f.x);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_free[bf]);
            const int4 ta = tile_at[nb];
            if (*reinterpret_cast<const uint64_t*>(v_bad[nb])) {
                // Values that are not finite, for the rows that see them.
                uint64_t rest = row_bad[nb][i];
                while (rest) {
                    const int k = __ffsll((long long)rest) - 1;
                    rest &= rest - 1;
                    const float* src = nullptr;
                    if (ta.z < 0) {
                        src = a.v_new + (packed_rows(a.cu_rows, ta.y, a.rows).row0 + k) * a.Hk * D;
                    } else {
                        const int key = ta.z + k;
                        const int64_t page = __ldg(a.block_table + (int64_t)ta.y * a.max_pages + key / a.page_size);
                        if (page >= 0 && page < a.pages)
                            src = a.v_pool + (page * a.page_size + key % a.page_size) * a.Hk * D;
                    }
                    if (!src) continue;
                    src += (int64_t)ta.w * D + side * (D / 2);
#pragma unroll
                    for (int d = 0; d < D / 2; ++d) {
                        const float x = __ldg(src + d);
                        if ((__float_as_uint(x) & 0x7f800000u) == 0x7f800000u) o[d] += x;
                    }
                }
            }
            if (ta.x) {
                float* to = row_out[nb][i];
                const float inv = row_inv[nb][i];
                if (to) {
                    to += side * (D / 2);
                    if (reinterpret_cast<uintptr_t>(to) & 15u) {
#pragma unroll
                        for (int d = 0; d < D / 2; ++d) to[d] = o[d] * inv;
                    } else {
#pragma unroll
                        for (int d = 0; d < D / 2; d += 4)
                            *reinterpret_cast<float4*>(to + d) =
                                make_float4(o[d] * inv, o[d + 1] * inv, o[d + 2] * inv, o[d + 3] * inv);
                    }
                }
#pragma unroll
                for (int d = 0; d < D / 2; ++d) o[d] = 0.f;
            }
            return true;
        };
        auto raw_tile = [&]() -> const unsigned char* {  // the next raw tile, once loaded
            const int st = it % ST;
            if (!__all_sync(FULL, mbar_wait(&raw_full[st], (uint32_t)((it / ST) & 1)))) {
                raise_device_error(&g_paged_device_error, kErrPgLoad);
                return nullptr;
            }
            return raw + (size_t)st * C::kRaw;
        };
        while (ok && walk.next(s)) {
            if (s.u1 <= s.u0) continue;
            for (int u = s.u0; u < s.u1; ++u, ++n) {
                const int key = tile_key(s.t, a.tree, u), nb = n & 3, bf = n & 1;
                const int rows = tile_rows(s.r, key);
                // K(n) once S(n - 1) is done; before the first one, the unit's queries.
                if (n > 0 && !__all_sync(FULL, mbar_wait(&k_free, (uint32_t)((n - 1) & 1)))) {
                    raise_device_error(&g_paged_device_error, kErrPgMma);
                    ok = false;
                    break;
                }
                if (u == s.u0) {
                    // Row i of the block: q scaled by qk_mul, then as any row; columns
                    // side * D / 4 .. + D / 4 of Q hi and Q lo (two elements each).
                    const int v = s.rb * kM + i, t = v / a.G;
                    const bool alive = v < s.r.T * a.G;
                    const float* q = a.q + (((int64_t)s.r.row0 + t) * a.H + (int64_t)s.hk * a.G + (v - t * a.G)) * D;
                    const bool vec = (reinterpret_cast<uintptr_t>(a.q) & 15u) == 0;
                    auto load4 = [&](int d) -> float4 {
                        if (!alive) return make_float4(0.f, 0.f, 0.f, 0.f);
                        float4 y = vec ? __ldg(reinterpret_cast<const float4*>(q + d))
                                       : make_float4(__ldg(q + d), __ldg(q + d + 1), __ldg(q + d + 2), __ldg(q + d + 3));
                        return make_float4(y.x * a.qk_mul, y.y * a.qk_mul, y.z * a.qk_mul, y.w * a.qk_mul);
                    };
                    float top = 0.f;
#pragma unroll 8
                    for (int d = 0; d < D; d += 4) {
                        const float4 y = load4(d);
                        top = fmaxf(top, fmaxf(fmaxf(fabsf(y.x), fabsf(y.y)), fmaxf(fabsf(y.z), fabsf(y.w))));
                    }
                    const uint32_t e = row_exponent(__float_as_uint(top));
                    const float sc = pow2_of(254u - e);
                    if (side == 0) q_scale[piece & 3][i] = pow2_of(e);
#pragma unroll 1
                    for (int c0 = 0; c0 < D / 4; c0 += 16) {
                        float qh[16], ql[16];
#pragma unroll
                        for (int c = 0; c < 16; c += 2) {
                            const float4 y = load4(side * (D / 2) + 2 * (c0 + c));
                            uint32_t h0, l0, h1, l1;
                            split2(y.x * sc, y.y * sc, h0, l0);
                            split2(y.z * sc, y.w * sc, h1, l1);
                            qh[c] = __uint_as_float(h0);
                            qh[c + 1] = __uint_as_float(h1);
                            ql[c] = __uint_as_float(l0);
                            ql[c + 1] = __uint_as_float(l1);
                        }
                        tmem_st16(tmem + lanes + C::kColQhi + side * (D / 4) + c0, qh);
                        tmem_st16(tmem + lanes + C::kColQlo + side * (D / 4) + c0, ql);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                }
                const unsigned char* rt = raw_tile();
                if (!rt) {
                    ok = false;
                    break;
                }
                split_tile<D, false>(rt, kt, kt + C::kHalf, k_scale[nb], nullptr, rows, w, lane);
                asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");  // generic writes -> MMA, TMA
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&k_ready);
                    mbar_arrive(&raw_empty[it % ST]);
                }
                ++it;
                // V(n) once O(n - 2) is done.
                if (n >= 2 && !__all_sync(FULL, mbar_wait(&o_full[bf], (uint32_t)(((n - 2) >> 1) & 1)))) {
                    raise_device_error(&g_paged_device_error, kErrPgMma);
                    ok = false;
                    break;
                }
                rt = raw_tile();
                if (!rt) {
                    ok = false;
                    break;
                }
                unsigned char* vb = vt + bf * 2 * C::kHalf;
                split_tile<D, true>(rt, vb, vb + C::kHalf, v_scale[nb], v_bad[nb], rows, w, lane);
                asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&v_ready[bf]);
                    mbar_arrive(&raw_empty[it % ST]);
                }
                ++it;
                if (n >= 2 && !fold(n - 2)) {
                    ok = false;
                    break;
                }
            }
            if (!ok) break;
            ++piece;
        }
        if (ok && n >= 2) ok = fold(n - 2);
        if (ok && n >= 1) fold(n - 1);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

// Joins the partials of the unit that CTA blockIdx.x started and its team's
// successors went on with: m* = max m_i, out = sum 2^(m_i - m*) o_i / sum 2^(m_i - m*) l_i.
// A warp per virtual row.
template <int D>
__global__ void __launch_bounds__(256) paged_merge_kernel(const PgArgs g) {
    pdl_wait();
    const PagedDesc& a = g.a;
    const int4 h = __ldcg(&g.head[blockIdx.x]);
    if (h.x < 0) return;
    const int hk = h.y, rb = h.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Req r = load_req(a, h.w);
    const int i = blockIdx.y * 8 + warp, v = rb * kM + i;
    if (v >= r.T * a.G) return;
    const int first = blockIdx.x, count = h.x - first / g.team + 1;
    auto slot_row = [&](int k) -> int64_t {  // piece k of the unit
        return (int64_t)(2 * (first + k * g.team) + (k == 0 ? 1 : 0)) * kM + i;
    };
    float m = -INFINITY;
    for (int k = lane; k < count; k += 32) m = fmaxf(m, __ldcg(g.part_m + slot_row(k)));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, off));
    constexpr int kPer = D / 32;
    float acc[kPer], den = 0.f;
#pragma unroll
    for (int c = 0; c < kPer; ++c) acc[c] = 0.f;
    for (int k0 = 0; k0 < count; k0 += 32) {
        float wgt = 0.f, ll = 0.f;
        if (k0 + lane < count) {
            const float mi = __ldcg(g.part_m + slot_row(k0 + lane));
            if (mi != -INFINITY) {  // a piece that saw nothing has no output to read
                wgt = fast_exp2(mi - m);
                ll = wgt * __ldcg(g.part_l + slot_row(k0 + lane));
            }
        }
        den += ll;
        const int here = min(count - k0, 32);
        for (int k = 0; k < here; ++k) {
            const float f = __shfl_sync(FULL, wgt, k);
            if (f == 0.f) continue;
            const float* src = g.part_o + slot_row(k0 + k) * D;
#pragma unroll
            for (int c = 0; c < kPer; ++c) acc[c] = fmaf(f, __ldcg(src + lane + 32 * c), acc[c]);
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) den += __shfl_xor_sync(FULL, den, off);
    const float inv = den != 0.f ? 1.f / den : 0.f;
    float* out = a.out + (((int64_t)r.row0 + v / a.G) * a.H + (int64_t)hk * a.G + v % a.G) * D;
#pragma unroll
    for (int c = 0; c < kPer; ++c) out[lane + 32 * c] = acc[c] * inv;
}

PFN_cuTensorMapEncodeTiled_v12000 pg_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    return fn;
}

// Row-major [rows, cols] f32, boxes of box_rows rows x D columns, no swizzle.
bool encode_rows(CUtensorMap* map, const float* p, int64_t rows, int64_t cols, int box_cols, int box_rows) {
    return cached_tensor_map(map, p, rows, cols, box_cols, box_rows, 0, [&](CUtensorMap* m) {
        auto fn = pg_encoder();
        if (!fn) return false;
        const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
        const cuuint64_t strides[1] = {(cuuint64_t)cols * sizeof(float)};
        const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
        const cuuint32_t estr[2] = {1, 1};
        return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<float*>(p), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    });
}

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

struct PgScratch {
    size_t m, l, o, head, total;
};
PgScratch scratch_of(int ctas, int D) {
    PgScratch s;
    const size_t rows = (size_t)2 * ctas * kM;
    s.m = kWorkspaceHeader;
    s.l = s.m + up256(rows * 4);
    s.o = s.l + up256(rows * 4);
    s.head = s.o + up256(rows * D * 4);
    s.total = s.head + up256((size_t)ctas * sizeof(int4));
    return s;
}

// CTAs per team: the row blocks of the largest request, at most eight.
int team_of(const PagedDesc& a) {
    const int64_t blocks = ((int64_t)a.max_rows * a.G + kM - 1) / kM;
    return blocks <= 1 ? 1 : blocks == 2 ? 2 : blocks <= 4 ? 4 : 8;
}

template <int D>
cudaError_t launch_d(const PagedDesc& a, int num_sms, void* workspace, cudaStream_t stream) {
    PgArgs g;
    std::memset(&g, 0, sizeof(g));
    g.a = a;
    g.team = team_of(a);
    g.sub = a.page_size < kKT ? a.page_size : kKT;
    int ctas = num_sms < kPagedMaxCtas ? num_sms : kPagedMaxCtas;
    ctas = ctas / g.team * g.team;
    if (ctas < g.team) ctas = g.team;
    const PgScratch sc = scratch_of(kPagedMaxCtas, D);
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    g.part_m = reinterpret_cast<float*>(ws + sc.m);
    g.part_l = reinterpret_cast<float*>(ws + sc.l);
    g.part_o = reinterpret_cast<float*>(ws + sc.o);
    g.head = reinterpret_cast<int4*>(ws + sc.head);
    const int64_t cols = (int64_t)a.Hk * D, pool = a.pages * a.page_size;
    CUtensorMap tk, tv, tkn, tvn;
    if (!encode_rows(&tk, a.k_pool, pool, cols, D, g.sub) || !encode_rows(&tv, a.v_pool, pool, cols, D, g.sub))
        return cudaErrorInvalidValue;
    tkn = tk;
    tvn = tv;
    if (a.tree && (!encode_rows(&tkn, a.k_new, a.rows, cols, D, kKT) || !encode_rows(&tvn, a.v_new, a.rows, cols, D, kKT)))
        return cudaErrorInvalidValue;
    cudaError_t e = set_smem_once(reinterpret_cast<const void*>(paged_tc_kernel<D>), (int)Cfg<D>::kSmem);
    if (e != cudaSuccess) return e;
    paged_tc_kernel<D><<<ctas, kThreads, Cfg<D>::kSmem, stream>>>(tk, tv, tkn, tvn, g);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int64_t most = (int64_t)a.max_rows * a.G;
    const unsigned rows8 = (unsigned)((most < kM ? most : kM) + 7) / 8;
    return launch_pdl(paged_merge_kernel<D>, dim3((unsigned)ctas, rows8), dim3(256), 0, stream, g);
}

}  // namespace

bool paged_tc_supported(const PagedDesc& a) {
    const bool page = a.page_size % kKT == 0 || a.page_size == 8 || a.page_size == 16 || a.page_size == 32;
    return (a.D == 64 || a.D == 128) && page && a.pages > 0 && a.pages * a.page_size < ((int64_t)1 << 31) - 256 &&
           (int64_t)a.max_rows * a.G < ((int64_t)1 << 30);
}

size_t paged_tc_workspace(const PagedDesc& a) { return scratch_of(kPagedMaxCtas, a.D).total; }

cudaError_t launch_paged_tc(const PagedDesc& a, int num_sms, void* workspace, cudaStream_t stream) {
    return a.D == 128 ? launch_d<128>(a, num_sms, workspace, stream) : launch_d<64>(a, num_sms, workspace, stream);
}

unsigned int paged_take_device_error() {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_paged_device_error, sizeof(v)) != cudaSuccess) return 0;
    if (v) {
        const unsigned int zero = 0;
        cudaMemcpyToSymbol(g_paged_device_error, &zero, sizeof(zero));
    }
    return v;
}

}  // namespace vtmu
