// paged_tc.cu -- attention of a ragged batch over a paged cache on the tcgen05
// tensor cores, headDim 64 or 128: single tokens, short runs, prompt chunks
// and trees of drafted tokens through one kernel.
//
// Mathematics.  For request b and KV head hk the T rows x G heads of the group
// are virtual rows v = t G + g; up to 128 of them (a row block) meet the same
// keys:   x2[v, s] = log2 e * softcap(scale q_v.k_s),  m = running max,
//         p = 2^(x2 - m),  l = sum p,  o = sum p v_s,  out = o / l.
// Both products run on f16 operands that carry 22 bits of an f32: an element x
// times a power of two (exact) is hi + lo with hi, lo in f16, and x.y = lo.hi +
// hi.lo + hi.hi, summed in f32.  What is dropped or rounded is at most 2^-22
// of the row's largest element.  Three f16 products cost 1.5 passes of a tf32
// one, so this is twice as fast as splitting into tf32 halves, at the same
// precision, and halves the bytes that the MMAs read from shared memory.  The
// power is 2^6 for a row of K or V whose largest element lies in [2^-9, 2^9), and
// one of its own for a row of Q and for any other row of K or V; those
// multiply the scores and the probabilities.  P has
// 2^11 as a factor, so that f16 holds small ones too; l has it as well.  (A weight is so
// kept to 2^-36 of the row's largest; in a tile with value rows that have a power of
// their own, the product of weight and value to 2^-36 of the tile's largest one.)  A
// row's reference maximum moves only when it is beaten by more than 2^4, so
// that the output seldom needs to be multiplied by alpha.
//
// Split of the work.  The lengths are on the device, so the launch is one
// persistent CTA per SM and the CTAs divide the 64-key tiles of all (request,
// KV head, row block) units evenly among themselves: CTA c takes tiles
// [total c / n, total (c + 1) / n) of their concatenation.  A unit inside one
// CTA is finished there; a unit cut by a boundary leaves partials (m, l, o / l) that
// paged_merge_kernel joins by the log-sum-exp rule, always in the same order.
// With more than 128 virtual rows per KV head, teams of R CTAs walk the same
// tiles for R row blocks at the same time, so the tiles come from HBM once (two blocks,
// 0.95 GB of cache: 0.97 GB read).
//
// Tiles of 64 keys, M = 128 virtual rows (padded: the MMAs of a tile take 1540
// cycles, its 64 KB 2800 at this SM's share of HBM, so padding costs no
// bandwidth).  Warps:
//   0, 2    page ids (32 at a time, one per lane) and TMA loads of f32 K and V tiles, one
//           box per page (with a box for each group of 8 rows the one warp that issued
//           them fell behind on pages of 16); drafted rows come as one tile of their own from k_new / v_new; rows of
//           no page are read out of bounds, as zeros;
//   1       the MMAs: S(n) = Q.K^T, then O(n - 1) = P.V;
//   4 - 7   a piece's queries to TMEM, and the fold acc = acc alpha + O of every two tiles
//           (kGroup: no sum runs long inside the pipe); acc stays in TMEM, so that 20
//           warps fit the registers;
//   8 - 11  softmax, thread = virtual row: no exchange between threads; P goes
//           back to TMEM over S as the A operand of P.V.  It waits for the values between the
//           maximum and the probabilities, since their scales go into P (waiting after
//           both was 1 to 2 % faster, but then a scale met weights that f16 had lost);
//   12 - 19 split: f32 rows to f16 hi and lo in place (K K-major, V MN-major: the same
//           bytes), four warps for the keys and four for the values.
// TMEM: Q hi, lo (D columns), S / P two buffers (128), O and its running sum (2 D).
// Every wait is bounded; a wait that gives up sets a bit of the device flag.
//
// Measured, headDim 128, 32 heads over 8: one row for each of 32 requests of 517 to 8111
// rows, pages of 16: 251-283 us for 1.176 GB, 4.2-4.7 TB/s (61-69 % of the copy
// rate).  Trees of 64 rows on 8 requests of 16384 to 32704, pages of 64: 579-622 us
// for 217 GFLOP, 348-374 TFLOP/s of f32 products, 54-58 % of a third of the f16 rate.
// What bounds it: the chain P.V(n - 1), S(n + 1), softmax(n + 1) on two score buffers:
// 1900-2300 cycles of softmax a tile, one thread per row, against 1540 of MMAs and
// the hand-overs between them.
#include <cstring>
#include <mutex>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_fp16.h>

#include "attn_common.cuh"
#include "launch_cache.h"
#include "paged.cuh"
#include "paged_kernels.h"
#include "pdl.cuh"
#include "softcap.cuh"
#include "tcgen05_ops.cuh"
#include "tma_sync.cuh"

namespace vtmu {

__device__ unsigned int g_paged_device_error;

namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int kKT = 64;        // keys per tile
constexpr int kM = 128;        // virtual rows per row block
constexpr int kThreads = 640;
// Warps of each role (its TMEM lanes: 32 (warp % 4)).
constexpr int kFoldWarp = 4, kSoftmaxWarp = 8, kSplitWarp = 12, kFoldWarps = 4;
constexpr int kFirst = 1 << 16, kLast = 1 << 17, kBad = 1 << 18;  // a piece's first and last tile; values that are not finite
constexpr int kPShift = 11;    // probabilities are scaled by 2^11 in f16
constexpr float kFar = 0x1p20f;  // base-2 scores from here on take the exact route
constexpr float kLazyLog2 = 4.f;  // and a row's reference maximum moves when beaten by more than 2^4: 2^15 at most
// Tiles that one accumulator takes before it is folded.  The tensor cores round their sums
// towards zero at every step: on 32 single-token requests the error against 64 bits is
// 5.6e-7 with one tile, 7.8e-7 with two, 9.3e-7 with three, 1.1e-6 with four.  One tile
// takes 2 % longer than two there (282 and 276 us side by side) and as long on large
// trees; four were 4 % faster than two.
constexpr int kGroup = 2;
constexpr int kRing = 8;       // what a tile leaves for later roles
static_assert(kRing >= kGroup + 2 && (kRing & (kRing - 1)) == 0, "a slot outlives its last reader");

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
    float* part_o;       // [2 CTAs][128][D], divided by l: of the output's size
    float* odd;          // [CTAs][128][D]: values that are not finite
    uint64_t* odd_rows;  // [CTAs][kRing][128]: such rows of a tile that a virtual row sees
    int4* head;          // [CTAs]: the unit that a CTA starts and others go on with
};

template <int D>
struct Cfg {
    static constexpr int kSlots = D == 128 ? 6 : 12;              // tiles: K(n), V(n), K(n + 1), ..
    static constexpr uint32_t kTile = kKT * D * 4;
    // A tile is a run of groups of 8 rows, a group a run of blocks [8 rows x 128 bytes]
    // (32 f32, or 64 f16 hi or lo; a swizzle atom), one for each 32 elements of the head.
    static constexpr int kBlocks = D / 32;
    static constexpr uint32_t kGroupRows = kBlocks * 1024;
    static constexpr int kSplitWarps = D == 128 ? 4 : 2;          // warps that split a tile
    static constexpr uint32_t kColQhi = 0, kColQlo = D / 2, kColS = D, kColO = D + 2 * kKT, kColAcc = kColO + D;
    static constexpr uint32_t kTmemCols = 512;
    static constexpr size_t kSmem = 1024 + (size_t)kSlots * kTile + (kPagedMaxRequests + 1) * 8;
    static_assert(kColAcc + D <= kTmemCols, "TMEM budget");
    static_assert(kSmem + 24 * 1024 <= 232448, "shared memory budget");
    static_assert(kSlots % 2 == 0, "K in the even slots, V in the odd ones");
    static_assert(kRing >= kSlots / 2 + 2, "the splitters are kSlots / 2 tiles ahead of scores that the softmax is behind by one");
};

// ---- the list of tiles --------------------------------------------------------------
// One request: packed rows [row0, row0 + T) are computed, n of them exist (their
// last one is the last row of the cache without a tree), len rows are cached.
struct Req {
    int row0, T, len, n;
};
struct Tiles {
    int lo_tile;  // first tile of the window's range
    int n_sink;   // tiles of sinks before it, or all of them without a main tile
    int n_main;
    int nt;       // with the drafted rows' tile; at least 1 when there are rows
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
__device__ __forceinline__ Tiles tiles_of(const PagedDesc& a, const Req& r) {
    Tiles t;
    int64_t lo = 0;
    if (a.window > 0) lo = clamp64((a.tree ? (int64_t)r.len : (int64_t)r.len - r.n) - a.window + 1, 0, r.len);
    t.lo_tile = (int)(lo / kKT);
    t.n_main = lo < r.len ? (int)(((int64_t)r.len + kKT - 1) / kKT) - t.lo_tile : 0;
    // Where the window leaves nothing of the cache (a tree's, at most 1), no main tile holds
    // the sinks of the cache's last tile.
    const int64_t sink_tiles = (min(a.sinks, (int64_t)r.len) + kKT - 1) / kKT;
    t.n_sink = (int)(t.n_main > 0 ? min(sink_tiles, (int64_t)t.lo_tile) : sink_tiles);
    t.nt = t.n_sink + t.n_main + a.tree;
    if (r.T == 0) t.nt = 0;
    else if (t.nt == 0) t.nt = 1;
    return t;
}

// A piece of a unit: what one CTA walks through, role by role.  Each warp keeps
// its place in the list in shared memory (the roles' registers are full).
struct Seg {
    long long pos, end;  // tiles left to this CTA
    int next_b;          // request of tile pos, or one before it
    int row0, T, len, n; // Req
    int lo_tile, n_sink, n_ctx, nt;  // Tiles; n_ctx: tiles of the cache, the drafted rows' tile follows
    int b, hk, rb;
    int u0, u1;          // tiles of the unit, this CTA's
    int slot;            // partial slot: 0 continues a unit, 1 starts one; -1: the whole unit
    int last_team;       // slot 1: the team that ends the unit
};

// This CTA's share of the list.  One lane.
__device__ __noinline__ void walk_start(const PgArgs& g, const long long* prefix, Seg& s) {
    const int c = blockIdx.x / g.team;
    const long long total = prefix[g.a.B];
    const long long teams = max(min((long long)(gridDim.x / g.team), total), 1ll);
    s.pos = c < teams ? total * c / teams : 0;
    s.end = c < teams ? total * (c + 1) / teams : 0;
    int b = 0, hi = g.a.B;  // the last request whose prefix is at most pos
    while (hi - b > 1) {
        const int mid = (b + hi) >> 1;
        if (prefix[mid] <= s.pos) b = mid; else hi = mid;
    }
    s.next_b = b;
}

// The next piece of a unit that this CTA has rows of; false at the end.  A
// piece may be empty (u1 <= u0) where causality leaves its tiles unseen.  One lane.
__device__ __noinline__ bool walk_next(const PgArgs& g, const long long* prefix, Seg& s) {
    const PagedDesc& a = g.a;
    const int team = g.team, member = blockIdx.x % team;
    const long long total = prefix[a.B];
    const long long teams = max(min((long long)(gridDim.x / team), total), 1ll);
    while (s.pos < s.end) {
        int b = s.next_b;
        while (prefix[b + 1] <= s.pos) ++b;
        s.next_b = b;
        const Req r = load_req(a, b);
        const Tiles t = tiles_of(a, r);
        const int blocks = (r.T * a.G + kM - 1) / kM, groups = (blocks + team - 1) / team;
        const long long rel = s.pos - prefix[b], unit = rel / t.nt;
        const int u0 = (int)(rel - unit * t.nt);
        int u1 = (int)min((long long)t.nt, u0 + (s.end - s.pos));
        const long long first = s.pos - u0;
        s.pos += u1 - u0;
        const int rb = (int)(unit % groups) * team + member;
        if (rb >= blocks) continue;
        s.slot = u0 > 0 ? 0 : u1 < t.nt ? 1 : -1;
        s.last_team = (int)(((first + t.nt) * teams - 1) / total);
        if (!a.tree) {  // tiles past the block's last row's position
            const int t_last = (min((rb + 1) * kM, r.T * a.G) - 1) / a.G;
            const int p_last = r.len - r.n + t_last;
            const int seen = p_last < 0 ? 0 : p_last / kKT + 1 - t.lo_tile;
            int cap = t.n_sink + max(seen, 0);
            if (cap < 1) cap = 1;  // a unit always has a first tile, so that its rows are written
            u1 = min(u1, cap);
        }
        s.row0 = r.row0;
        s.T = r.T;
        s.len = r.len;
        s.n = r.n;
        s.lo_tile = t.lo_tile;
        s.n_sink = t.n_sink;
        s.n_ctx = t.n_sink + t.n_main;
        s.nt = t.nt;
        s.b = b;
        s.hk = (int)(unit / groups);
        s.rb = rb;
        s.u0 = u0;
        s.u1 = u1;
        return true;
    }
    return false;
}
// The same for a whole warp.
__device__ __forceinline__ bool warp_next(const PgArgs& g, const long long* prefix, Seg& s) {
    __syncwarp();  // every lane is done with the last piece
    int more = 0;
    if ((threadIdx.x & 31) == 0) more = walk_next(g, prefix, s);
    return __shfl_sync(FULL, more, 0) != 0;  // orders lane 0's writes before the other lanes' reads
}

// First key of tile u, or -1 for the drafted rows' tile (n_sink, n_ctx, lo_tile: Seg's).
__device__ __forceinline__ int tile_key(int n_sink, int n_ctx, int lo_tile, int tree, int u) {
    const int key = (u < n_sink ? u : lo_tile + u - n_sink) * kKT;
    return u < n_ctx ? key : tree ? -1 : 0;  // 0: a unit without keys
}
// Rows of the tile that hold keys.
__device__ __forceinline__ int tile_rows(const Seg& s, int key) {
    return key < 0 ? min(s.T, kKT) : max(min(s.len - key, kKT), 0);
}

// Tiled TMA loads of 3 and 4 dimensions, as tma_load_2d.
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];\n" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];\n" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
        : "memory");
}

// ---- f16 operands ---------------------------------------------------------------------
// Descriptor of an f16 kind MMA: f32 accumulator, A K-major, B K-major or (mn) MN-major.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool mn) {
    return (1u << 4) | (mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// Shared-memory descriptors of a tile's hi (or lo) blocks with the 128-byte swizzle, groups
// of 8 rows `group` bytes apart.  K-major: 64 elements of a row along K.  MN-major: the
// rows are K, and the next 64 elements of a row lie two blocks on.
__device__ __forceinline__ uint64_t smem_desc_rows(const void* tile, uint32_t group, uint32_t next) {
    const uint64_t addr = smem_u32(tile);
    uint64_t d = (addr >> 4) & 0x3FFFull;
    d |= (uint64_t)(next >> 4) << 16;
    d |= (uint64_t)(group >> 4) << 32;
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

// Barrier `id` over `threads` threads; the AND of `v` over them.
__device__ __forceinline__ bool sync_and(int id, int threads, bool v) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n bar.red.and.pred p, %2, %3, q;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(id), "r"(threads)
        : "memory");
    return r != 0;
}

// True for one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
    return r != 0;
}

// The power of two of a row whose largest |element| has the bits `top`: its
// exponent, kept where both the scale and its inverse are normal and sums of
// scaled probabilities stay finite.
__device__ __forceinline__ uint32_t row_exponent(uint32_t top) {
    const uint32_t e = top >> 23;
    return e < 27u ? 27u : e > 253u ? 253u : e;
}
__device__ __forceinline__ float pow2_of(uint32_t biased) { return __uint_as_float(biased << 23); }

// A pair of f32 as f16 pairs hi and lo.
__device__ __forceinline__ void split2(uint64_t x, uint32_t& hi, uint32_t& lo) {
    float x0, x1;
    f2_unpack(x, x0, x1);
    const __half2 h = __floats2half2_rn(x0, x1);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(x0 - f.x, x1 - f.y);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = *reinterpret_cast<const uint32_t*>(&l);
}

// The largest of t and |x.x| .. |x.w|; NaN if one of them is.
__device__ __forceinline__ float abs_top(float t, const float4& x) {
    float r;
    asm("{\n .reg .f32 u;\n max.NaN.f32 u, %1, %2, %3;\n max.NaN.f32 %0, u, %4, %5;\n}\n"
        : "=f"(r)
        : "f"(t), "f"(fabsf(x.x)), "f"(fabsf(x.y)), "f"(fabsf(x.z)), "f"(fabsf(x.w)));
    return r;
}
__device__ __forceinline__ float nan_max(float x, float y) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}

__device__ __forceinline__ float finite_or_zero(float x) {
    return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u ? 0.f : x;
}

__device__ __forceinline__ float4 lds4(uint32_t at) {
    float4 x;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(at));
    return x;
}
__device__ __forceinline__ void sts4(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// Rows whose largest |element| lies in [2^-9, 2^9) (or is zero) are taken times kScale:
// f16 then holds hi and lo to 2^-22 of that element, as it does with a power of
// two of the row's own, which the other rows take (a second look at them, in
// global memory: rare). One pass over the tile instead of two: its shared-memory
// traffic is what bounds the kernel.
constexpr float kScale = 64.f, kUnscale = 1.f / 64.f, kTopMost = 512.f, kTopLeast = 1.f / 512.f;
// The running output has the factors of P and V, 2^17, and up to 2^4 and the number of keys
// more: from the first tile on whose largest product of weight and value passes 2^kBigLog2 a row's is
// kept times kBigUnit, where the largest products, 2^132, fit and ordinary ones are far from the smallest
// normal number.
constexpr float kBigLog2 = 50.f, kBigUnit = 0x1p-64f;

// 64 elements of a row of a tile (two blocks from `at` on, swizzled by sw = (row % 8)
// 16) times kScale as f16: hi over the first block, lo over the second, in place:
// chunk c (16 bytes) of both takes the elements that chunk c of the two blocks had,
// 4 c .. 4 c + 3 and 32 + 4 c .. 32 + 4 c + 3.  (So a tile's elements come in
// another order; the queries are laid out in the same one, and the fold puts the
// outputs back.)  A short loop on purpose: five warps with code of their own share a
// scheduler, and unrolled it ran at the rate of instruction fetches.  Returns the
// largest |element| (NaN if one is).
__device__ __forceinline__ float row_split(uint32_t at, uint32_t sw) {
    const uint64_t s2 = f2_pack(kScale, kScale);
    float t = 0.f;
#pragma unroll 2
    for (uint32_t c = 0; c < 128; c += 16) {
        const uint32_t to = at + (c ^ sw);
        const float4 x = lds4(to), y = lds4(to + 1024);
        t = abs_top(abs_top(t, x), y);
        uint32_t h[4], l[4];
        split2(f2_mul(f2_pack(x.x, x.y), s2), h[0], l[0]);
        split2(f2_mul(f2_pack(x.z, x.w), s2), h[1], l[1]);
        split2(f2_mul(f2_pack(y.x, y.y), s2), h[2], l[2]);
        split2(f2_mul(f2_pack(y.z, y.w), s2), h[3], l[3]);
        sts4(to, h[0], h[1], h[2], h[3]);
        sts4(to + 1024, l[0], l[1], l[2], l[3]);
    }
    return t;
}
// First element of the c-th (0 .. D / 4 - 1) group of four in a tile's order.
__device__ __forceinline__ int tile_order(int c) { return (c >> 4) * 64 + (c & 1) * 32 + ((c >> 1) & 7) * 4; }

// Row k of a tile (first key `key` of request b, or its drafted rows) in global memory,
// KV head hk; null for a page id outside the pool.
__device__ __forceinline__ const float* global_row(const PagedDesc& a, const float* pool, const float* fresh, int b, int key,
                                                   int k, int hk) {
    if (key < 0) return fresh + ((packed_rows(a.cu_rows, b, a.B, a.rows).row0 + k) * a.Hk + hk) * a.D;
    const int64_t page = __ldg(a.block_table + (int64_t)b * a.max_pages + (key + k) / a.page_size);
    if (page < 0 || page >= a.pages) return nullptr;
    return pool + ((page * a.page_size + (key + k) % a.page_size) * a.Hk + hk) * a.D;
}

// A row outside row_split's range once more, elements 64 half .. of it: with its own
// power of two, which is returned.  Values that are not finite become zeros
// (`odd`), keys that are not finite stay so.
__device__ __noinline__ float row_rescue(const float* row, int D, int half, bool values, uint32_t at, uint32_t sw, bool* odd) {
    float t = 0.f, all = 0.f;  // of the finite elements; of all
    for (int d = 0; d < D; d += 4) {
        float4 x = *reinterpret_cast<const float4*>(row + d);
        all = abs_top(all, x);
        x = make_float4(finite_or_zero(x.x), finite_or_zero(x.y), finite_or_zero(x.z), finite_or_zero(x.w));
        t = abs_top(t, x);
    }
    *odd = !(all < __int_as_float(0x7f800000));
    if (*odd && !values) t = 1.f;
    t = fminf(fmaxf(t, 0x1p-125f), 0x1p126f);  // the scale and its inverse are normal numbers
    const uint32_t e = __float_as_uint(t) & 0x7f800000u;  // 2^E in f32; 2^-E is 0x7f000000 - e
    const float s = __uint_as_float(0x7f000000u - e);
    for (int c = 0; c < 8; ++c) {
        float x[8];
        for (int i = 0; i < 8; ++i) {
            x[i] = row[tile_order(16 * half + 2 * c + (i >> 2)) + (i & 3)];
            if (values) x[i] = finite_or_zero(x[i]);
        }
        uint32_t h[4], l[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) split2(f2_pack(x[2 * i] * s, x[2 * i + 1] * s), h[i], l[i]);
        sts4(at + ((c << 4) ^ sw), h[0], h[1], h[2], h[3]);
        sts4(at + 1024 + ((c << 4) ^ sw), l[0], l[1], l[2], l[3]);
    }
    return __uint_as_float(e);
}

// One tile of f32 rows to f16 hi and lo, in place; the rows' inverse scales to
// `scale`.  TMA leaves 32 elements (128 bytes) of a row in a row of each block of its
// group, 128-byte swizzled; a thread takes 64 elements of one row (two blocks, which
// become their hi and lo), neighbouring lanes neighbouring rows, so that the swizzle makes
// its 16-byte accesses free of bank conflicts.  headDim 128: lanes 0 - 15 the first
// halves of 16 rows, lanes 16 - 31 the second ones.  Rows past `rows` are
// zeros.  In value tiles elements that are not finite become zeros and `bad` gets the
// rows that had one (they are added in the fold, to the rows that see them
// only); in key tiles they make their own scores not finite, which the mask
// discards.  `rescued` tells whether a row has a scale of its own.
template <int D>
__device__ __forceinline__ void split_tile(const PagedDesc& a, bool values, uint32_t tile, float* scale, uint32_t* bad,
                                           uint8_t* rescued, const Seg& s, int key, int w, int lane) {
    const int half = D == 128 ? lane >> 4 : 0, row = D == 128 ? 16 * w + (lane & 15) : 32 * (w & 1) + lane;
    uint32_t at = tile + (row >> 3) * Cfg<D>::kGroupRows + half * 2048 + (row & 7) * 128;
    asm volatile("" : "+r"(at));  // addresses are worked out here, not kept over the tile loop
    const uint32_t sw = (row & 7) << 4;
    const int rows = tile_rows(s, key);
    if (rows < kKT && row >= rows) {  // the last tile of a cache, or drafted rows
        for (int c = 0; c < 16; ++c) sts4(at + (c >> 3) * 1024 + (c & 7) * 16, 0, 0, 0, 0);
    }
    float t = row_split(at, sw), unscale = kUnscale;
    if constexpr (D == 128) t = nan_max(t, __shfl_xor_sync(FULL, t, 16));
    uint32_t odd_rows = 0;
    const bool rescue = !(t < kTopMost) || (t < kTopLeast && t > 0.f);
    const bool any = __any_sync(FULL, rescue);
    if (any) {
        bool odd = false;
        if (rescue) {
            const float* src = global_row(a, values ? a.v_pool : a.k_pool, values ? a.v_new : a.k_new, s.b, key, row, s.hk);
            if (src) unscale = row_rescue(src, D, half, values, at, sw, &odd);
        }
        odd_rows = __ballot_sync(FULL, odd);
    }
    if (half == 0) scale[row] = unscale;
    if (lane == 0) {
        rescued[w] = any;
        if (values) bad[w] = D == 128 ? odd_rows & 0xffffu : odd_rows;
    }
}

// mbar_wait, bounded in the same way, that looks at the clock after 4096 tries and then
// after every 64: reading the global timer takes as long as a whole hand-over.
__device__ __noinline__ bool wait_timed(uint64_t* bar, uint32_t parity) {
    const uint64_t t0 = global_ns();
    do {
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (mbar_try_wait(bar, parity)) return true;
    } while (global_ns() - t0 <= kWaitLimitNs);
    return false;
}
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity) {
#pragma unroll 1
    for (int i = 0; i < 4096; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    return wait_timed(bar, parity);
}
// A wait of the warps that share a tile: the first one looks at the mbarrier while the
// others sleep at barrier `id` and leave it the issue slots, then each looks
// once, for what the mbarrier orders.
__device__ __forceinline__ bool team_wait(bool leads, int id, int threads, uint64_t* bar, uint32_t parity) {
    bool ok = true;
    if (leads) ok = __all_sync(FULL, wait_for(bar, parity));
    ok = sync_and(id, threads, ok);
    return ok && (leads || __all_sync(FULL, wait_for(bar, parity)));
}

// Rows of a value tile with elements that are not finite, from what its warps found.
template <int D>
__device__ __forceinline__ uint64_t bad_rows(const uint32_t* b) {
    const uint4 v = *reinterpret_cast<const uint4*>(b);
    return D == 128 ? (v.x | v.y << 16) | (uint64_t)(v.z | v.w << 16) << 32 : (v.x | v.z) | (uint64_t)(v.y | v.w) << 32;
}
// Values that are not finite would reach every row of a tile through 0 x inf =
// NaN, so the tile has zeros in their place and they are added here, to the rows
// that see them.  `rows_bad`: such keys of the tile; columns col .. col + n of each
// go to `odd` (thread-private; `more`: it holds earlier ones already).
__device__ __noinline__ bool add_odd_values(const PagedDesc& a, int4 tile, uint64_t rows_bad, float* odd, int col, int n,
                                            bool more) {
    while (rows_bad) {
        const int k = __ffsll((long long)rows_bad) - 1;
        rows_bad &= rows_bad - 1;
        const float* src = global_row(a, a.v_pool, a.v_new, tile.y, tile.z, k, tile.w);
        if (!src) continue;
        src += col;
        for (int d = 0; d < n; ++d) {
            const float x = src[d];
            const float y = (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u ? x : 0.f;
            odd[d] = more ? odd[d] + y : y;
        }
        more = true;
    }
    return more;
}
// ... and from there to the row's output once it is written.
__device__ __noinline__ bool join_odd_values(float* to, const float* odd, int n) {
    for (int d = 0; d < n; ++d) to[d] += odd[d];
    return false;
}

// Keys of a tile that a row sees: in the cache [lo, hi] and those before `sinks`, among the
// drafted rows its mask's, with a window those near its position p.
__device__ __noinline__ uint64_t tile_mask(const PagedDesc& a, const Seg& s, int key, int hi, int lo, int sinks, int p, int t) {
    auto below = [](int c) -> uint64_t { return c <= 0 ? 0ull : c >= 64 ? ~0ull : (1ull << c) - 1; };
    if (key >= 0) return below(hi - key + 1) & (~below(lo - key) | below(sinks - key));
    uint64_t see = __ldg(reinterpret_cast<const unsigned long long*>(a.masks) + s.row0 + t) & below(s.T);
    if (a.window > 0)
        for (int j = 0; j < s.T; ++j)
            if (__ldg(a.positions + s.row0 + j) <= p - a.window) see &= ~(1ull << j);
    return see;
}

// ---- softmax of one row of a tile -----------------------------------------------------
// What a thread needs of the tile: its scores (TMEM columns `at`), the keys' and
// values' scales, the mask.
struct RowTile {
    uint32_t at;
    uint64_t see;         // keys that the row sees (not read when WHOLE)
    float mul;            // a score of the MMA times this is one in base-2 units (the argument of tanh with a cap)
    float cap;            // softcap in base-2 units
};

// 32 scores from key 32 c on, masked, in base-2 units with a cap, else still to be
// multiplied by r.mul (in the exponent's FMA).
template <bool CAP, bool WHOLE>
__device__ __forceinline__ void row_scores(const RowTile& r, int c, float (&x)[32]) {
    tmem_ld32(r.at + 32 * c, x);
    tmem_wait_ld();
    if constexpr (CAP) softcap_tile<32>(x, r.mul, r.cap);
    if constexpr (!WHOLE) {
        const uint32_t bits = (uint32_t)(r.see >> (32 * c));
#pragma unroll
        for (int k = 0; k < 32; ++k) x[k] = (bits >> k) & 1u ? x[k] : -INFINITY;
    }
}

// The online softmax's step in two passes over the scores (64 of them do not fit the
// registers at once).  First the largest one, in base-2 units.
template <bool CAP, bool WHOLE>
__device__ __forceinline__ float row_max(const RowTile& r) {
    float mt = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < 2; ++c) {
        float x[32];
        row_scores<CAP, WHOLE>(r, c, x);
#pragma unroll
        for (int k = 0; k < 32; k += 2) mt = fmaxf(fmaxf(mt, x[k]), x[k + 1]);
    }
    return CAP ? mt : mt * r.mul;
}

// 32 probabilities as f16 hi and lo over their scores' columns.
__device__ __forceinline__ void store_probs(uint32_t at, const float (&phi)[16], const float (&plo)[16]) {
    tmem_st16(at, phi);
    tmem_st16(at + 16, plo);
}
__device__ __forceinline__ void split_probs(uint64_t p, float& hi, float& lo) {
    uint32_t h, l;
    split2(p, h, l);
    hi = __uint_as_float(h);
    lo = __uint_as_float(l);
}

// Then P = 2^(score - mu + kPShift), which goes over the scores (keys 32 c .. as f16 hi in
// 16 columns, lo in 16).  Returns its sum.
template <bool CAP, bool WHOLE>
__device__ __forceinline__ float row_probs(const RowTile& r, float mu) {
    const float mul = CAP ? 1.f : r.mul, shift = (float)kPShift - mu;
    const uint64_t mul2 = f2_pack(mul, mul), shift2 = f2_pack(shift, shift);
    uint64_t sum0 = 0, sum1 = 0;
#pragma unroll 1
    for (int c = 0; c < 2; ++c) {
        float x[32];
        row_scores<CAP, WHOLE>(r, c, x);
        float phi[16], plo[16];
#pragma unroll
        for (int k = 0; k < 32; k += 4) {
            float e0, e1, e2, e3;
            f2_unpack(f2_fma(f2_pack(x[k], x[k + 1]), mul2, shift2), e0, e1);
            f2_unpack(f2_fma(f2_pack(x[k + 2], x[k + 3]), mul2, shift2), e2, e3);
            const uint64_t p0 = f2_pack(fast_exp2(e0), fast_exp2(e1)), p1 = f2_pack(fast_exp2(e2), fast_exp2(e3));
            sum0 = f2_add(sum0, p0);
            sum1 = f2_add(sum1, p1);
            split_probs(p0, phi[k / 2], plo[k / 2]);
            split_probs(p1, phi[k / 2 + 1], plo[k / 2 + 1]);
        }
        store_probs(r.at + 32 * c, phi, plo);
    }
    float a0, a1, b0, b1;
    f2_unpack(sum0, a0, a1);
    f2_unpack(sum1, b0, b1);
    return (a0 + a1) + (b0 + b1);
}

// The same two passes for a tile that has rows with scales of their own, or for rows
// with a far reference (both rare).  Keys: their scores times `ks` (null: keys without one).
template <bool CAP>
__device__ __forceinline__ void scaled_scores(const RowTile& r, const float* ks, int c, float (&x)[32]) {
    tmem_ld32(r.at + 32 * c, x);
    tmem_wait_ld();
    if (ks) {
#pragma unroll
        for (int k = 0; k < 32; ++k) x[k] *= ks[32 * c + k];
    }
    if constexpr (CAP) {
        softcap_tile<32>(x, r.mul, r.cap);
    } else {
#pragma unroll
        for (int k = 0; k < 32; ++k) x[k] *= r.mul;
    }
    const uint32_t bits = (uint32_t)(r.see >> (32 * c));
#pragma unroll
    for (int k = 0; k < 32; ++k) x[k] = (bits >> k) & 1u ? x[k] : -INFINITY;
}
template <bool CAP>
__device__ __noinline__ float scaled_max(const RowTile& r, const float* ks) {
    float mt = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < 2; ++c) {
        float x[32];
        scaled_scores<CAP>(r, ks, c, x);
#pragma unroll
        for (int k = 0; k < 32; ++k) mt = fmaxf(mt, x[k]);
    }
    return mt;
}
// Values (`vs` their scales, powers of two; null: values without one): the products
// p v decide, not the scales, since a value row of any size may weigh nothing, and one that
// weighs little may count.  So P takes the exponent E of its value row's scale, less the
// largest (score - mu + E) of the keys that are seen, rounded up: `lift`, which the
// tile's output gets back.  The sum of the probabilities has no part in it.
template <bool CAP>
__device__ __noinline__ float scaled_probs(const RowTile& r, const float* ks, const float* vs, float mu, float* lift) {
    auto exponent = [&](int k) -> float { return (float)((int)(__float_as_uint(vs[k]) >> 23) - 127); };
    float top = 0.f;
    if (vs) {
        top = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
            float x[32];
            scaled_scores<CAP>(r, ks, c, x);
#pragma unroll
            for (int k = 0; k < 32; ++k) top = fmaxf(top, (x[k] - mu) + exponent(32 * c + k));
        }
        top = ceilf(fmaxf(top, -300.f));  // nothing seen: any number does
    }
    *lift = top;
    float sum = 0.f;
#pragma unroll 1
    for (int c = 0; c < 2; ++c) {
        float x[32], phi[16], plo[16];
        scaled_scores<CAP>(r, ks, c, x);
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
            const float e0 = (x[k] - mu) + (float)kPShift, e1 = (x[k + 1] - mu) + (float)kPShift;
            const float p0 = fast_exp2(e0), p1 = fast_exp2(e1);
            sum += p0 + p1;
            split_probs(vs ? f2_pack(fast_exp2(e0 + (exponent(32 * c + k) - top)), fast_exp2(e1 + (exponent(32 * c + k + 1) - top)))
                           : f2_pack(p0, p1),
                        phi[k / 2], plo[k / 2]);
        }
        store_probs(r.at + 32 * c, phi, plo);
    }
    return sum;
}

// ---- the kernel -------------------------------------------------------------------------
template <int D, bool CAP>
__global__ void __launch_bounds__(kThreads, 1)
    paged_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ CUtensorMap tm_kn, const __grid_constant__ CUtensorMap tm_vn,
                    const __grid_constant__ PgArgs g) {
    using C = Cfg<D>;
    constexpr int ST = C::kSlots;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* tiles = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                            ~uintptr_t(1023));  // tile 2 n: K(n), 2 n + 1: V(n)
    long long* prefix = reinterpret_cast<long long*>(tiles + (size_t)ST * C::kTile);
    // A slot is loaded by TMA (full), split in place (ready), read by the MMAs (free).
    __shared__ __align__(8) uint64_t full[ST], ready[ST], freed[ST], q_full, s_full[2], p_full[2], o_full, o_free;
    __shared__ uint32_t tmem_base_s;
    __shared__ long long scan_s[kThreads / 32];
    __shared__ Seg seg_s[kThreads / 32];
    // What tile n leaves for the roles that come later, at n % kRing.  The splitters get to
    // tile n once S(n - kSlots / 2) is done, three tiles (headDim 128) or six (64), while the
    // softmax may still read the tile before that one; while a group of kGroup tiles waits
    // for its fold, the softmax gets two tiles further: S(n) is issued before P.V of
    // tile n - 1, which waits.
    __shared__ __align__(16) float k_scale[kRing][kKT], v_scale[kRing][kKT];
    __shared__ __align__(16) uint32_t v_bad[kRing][4];
    __shared__ __align__(8) uint8_t rescued[kRing][2][4];  // keys, values: a split warp's rows have a scale of their own
    __shared__ float q_scale[4][kM];             // by piece % 4
    __shared__ float2 fold_f[kRing][kM];         // alpha, output scale of such a tile
    __shared__ float row_inv[kRing][kM];         // last tile of a piece: 1 / l
    __shared__ __align__(16) int group_tag[kRing][4];  // by softmax warp, n + 1: tile n begins a group, its fold_f counts
    __shared__ int2 group_at[2];                 // a group's first and last tile
    __shared__ int4 tile_at[kRing];              // rows of the block (kFirst, kLast, kBad), request, first key, KV head

    const PagedDesc& a = g.a;
    const int warp = __shfl_sync(FULL, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // warp: uniform, to the compiler too

    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&ready[i], C::kSplitWarps);
            mbar_init(&freed[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
        }
        mbar_init(&q_full, kFoldWarps);
        mbar_init(&o_full, 2);  // the MMAs' commit, and an arrival that publishes group_at
        mbar_init(&o_free, kFoldWarps);
        fence_barrier_init();
    }
    if (warp == 1) tmem_alloc(&tmem_base_s, C::kTmemCols);
    if (threadIdx.x == 32) g.head[blockIdx.x] = make_int4(-1, 0, 0, 0);
    if (threadIdx.x < 4 * kRing) (&group_tag[0][0])[threadIdx.x] = 0;
    if (threadIdx.x < 4 * kRing)  // headDim 64: two words of a tile's four are never written
        (&v_bad[0][0])[threadIdx.x] = (&rescued[0][0][0])[threadIdx.x] = (&rescued[0][0][0])[4 * kRing + threadIdx.x] = 0;

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

    Seg& s = seg_s[warp];
    if (lane == 0) walk_start(g, prefix, s);

    if (warp == 0 || warp == 2) {
        // ---- producers: warp 0 the K tiles, warp 2 the V tiles -------------------------
        const int kv = warp >> 1;
        const CUtensorMap *tm = kv ? &tm_v : &tm_k, *tmn = kv ? &tm_vn : &tm_kn;
        if (lane == 0) prefetch_tensormap(tm);
        const int nsub = kKT / g.sub;
        const int nowhere = (int)(a.pages * a.page_size);  // a row out of bounds: zeros
        int n = 0;
        bool ok = true;
        while (ok && warp_next(g, prefix, s)) {
            int batch = -1, y_cur = nowhere;
            const int subs = (int)(((int64_t)s.len + g.sub - 1) / g.sub), u1 = s.u1, n_sink = s.n_sink, n_ctx = s.n_ctx, lo_tile = s.lo_tile;
            for (int u = s.u0; u < u1; ++u, ++n) {
                const int key = tile_key(n_sink, n_ctx, lo_tile, a.tree, u);
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
                const int it = 2 * n + kv, st = it % ST;
                if (it >= ST && !__all_sync(FULL, wait_for(&freed[st], (uint32_t)((it / ST - 1) & 1)))) {
                    raise_device_error(&g_paged_device_error, kErrPgFree);
                    ok = false;
                    break;
                }
                if (lane == 0) mbar_arrive_expect_tx(&full[st], C::kTile);
                __syncwarp();
                // A lane for each box: the groups of a page (or of the tile), all their blocks;
                // drafted rows, which start anywhere, one group at a time.
                unsigned char* dst = tiles + (size_t)st * C::kTile;
                if (key < 0) {
                    if (lane < kKT / 8)
                        tma_load_3d(dst + lane * C::kGroupRows, tmn, 0, s.row0 + 8 * lane, s.hk * C::kBlocks, &full[st]);
                } else if (lane < nsub) {
                    tma_load_4d(dst + lane * (g.sub / 8) * C::kGroupRows, tm, 0, 0, s.hk * C::kBlocks, y >> 3, &full[st]);
                }
            }
        }
        // No copy may be in flight when the CTA exits.
        const int slots = ST / 2;
        for (int j = n < slots ? 0 : n - slots; j < n; ++j)
            if (!wait_for(&full[(2 * j + kv) % ST], (uint32_t)(((2 * j + kv) / ST) & 1)))
                raise_device_error(&g_paged_device_error, kErrPgFree);
    } else if (warp == 1) {
        // ---- MMAs: the warp stays together and one elected lane issues (behind a
        // lane == 0 test an MMA took 45 cycles to issue, behind elect 10) ----
        constexpr uint32_t id_s = idesc_f16(kM, kKT, false), id_o = idesc_f16(kM, D, true);
        const uint32_t tm = __shfl_sync(FULL, tmem, 0);
        const uint64_t k0 = smem_desc_rows(tiles, C::kGroupRows, 16), v0 = smem_desc_rows(tiles, C::kGroupRows, 2048);
        int n = 0, piece = 0;
        // Groups of tiles share an accumulator: `len` tiles in the open one, the first
        // of them `from`; `groups` are closed.
        int len = 0, from = 0, groups = 0;
        bool ok = true;
        auto close = [&](int j) {
            if (elect_one()) {
                group_at[groups & 1] = make_int2(from, j);
                mbar_arrive(&o_full);
                mma_commit(&o_full);
            }
            __syncwarp();
            ++groups;
            len = 0;
        };
        auto pv = [&](int j, bool first, bool last) -> bool {  // O (+)= P(j).V(j)
            const int bf = j & 1, it = 2 * j + 1, st = it % ST;
            const uint32_t ph = (uint32_t)((j >> 1) & 1);
            if (!__all_sync(FULL, wait_for(&p_full[bf], ph) && wait_for(&ready[st], (uint32_t)((it / ST) & 1)))) {
                raise_device_error(&g_paged_device_error, kErrPgMma);
                return false;
            }
            if (len > 0 && (first || __any_sync(FULL, group_tag[j % kRing][lane & 3] == j + 1))) close(j - 1);
            if (len == 0) {
                from = j;
                if (groups > 0 && !__all_sync(FULL, wait_for(&o_free, (uint32_t)((groups - 1) & 1)))) {
                    raise_device_error(&g_paged_device_error, kErrPgMma);
                    return false;
                }
            }
            tc_fence_after();
            const uint32_t d = tm + C::kColO;
            const uint32_t p = tm + C::kColS + bf * kKT;  // 32 keys: hi in 16 columns, lo in 16
            const uint64_t vhi = v0 + st * (C::kTile >> 4);
            const uint64_t vlo = vhi + (1024 >> 4);
            if (elect_one()) {
                // 16 keys: 8 columns of P, two groups of V's rows.  The small products
                // come first: the accumulator's rounding (towards zero, at every step) then
                // meets the full sum a third as often.
#pragma unroll 2
                for (int k = 0; k < kKT / 16; ++k) {
                    const uint32_t phi = p + 32 * (k >> 1) + 8 * (k & 1), plo = phi + 16;
                    mma_f16_ts(d, plo, vhi + (2 * C::kGroupRows >> 4) * k, id_o, k > 0 || len > 0 ? 1u : 0u);
                    mma_f16_ts(d, phi, vlo + (2 * C::kGroupRows >> 4) * k, id_o, 1u);
                }
#pragma unroll 2
                for (int k = 0; k < kKT / 16; ++k)
                    mma_f16_ts(d, p + 32 * (k >> 1) + 8 * (k & 1), vhi + (2 * C::kGroupRows >> 4) * k, id_o, 1u);
                mma_commit(&freed[st]);
            }
            __syncwarp();
            if (++len == kGroup || last) close(j);
            return true;
        };
        bool prev_first = false, prev_last = false;
        while (ok && warp_next(g, prefix, s)) {
            const int u0 = s.u0, u1 = s.u1;
            for (int u = u0; u < u1; ++u, ++n) {
                const int it = 2 * n, st = it % ST;
                if (!__all_sync(FULL, (u > u0 || wait_for(&q_full, (uint32_t)(piece & 1))) &&
                                          wait_for(&ready[st], (uint32_t)((it / ST) & 1)))) {
                    raise_device_error(&g_paged_device_error, kErrPgMma);
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tm + C::kColS + (n & 1) * kKT;
                const uint64_t khi = k0 + st * (C::kTile >> 4), klo = khi + (1024 >> 4);
                if (elect_one()) {
                    // 16 dims: 8 columns of Q, 32 bytes of a K row.
                    auto off = [](int k) -> uint64_t { return (uint64_t)(k >> 2) * (2048 >> 4) + 2 * (k & 3); };
#pragma unroll 2
                    for (int k = 0; k < D / 16; ++k) {
                        mma_f16_ts(d, tm + C::kColQlo + 8 * k, khi + off(k), id_s, k > 0 ? 1u : 0u);
                        mma_f16_ts(d, tm + C::kColQhi + 8 * k, klo + off(k), id_s, 1u);
                    }
#pragma unroll 2
                    for (int k = 0; k < D / 16; ++k) mma_f16_ts(d, tm + C::kColQhi + 8 * k, khi + off(k), id_s, 1u);
                    mma_commit(&freed[st]);
                    mma_commit(&s_full[n & 1]);
                }
                __syncwarp();
                if (n > 0 && !pv(n - 1, prev_first, prev_last)) {
                    ok = false;
                    break;
                }
                prev_first = u == u0;
                prev_last = u == u1 - 1;
            }
            if (u1 > u0) ++piece;
        }
        if (ok && n > 0) pv(n - 1, prev_first, prev_last);
    } else if (warp >= kSoftmaxWarp && warp < kSoftmaxWarp + 4) {
        // ---- softmax: thread = virtual row -------------------------------------------
        const int i = threadIdx.x - 32 * kSoftmaxWarp;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        int n = 0, piece = 0, v_slot = 1;
        uint32_t v_phase = 0;
        bool ok = true;
        while (ok && warp_next(g, prefix, s)) {
            const int v = s.rb * kM + i, t = v / a.G;
            const bool alive = v < s.T * a.G;
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
            int p = a.tree ? s.len : s.len - s.n + t;
            if (a.tree && a.window > 0 && alive) p = __ldg(a.positions + s.row0 + t);
            const int hi = a.tree ? s.len - 1 : min(p, s.len - 1);
            const int lo = a.window > 0 ? (int)max((int64_t)p - a.window + 1, (int64_t)0) : 0;
            const int sinks = (int)min(a.sinks, (int64_t)s.len);
            float m = -INFINITY, l = 0.f, unit = 1.f;  // of the running output: 1 or kBigUnit
            bool was_scaled = false;
            const int rows = min(s.T * a.G - s.rb * kM, kM);
            const int u0 = s.u0, u1 = s.u1, n_sink = s.n_sink, n_ctx = s.n_ctx, lo_tile = s.lo_tile;
            // A warp without rows waits at the barrier that ends the piece; the first
            // warp, which always has one, arrives for it.
            const int arrivals = warp == kSoftmaxWarp ? 4 - (rows + 31) / 32 + 1 : 1;
            const bool idle = !__any_sync(FULL, alive);
            for (int u = idle ? u1 : u0; u < u1; ++u, ++n) {
                const int key = tile_key(n_sink, n_ctx, lo_tile, a.tree, u), nb = n % kRing, bf = n & 1;
                if (!__all_sync(FULL, wait_for(&s_full[bf], (uint32_t)((n >> 1) & 1)))) {
                    raise_device_error(&g_paged_device_error, kErrPgMma);
                    ok = false;
                    break;
                }
                // Keys of the tile that the row sees (a row of no request: anything).
                const bool all = !alive || (key >= 0 && hi - key >= kKT - 1 && lo <= key);
                const bool whole = __all_sync(FULL, all);
                tc_fence_after();
                RowTile rt;
                rt.at = tmem + lanes + C::kColS + bf * kKT;
                rt.see = ~0ull;
                rt.mul = q_scale[piece & 3][i] * kUnscale;
                rt.cap = a.cap_log2;
                if (!all) rt.see = tile_mask(a, s, key, hi, lo, sinks, p, t);
                const float* ks = nullptr;
                float mt;
                if (*reinterpret_cast<const uint32_t*>(rescued[nb][0])) {  // rare
                    ks = k_scale[nb];
                    rt.mul *= kScale;
                    mt = scaled_max<CAP>(rt, ks);
                } else {
                    mt = whole ? row_max<CAP, true>(rt) : row_max<CAP, false>(rt);
                }
                // m, the row's reference, moves when it is beaten.
                const bool moved = mt > m + kLazyLog2;
                const float mn = moved ? mt : m, mu = mn == -INFINITY ? 0.f : mn;
                float alpha = moved ? fast_exp2(m - mu) : 1.f;
                m = mn;
                // The values' scales go into P.
                if (!__all_sync(FULL, wait_for(&ready[v_slot], v_phase))) {
                    raise_device_error(&g_paged_device_error, kErrPgMma);
                    ok = false;
                    break;
                }
                if ((v_slot += 2) >= ST) {
                    v_slot = 1;
                    v_phase ^= 1;
                }
                const bool scaled = *reinterpret_cast<const uint32_t*>(rescued[nb][1]) != 0;
                // kPShift - mu rounds to a multiple that grows with mu: from 2^24 on P would
                // leave f16.  Past kFar the difference to mu comes before kPShift.
                const bool far = __any_sync(FULL, fabsf(mu) > kFar);
                float lift = 0.f, sum;
                if (ks || scaled || far)  // rare
                    sum = scaled_probs<CAP>(rt, ks, scaled ? v_scale[nb] : nullptr, mu, &lift);
                else
                    sum = whole ? row_probs<CAP, true>(rt, mu) : row_probs<CAP, false>(rt, mu);
                l = fmaf(l, alpha, sum);
                int flags = rows;
                // A tile with another reference or scale than the one before begins a group.
                if (__any_sync(FULL, (moved && alive) || unit != 1.f) || scaled || was_scaled) {
                    if (lift > kBigLog2 && unit == 1.f) alpha *= unit = kBigUnit;
                    float o_scale = unit;  // of the tile's output, times kScale
                    if (scaled) {
                        // Below 2^-126 the tile's output is lost, as its sums would be.
                        o_scale = fast_exp2(lift + (unit == 1.f ? 6.f : -58.f));
                        static_assert(kScale == 64.f && kBigUnit == 0x1p-64f, "their exponents");
                        const uint64_t bad = bad_rows<D>(v_bad[nb]);
                        if (bad) {  // which of them the row sees, for the fold
                            g.odd_rows[((int64_t)blockIdx.x * kRing + nb) * kM + i] = alive ? bad & rt.see : 0;
                            flags += kBad;
                        }
                    }
                    fold_f[nb][i] = make_float2(alpha, o_scale);
                    group_tag[nb][warp & 3] = n + 1;
                }
                was_scaled = scaled;
                if (u == u0) flags += kFirst;
                if (u == u1 - 1) {
                    flags += kLast;
                    if (s.slot >= 0) {
                        g.part_m[prow] = m;
                        g.part_l[prow] = l;
                    }
                    row_inv[nb][i] = l != 0.f ? 1.f / l / unit : 0.f;
                }
                if (i == 0) tile_at[nb] = make_int4(flags, s.b, key, s.hk);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_n(&p_full[bf], arrivals);
            }
            if (idle) {  // past the tiles of the piece
                n += u1 - u0;
                const int it = 2 * n + 1;
                v_slot = it % ST;
                v_phase = (uint32_t)((it / ST) & 1);
            }
            // One barrier a piece keeps the four warps' tile counts together; a failed
            // wait ends the role for all of them.
            ok = sync_and(1, 128, ok);
            ++piece;
        }
    } else if (warp >= kSplitWarp) {
        // ---- split: four warps the keys, four the values ------------------------
        const int w = warp & 3, side = (warp - kSplitWarp) >> 2;
        int n = 0;
        bool ok = true;
        while (ok && warp_next(g, prefix, s)) {
            const int u1 = s.u1, n_sink = s.n_sink, n_ctx = s.n_ctx, lo_tile = s.lo_tile;
            for (int u = s.u0; u < u1; ++u, ++n) {
                if (D == 64 && (n & 1) != (w >> 1)) continue;  // a tile's two warps of the four
                const int it = 2 * n + side, st = it % ST;
                // The warps that share the tile: four, or a pair.
                if (!team_wait(D == 128 ? w == 0 : (w & 1) == 0, 3 + side + (D == 128 ? 0 : w & 2), 32 * C::kSplitWarps, &full[st],
                               (uint32_t)((it / ST) & 1))) {
                    raise_device_error(&g_paged_device_error, kErrPgLoad);
                    ok = false;
                    break;
                }
                split_tile<D>(a, side != 0, smem_u32(tiles) + st * C::kTile, side ? v_scale[n % kRing] : k_scale[n % kRing],
                              v_bad[n % kRing], rescued[n % kRing][side], s,
                              tile_key(n_sink, n_ctx, lo_tile, a.tree, u), w, lane);
                asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");  // generic writes -> MMA
                __syncwarp();
                if (lane == 0) mbar_arrive(&ready[st]);
            }
        }
    } else if (warp >= kFoldWarp && warp < kFoldWarp + 4) {
        // ---- queries and fold: thread = virtual row -----------------------------------
        const int w = warp & 3, i = 32 * w + lane;
        const uint32_t lanes = (uint32_t)(32 * w) << 16;
        int n = 0, piece = 0;
        bool ok = true, odd = false;
        float *to = nullptr, *next_to = nullptr;  // where the row goes: this piece's, the next one's
        // Row i of the piece's block: q scaled by qk_mul, then as a row of a tile, with a
        // power of two of its own; two elements to a column of Q hi and Q lo.
        auto load_queries = [&]() {
            const int v = s.rb * kM + i, t = v / a.G;
            const bool alive = v < s.T * a.G;
            const float* q = a.q + (((int64_t)s.row0 + t) * a.H + (int64_t)s.hk * a.G + (v - t * a.G)) * D;
            auto load4 = [&](int d) -> float4 {
                if (!alive) return make_float4(0.f, 0.f, 0.f, 0.f);
                const float4 y = __ldg(reinterpret_cast<const float4*>(q + d));
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
            q_scale[piece & 3][i] = pow2_of(e);
#pragma unroll 1
            for (int c0 = 0; c0 < D / 2; c0 += 16) {
                float qh[16], ql[16];
#pragma unroll
                for (int c = 0; c < 16; c += 2) {
                    const float4 y = load4(tile_order((c0 + c) / 2));
                    uint32_t h0, l0, h1, l1;
                    split2(f2_pack(y.x * sc, y.y * sc), h0, l0);
                    split2(f2_pack(y.z * sc, y.w * sc), h1, l1);
                    qh[c] = __uint_as_float(h0);
                    qh[c + 1] = __uint_as_float(h1);
                    ql[c] = __uint_as_float(l0);
                    ql[c + 1] = __uint_as_float(l1);
                }
                tmem_st16(tmem + lanes + C::kColQhi + c0, qh);
                tmem_st16(tmem + lanes + C::kColQlo + c0, ql);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full);
            ++piece;
            next_to = s.slot < 0 ? a.out + (q - a.q)
                                 : g.part_o + ((int64_t)(2 * blockIdx.x + (s.slot > 0 ? 1 : 0)) * kM + i) * D;
        };
        // acc = acc alpha + O of group k (times kScale, as the tiles' values are); after a
        // piece's last tile to where the row goes.  Returns the tile after the group (0:
        // a wait gave up).
        auto fold = [&](int k) -> int {
            if (!__all_sync(FULL, wait_for(&o_full, (uint32_t)(k & 1)))) {
                raise_device_error(&g_paged_device_error, kErrPgMma);
                return 0;
            }
            tc_fence_after();
            const int2 group = group_at[k & 1];
            const int nb = group.x % kRing, ne = group.y % kRing;
            static_assert(kGroup <= 2, "nb and ne are all of the group's tiles");
            const int flags = tile_at[nb].x, flags_e = tile_at[ne].x, rows = flags & (kFirst - 1);
            const bool first = flags & kFirst, last = flags_e & kLast;
            if (32 * w < rows) {
                const float2 f = group_tag[nb][w] == group.x + 1 ? fold_f[nb][i] : make_float2(1.f, 1.f);
                const float fin = last ? row_inv[ne][i] * kUnscale : 1.f;
                const bool plain = __all_sync(FULL, (first || f.x == 1.f) && f.y == 1.f && !last);
                const uint64_t fx = f2_pack(f.x, f.x), fy = f2_pack(f.y, f.y), fin2 = f2_pack(fin, fin);
                const uint32_t at = tmem + lanes + C::kColO;
                if ((flags | flags_e) & kBad)  // rare
                    for (int j = group.x; j <= group.y; ++j) {
                        const uint64_t mask = g.odd_rows[((int64_t)blockIdx.x * kRing + j % kRing) * kM + i];
                        if ((tile_at[j % kRing].x & kBad) && i < rows && mask)
                            odd = add_odd_values(a, tile_at[j % kRing], mask, g.odd + ((int64_t)blockIdx.x * kM + i) * D, 0, D,
                                                 odd);
                    }
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 32) {
                    float x[32], y[32];
                    tmem_ld32(at + c0, x);
                    if (!first) tmem_ld32(at + (C::kColAcc - C::kColO) + c0, y);
                    tmem_wait_ld();
                    // The accumulator, and what the group left in shared memory, have been read: the
                    // next P.V need not wait for the rest (288 -> 275 us and 638 -> 590 us side by side).
                    if (c0 == D - 32) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&o_free);
                    }
                    if (plain) {
                        if (!first) {
#pragma unroll
                            for (int d = 0; d < 32; d += 2)
                                f2_unpack(f2_add(f2_pack(x[d], x[d + 1]), f2_pack(y[d], y[d + 1])), x[d], x[d + 1]);
                        }
                    } else {
#pragma unroll
                        for (int d = 0; d < 32; d += 2) {
                            uint64_t v = f2_mul(f2_pack(x[d], x[d + 1]), fy);
                            if (!first) v = f2_fma(f2_pack(y[d], y[d + 1]), fx, v);
                            f2_unpack(f2_mul(v, fin2), x[d], x[d + 1]);
                        }
                    }
                    if (!last) {
                        tmem_st32(at + (C::kColAcc - C::kColO) + c0, x);
                    } else if (i < rows) {
#pragma unroll
                        for (int d = 0; d < 32; d += 4)
                            *reinterpret_cast<float4*>(to + tile_order((c0 + d) / 4)) = make_float4(x[d], x[d + 1], x[d + 2], x[d + 3]);
                    }
                }
                tmem_wait_st();
                if (last && odd) odd = join_odd_values(to, g.odd + ((int64_t)blockIdx.x * kM + i) * D, D);
            } else {
                __syncwarp();
                if (lane == 0) mbar_arrive(&o_free);
            }
            if (last) to = next_to;
            return group.y + 1;
        };
        auto next_piece = [&]() -> bool {  // the next one that has tiles
            bool more;
            do more = warp_next(g, prefix, s);
            while (more && s.u1 <= s.u0);
            return more;
        };
        bool more = next_piece();
        if (more) load_queries();
        to = next_to;
        for (int k = 0; ok && more;) {
            const int end = n + s.u1 - s.u0;
            bool loaded = false;
            // The K slot of the piece's last tile is freed once by every kStep-th tile, and a
            // wait tells two frees of a slot apart only one after the other: `due` is the
            // first of them that is not known to have come.  (P.V of tile n - 1, folded,
            // means that S(n) is done.)
            constexpr int kStep = ST / 2;
            int due = (end - 1) % kStep;
            auto due_done = [&]() { return __all_sync(FULL, mbar_try_wait(&freed[(2 * due) % ST], (uint32_t)(((2 * due) / ST) & 1))); };
            while (n < end) {
                // The next piece's queries go in once the last scores with this one's are done:
                // before the fold that ends the piece, since its P.V comes after the
                // next piece's first scores; but those last scores may wait for a fold
                // that comes first.
                if (end - n <= kGroup && !loaded) {
                    if (n > 0 && due <= n) due += (n - due + kStep) / kStep * kStep;
                    uint64_t t0 = 0;
                    for (int i = 1; due < end; ++i) {
                        if (due_done())
                            due += kStep;
                        else if (__all_sync(FULL, mbar_try_wait(&o_full, (uint32_t)(k & 1))))
                            break;
                        if ((i & 1023) == 0) {  // bounded as wait_for is; the fold's own wait reports it
                            const uint64_t now = __shfl_sync(FULL, global_ns(), 0);
                            if (t0 == 0) t0 = now;
                            if (now - t0 > kWaitLimitNs) break;
                        }
                    }
                    if (due >= end) {
                        loaded = true;
                        more = next_piece();
                        tc_fence_after();
                        if (more) load_queries();
                    }
                }
                n = fold(k++);
                if (n == 0) {
                    ok = false;
                    break;
                }
            }
            if (ok && !loaded) {  // the last fold came first: all of the piece's scores are done
                more = next_piece();
                if (more) load_queries();
                to = next_to;
            }
        }
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
// successors went on with: m* = max m_i, out = sum w_i o_i / sum w_i, w_i = 2^(m_i - m*) l_i,
// o_i the pieces' own outputs, so that nothing on the way is larger than they are.
// A warp per virtual row.  Its launch overlaps the pieces' kernel; it reads at most
// 20 MB of partials out of L2 and is a few microseconds of any call.
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
    auto load = [&](int k) -> float2 {  // m and l of piece k
        return k < count ? make_float2(__ldcg(g.part_m + slot_row(k)), __ldcg(g.part_l + slot_row(k)))
                         : make_float2(-INFINITY, 0.f);
    };
    const float2 own = load(lane);  // more than 32 pieces: the others are loaded at every use
    float m = own.x;
    for (int k = lane + 32; k < count; k += 32) m = fmaxf(m, __ldcg(g.part_m + slot_row(k)));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, off));
    // A piece's weight; -0 where it saw nothing and left no output (l tells that, not m: NaN
    // scores leave m at -inf).  One that comes to +0 counts: 0 x inf is NaN, as in the other rows.
    auto weight = [&](float2 p) -> float { return p.y != 0.f ? fast_exp2(p.x - m) * p.y : -0.f; };
    float den = weight(own);
    for (int k = lane + 32; k < count; k += 32) den += weight(load(k));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) den += __shfl_xor_sync(FULL, den, off);
    const float inv = den != 0.f ? 1.f / den : 0.f;
    constexpr int kPer = D / 32;
    float acc[kPer];
#pragma unroll
    for (int c = 0; c < kPer; ++c) acc[c] = 0.f;
    for (int k0 = 0; k0 < count; k0 += 32) {
        const float wgt = weight(k0 == 0 ? own : load(k0 + lane)) * inv;
        const int here = min(count - k0, 32);
        for (int k = 0; k < here; ++k) {
            const float f = __shfl_sync(FULL, wgt, k);
            if (__float_as_uint(f) == 0x80000000u) continue;
            const float* src = g.part_o + slot_row(k0 + k) * D;
#pragma unroll
            for (int c = 0; c < kPer; ++c) acc[c] = fmaf(f, __ldcg(src + lane + 32 * c), acc[c]);
        }
    }
    float* out = a.out + (((int64_t)r.row0 + v / a.G) * a.H + (int64_t)hk * a.G + v % a.G) * D;
#pragma unroll
    for (int c = 0; c < kPer; ++c) out[lane + 32 * c] = acc[c];
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

// Boxes of a tile's layout out of row-major [rows, cols] f32, 128-byte swizzle.  A pool
// (rows in whole groups): elements, rows of a group, blocks, groups; a box has the
// `groups` of a page.  Drafted rows (groups = 0), which start anywhere: elements, rows,
// blocks; a box is one group.
bool encode_boxes(CUtensorMap* map, const float* p, int64_t rows, int64_t cols, int blocks, int groups) {
    return cached_tensor_map(map, p, rows, cols, 32 * blocks, groups, 4, [&](CUtensorMap* m) {
        auto fn = pg_encoder();
        if (!fn) return false;
        const cuuint64_t row = (cuuint64_t)cols * sizeof(float), nblk = (cuuint64_t)cols / 32;
        const cuuint32_t ones[4] = {1, 1, 1, 1};
        if (groups == 0) {
            const cuuint64_t dims[3] = {32, (cuuint64_t)rows, nblk}, strides[2] = {row, 128};
            const cuuint32_t box[3] = {32, 8, (cuuint32_t)blocks};
            return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<float*>(p), dims, strides, box, ones,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
        }
        const cuuint64_t dims[4] = {32, 8, nblk, (cuuint64_t)rows / 8}, strides[3] = {row, 128, 8 * row};
        const cuuint32_t box[4] = {32, 8, (cuuint32_t)blocks, (cuuint32_t)groups};
        return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, const_cast<float*>(p), dims, strides, box, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    });
}

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

struct PgScratch {
    size_t m, l, o, odd, odd_rows, head, total;
};
PgScratch scratch_of(int ctas, int D) {
    PgScratch s;
    const size_t rows = (size_t)2 * ctas * kM;
    s.m = kWorkspaceHeader;
    s.l = s.m + up256(rows * 4);
    s.o = s.l + up256(rows * 4);
    s.odd = s.o + up256(rows * D * 4);
    s.odd_rows = s.odd + up256(rows / 2 * D * 4);
    s.head = s.odd_rows + up256(rows / 2 * kRing * 8);
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
    g.odd = reinterpret_cast<float*>(ws + sc.odd);
    g.odd_rows = reinterpret_cast<uint64_t*>(ws + sc.odd_rows);
    g.head = reinterpret_cast<int4*>(ws + sc.head);
    const int64_t cols = (int64_t)a.Hk * D, pool = a.pages * a.page_size;
    CUtensorMap tk, tv, tkn, tvn;
    constexpr int nb = Cfg<D>::kBlocks;
    if (!encode_boxes(&tk, a.k_pool, pool, cols, nb, g.sub / 8) || !encode_boxes(&tv, a.v_pool, pool, cols, nb, g.sub / 8))
        return cudaErrorInvalidValue;
    tkn = tk;
    tvn = tv;
    if (a.tree && (!encode_boxes(&tkn, a.k_new, a.rows, cols, nb, 0) || !encode_boxes(&tvn, a.v_new, a.rows, cols, nb, 0)))
        return cudaErrorInvalidValue;
    auto kern = a.softcap_on ? paged_tc_kernel<D, true> : paged_tc_kernel<D, false>;
    cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kern), (int)Cfg<D>::kSmem);
    if (e != cudaSuccess) return e;
    kern<<<ctas, kThreads, Cfg<D>::kSmem, stream>>>(tk, tv, tkn, tvn, g);
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
