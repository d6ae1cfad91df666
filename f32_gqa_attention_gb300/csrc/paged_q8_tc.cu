// paged_q8_tc.cu -- attention of many query rows per request over an 8-bit paged cache on
// the tcgen05 tensor cores, headDim 64 or 128: trees of drafted tokens, chunks of prompts.
//
// Mathematics as in paged_q8_mma.cu, for row blocks of 128 virtual rows (t G + g) and tiles of
// 128 keys.  Codes are exact in f16, so S = Q K^T and O = P V are two f16 products each: hi and
// lo of the queries and of the weights, lo first.  Every tile stands alone: its weights are
// 2^(x2 - m_t), m_t the row's largest score in the tile, times the value's scale over 2^E, E
// the largest scale's exponent; its output O_t and sum l_t come with m_t and E, and the
// fold joins them in f32 by the log-sum-exp rule,
//   acc = acc 2^(M - M') + O_t 2^(m_t + E - M'),  M' = max(M, m_t).
// So no tile waits for another one's maximum, and no sum runs long inside the tensor cores,
// which round towards zero at every step.
// A weight has 2^14 as a factor: kept to 2^-39 of the largest scale times 1.  Where a tile's
// scales differ by more than 2^6 a small one may be what counts, so each row of such a tile
// takes the exponent of its own largest product instead (rare).
//
// Work.  One persistent CTA per SM; the CTAs divide the tiles of all (request, KV head, row
// block) units evenly, each counted with its request's whole range (paged_q8_list.cuh).  A unit cut
// by a CTA's end leaves partials (m, l, o / l) that q8_tc_merge_kernel joins in a fixed order.
//
// Warps, with their share of the 480 registers a lane that six warpgroups launch with:
//   0, 2    page ids, TMA loads of K and of V codes (a box per page) and copies of scales
//   1       MMAs; one elected lane issues
//   3       the range of a tile's value scales                                      (56)
//   4 - 7   queries to TMEM, and the fold; a thread is a row, acc in registers     (184)
//   8 - 15  softmax, a warpgroup for either half of a tile; a thread is a row    (2 x 72)
//   16 - 23 codes to f16 tiles, four warps for K, four for V                     (2 x 48)
// TMEM: Q hi, lo (D columns), two S / P buffers (256), O (D).
// Every wait is bounded; one that gives up sets a bit of the device flag.
//
// What bounds it.  8 trees of 64 rows beside 16384 to 32704 cached ones, 32 heads of 128 over 8 (large
// trees below), take 411 us with the drafted rows' part and the join; the two f16 products of 2.17e11
// FLOP would take 220 at the measured rate.  The scores and outputs of a tile take 1024 cycles of MMAs, a
// tile 3900 to 4200: the softmax warps are at it all of that time (1100 to the maximum, 2600 from
// there to the weights), and the roles together issue most of a tile's slots once packed f32
// instructions count twice.  More instructions in the softmax show (always masked: 476 us where 446
// was), and so does more code: with the next 16 scores loaded ahead in a loop twice as long, 463; the places of
// the rare paths alone move it by some per cent (433 with the far scales' path left out).  A
// change of piece costs a CTA some 16 000 cycles more: queries, the output's rows, an empty pipeline.
#include <cstring>
#include <mutex>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "attn_common.cuh"
#include "launch_cache.h"
#include "paged_q8_list.cuh"
#include "paged_q8_mma.cuh"
#include "pdl.cuh"
#include "softcap.cuh"
#include "tcgen05_ops.cuh"
#include "tma_sync.cuh"

namespace vtmu {

__device__ unsigned int g_q8_tc_device_error;

namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int kKT = 128, kHalf = 64;  // keys of a tile, and of a softmax warp's half
constexpr int kM = 128, kThreads = 768;
constexpr int kStages = 2;      // tiles of codes
constexpr int kSlots = 2;       // tiles of f16
constexpr int kScores = 2;      // S / P buffers
constexpr int kConverters = 4;  // warps that convert K; as many V
constexpr int kRing = 8;   // scales of K: tile n is loaded once S(n - 4) is done, and so O(n - 6) issued
constexpr int kRingV = 4;  // of V: once O(n - 4) is done
constexpr int kStats = 4;  // a tile's maximum and sum: S(n) is issued once O(n - 3) is folded
constexpr int kTiles = 16;  // what it is: the fold of a tile that far back may not have begun
constexpr int kShift = 14;  // of weights in f16
constexpr int kFar = 6;     // log2 by which a tile's scales may differ on the short way
// Scores of the MMA are sums of headDim products of at most 2^14 and 448, below 2^30: times a key's scale
// below this one they stay in f32.
constexpr float kFarKey = 0x1p98f;
// A tile's output, below 2^31, times its factor and added to those of up to 2^24 tiles stays in f32 where the
// factor is below this one.  Rows that meet a larger one keep their sums times 2^-32 from there on: up to 2^31
// weights of at most 1 times any value fit, and what that drops lies below 2^-117.
constexpr float kHugeFactor = 0x1p72f;
// Flags of a tile; slot + 1 in two bits from kSlotShift on.  K's converters add kFarKeys where a key's
// scale is kFarKey or more.
enum : int { kFirst = 1, kLast = 2, kStop = 4, kSlotShift = 3, kFarKeys = 32 };
enum : unsigned int {
    kErrQ8Load = 1u << 3,  // the paged kernels' bits: a tile that did not come,
    kErrQ8Free = 1u << 4,  // a buffer that was not given back,
    kErrQ8Mma = 1u << 5,   // a wait around the MMAs
};

struct TcArgs {
    PagedDesc a;
    Q8Pools p;
    int32_t page_shift;
    int32_t sub_shift;  // log2 of the rows of a TMA box: the largest power of two that divides a page, at most 64
    float* part_m;  // [2 CTAs][128]: slot 0 goes on with a unit, slot 1 starts one
    float* part_l;
    float* part_o;  // [2 CTAs][128][D], divided by l
    const float2* draft;
    int4* head;     // [2 CTAs]: the unit a CTA starts: last CTA, first virtual row, rows x group, first packed row; KV head
};

template <int D>
struct Cfg {
    static constexpr uint32_t kCodes = kKT * D, kTile = 2 * kCodes;  // bytes of a tile, as codes and as f16
    static constexpr size_t kSmem = 1024 + 2 * (kSlots * kTile + kStages * kCodes) + (kPagedMaxRequests + 1) * 8;
    static constexpr uint32_t kColQhi = 0, kColQlo = D / 2, kColS = D, kColO = D + kScores * kKT;
    static_assert(kColO + D <= 512, "TMEM budget");
    static_assert(kSmem + 24 * 1024 <= 232448, "shared memory budget");
};

struct Tile {
    int b, rb, key, flags, hk, piece, pad[2];
};

// A CTA's place in the list, for the producers.
struct Walk {
    long long pos, end, total, ctas;
    int b, rb, hk, u, u1, len, lo_tile, n_sink, slot, piece;
    bool first;
    int4 starts;  // the cut unit that this CTA starts (x < 0: none)
    int starts_head;

    __device__ void start(const PagedDesc& a, const long long* prefix) {
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
        piece = -1;
        starts = make_int4(-1, 0, 0, 0);
        starts_head = 0;
    }
    template <class Empty>
    __device__ bool next(const PagedDesc& a, const long long* prefix, Tile& t, Empty empty) {
        while (u >= u1) {
            if (pos >= end) return false;
            while (prefix[b + 1] <= pos) ++b;
            const Q8Req r = q8_load_req(a, b);
            const Q8Units w = q8_units(a, r, kKT);
            const long long rel = pos - prefix[b], unit = rel / w.nt;
            const int blocks = (r.T * a.G + kM - 1) / kM;
            hk = (int)(unit / blocks);
            rb = (int)(unit - (long long)hk * blocks);
            u = (int)(rel - unit * w.nt);
            u1 = (int)min((long long)w.nt, u + (end - pos));
            const long long from = pos - u;
            pos += u1 - u;
            slot = u > 0 ? 0 : u1 < w.nt ? 1 : -1;
            if (slot == 1) {
                starts = make_int4((int)(((from + w.nt) * ctas - 1) / total), rb * kM, r.T * a.G, r.row0);
                starts_head = hk;
            }
            if (!a.tree) u1 = min(u1, q8_seen_tiles(r, w, (min((rb + 1) * kM, r.T * a.G) - 1) / a.G, kKT));
            len = r.len;
            lo_tile = w.lo_tile;
            n_sink = w.n_sink;
            first = true;
            if (u >= u1) empty(slot);
            else ++piece;
        }
        t.b = b;
        t.rb = rb;
        t.hk = hk;
        t.piece = piece;
        t.key = (u < n_sink ? u : lo_tile + u - n_sink) * kKT;
        t.flags = (first ? kFirst : 0) | (u + 1 == u1 ? kLast : 0) | (slot + 1) << kSlotShift;
        first = false;
        ++u;
        return true;
    }
};

// ---- f16 MMAs (as the f32 cache's kernel) ---------------------------------------------------
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool mn) {
    return (1u << 4) | (mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// A tile's blocks of 64 channels, [128 rows][128 bytes] with the 128-byte swizzle, kBlock bytes apart.
// K-major: a row's channels along K.  MN-major: the rows are K, the next 64 channels a block on.
constexpr uint32_t kBlock = kKT * 128;
__device__ __forceinline__ uint64_t smem_desc(const void* tile, uint32_t next) {
    const uint64_t addr = smem_u32(tile);
    uint64_t d = (addr >> 4) & 0x3FFFull;
    d |= (uint64_t)(next >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}
// The descriptor in its words: the upper one is the same for every tile.
template <bool ACC>
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi, uint32_t idesc) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 b;\n mov.b64 b, {%2, %3};\n setp.ne.b32 p, %5, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n}\n" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(idesc), "n"(ACC ? 1 : 0)
        : "memory");
}
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
    return r != 0;
}
// Whether the phase is over, without a wait.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return done != 0;
}
// mbar_wait, bounded in the same way, that looks at the clock late and seldom: reading the
// global timer takes as long as a whole hand-over.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, int phase, unsigned int error) {
    const uint32_t parity = (uint32_t)(phase & 1);
    uint64_t t0 = 0;
    bool ok = mbar_try_wait(bar, parity);
#pragma unroll 1
    for (int i = 1; !ok; ++i) {
        ok = mbar_try_wait(bar, parity);
        if ((i & 1023) == 0 && !ok) {
            const uint64_t now = global_ns();
            if (t0 == 0) t0 = now;
            if (now - t0 > kWaitLimitNs) break;
        }
    }
    if (__all_sync(FULL, ok)) return true;
    raise_device_error(&g_q8_tc_device_error, error);
    return false;
}

// Three at once: a look at each takes as long as one.
__device__ __forceinline__ bool warp_wait3(uint64_t* a, int pa, uint64_t* b, int pb, uint64_t* c, int pc, unsigned int error) {
    const uint32_t xa = smem_u32(a), xb = smem_u32(b), xc = smem_u32(c);
    const uint32_t ya = (uint32_t)(pa & 1), yb = (uint32_t)(pb & 1), yc = (uint32_t)(pc & 1);
    uint64_t t0 = 0;
    uint32_t done = 0;
#pragma unroll 1
    for (int i = 1;; ++i) {
        asm volatile(
            "{\n .reg .pred p, q, r;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
            " mbarrier.test_wait.parity.shared::cta.b64 q, [%3], %4;\n mbarrier.test_wait.parity.shared::cta.b64 r, [%5], %6;\n"
            " and.pred p, p, q;\n and.pred p, p, r;\n selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(done)
            : "r"(xa), "r"(ya), "r"(xb), "r"(yb), "r"(xc), "r"(yc)
            : "memory");
        if (__all_sync(FULL, done != 0)) return true;
        if ((i & 1023) == 0) {
            const uint64_t now = global_ns();
            if (t0 == 0) t0 = now;
            if (__any_sync(FULL, now - t0 > kWaitLimitNs)) break;
        }
    }
    raise_device_error(&g_q8_tc_device_error, error);
    return false;
}

// No copy may be in flight when the CTA exits, whether the producer gave up or those that wait for its tiles
// did: of n tiles asked for the last one of each stage has to be there (the one before it was when that
// one was asked for).
__device__ __noinline__ void drain(uint64_t* staged, int n) {
    cp_async_wait_all();
#pragma unroll 1
    for (int i = max(n - kStages, 0); i < n; ++i)
        if (!warp_wait(staged + i % kStages, i / kStages, kErrQ8Free)) break;
}

// Codes of a tile to f16: four warps, 32 rows each, a lane 16 codes at a time.  TMA leaves
// chunk c (16 bytes) of row r at c ^ (r % 8) (headDim 128; 64: where it was).  A quarter of the
// warp takes 64 bytes of two rows; rows r and r ^ 5 (64: neighbours) meet no bank twice, neither
// as codes nor in the f16 tile's swizzle.  A lane's places in 8 rows are its places in the next 8.
template <int D, int FORM>
__device__ __forceinline__ void convert(const unsigned char* codes, unsigned char* tile, int w, int lane) {
    const int sub = lane & 7, q = lane >> 3;
    const int row = 32 * w + (D == 128 ? q ^ (sub & 4 ? 5 : 0) : 2 * q + (sub >> 2));
    const int c = sub & 3, sw = row & 7, j = 2 * c;  // 16 codes; the other 64 channels' are 4 chunks on
    const unsigned char* from = codes + row * D;
    unsigned char* to = tile + row * 128;
#pragma unroll
    for (int i = 0; i < D / 64; ++i)
#pragma unroll
        for (int r = 0; r < 32; r += 8) {
            const uint4 x = *reinterpret_cast<const uint4*>(from + 16 * (D == 128 ? (c + 4 * i) ^ sw : c) + r * D);
            uint32_t h[8];
            q8_halves<FORM>(x.x, h[0], h[1]);
            q8_halves<FORM>(x.y, h[2], h[3]);
            q8_halves<FORM>(x.z, h[4], h[5]);
            q8_halves<FORM>(x.w, h[6], h[7]);
            *reinterpret_cast<uint4*>(to + 16 * (j ^ sw) + i * kBlock + r * 128) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(to + 16 * ((j + 1) ^ sw) + i * kBlock + r * 128) = make_uint4(h[4], h[5], h[6], h[7]);
        }
}
// Rows from `rows` on of a tile of value codes, a warp's 32: what a page holds behind a request's last
// row may be a NaN, which no weight of zero takes away.
template <int D>
__device__ __noinline__ void clear_rows(unsigned char* codes, int rows, int w, int lane) {
    for (int i = 32 * w * D + 16 * lane; i < 32 * (w + 1) * D; i += 512)
        if (i / D >= rows) *reinterpret_cast<uint4*>(codes + i) = make_uint4(0, 0, 0, 0);
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");  // before the next tile's copies
    __syncwarp();
}

// What a softmax thread needs of its row and its half of a tile.
struct RowTile {
    uint32_t at;       // TMEM of its scores
    const float* ks;   // the keys' scales
    uint64_t see;      // keys that it sees (not read when WHOLE)
    float rf, cap;     // a score of the MMA times ks rf is one in base-2 units (the argument of tanh with a cap)
};
// Scores beside keys of kFarKey and more (rare): times ks rf in one, which is in range where the score is,
// back to tensor memory; their keys then have scales of 1.
__device__ __noinline__ void far_scores(uint32_t at, const float* ks, float rf) {
#pragma unroll 1
    for (int c = 0; c < kHalf; c += 16) {
        float x[16];
        tmem_ld16(at + c, x);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] *= q8_score_unit(ks[c + k], rf);
        tmem_st16(at + c, x);
    }
    tmem_wait_st();
}
// 16 scores from key k0 on: in base-2 units with a cap, else still to be multiplied by rf.
template <bool CAP, bool WHOLE>
__device__ __forceinline__ void row_scores(const RowTile& r, int k0, float (&x)[16]) {
    tmem_ld16(r.at + k0, x);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 16; k += 4) {
        const float4 s = *reinterpret_cast<const float4*>(r.ks + k0 + k);
        f2_unpack(f2_mul(f2_pack(x[k], x[k + 1]), f2_pack(s.x, s.y)), x[k], x[k + 1]);
        f2_unpack(f2_mul(f2_pack(x[k + 2], x[k + 3]), f2_pack(s.z, s.w)), x[k + 2], x[k + 3]);
    }
    if constexpr (CAP) softcap_tile<16>(x, r.rf, r.cap);
    if constexpr (!WHOLE) {
        const uint32_t bits = (uint32_t)(r.see >> k0);
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] = (bits >> k) & 1u ? x[k] : -INFINITY;
    }
}
// 16 weights as f16 hi (8 columns) and lo (8).
__device__ __forceinline__ void store_weights(uint32_t at, const float* w) {
    float y[16];
#pragma unroll
    for (int k = 0; k < 16; k += 2) {
        uint32_t h, l;
        mma_split(w[k], w[k + 1], h, l);
        y[k / 2] = __uint_as_float(h);
        y[8 + k / 2] = __uint_as_float(l);
    }
    tmem_st16(at, y);
}
// The row's largest score of the half, in base-2 units; leaves the masked scores as row_scores makes them.
// Short loops on purpose: the roles' code has to stay in the instruction cache together (with
// these unrolled, in tiles of 64 keys, large trees took 695 us instead of 613).
template <bool CAP, bool WHOLE>
__device__ __forceinline__ float row_max(const RowTile& r) {
    float m = -INFINITY;
#pragma unroll 1
    for (int k0 = 0; k0 < kHalf; k0 += 16) {
        float x[16];
        row_scores<CAP, WHOLE>(r, k0, x);
        tmem_st16(r.at + k0, x);
#pragma unroll
        for (int k = 0; k < 16; k += 2) m = fmaxf(fmaxf(m, x[k]), x[k + 1]);
    }
    tmem_wait_st();
    return CAP ? m : m * r.rf;
}
// Weights 2^(x2 - mu) vn over its scores (vn: the values' scales times 2^(kShift - E)); returns the
// sum of the exponentials.
template <bool CAP, bool WHOLE>
__device__ __forceinline__ float row_weights(const RowTile& r, const float* vn, float mu) {
    const float mul = CAP ? 1.f : r.rf;
    const uint64_t mul2 = f2_pack(mul, mul), sub2 = f2_pack(-mu, -mu);
    uint64_t sum = 0;
#pragma unroll 1
    for (int k0 = 0; k0 < kHalf; k0 += 16) {
        float x[16];
        tmem_ld16(r.at + k0, x);
        tmem_wait_ld();
        const uint32_t bits = (uint32_t)(r.see >> k0);
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
            const float4 v = *reinterpret_cast<const float4*>(vn + k0 + k);
            const float vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                float e0, e1;
                f2_unpack(f2_fma(f2_pack(x[k + j], x[k + j + 1]), mul2, sub2), e0, e1);
                const uint64_t p = f2_pack(fast_exp2(e0), fast_exp2(e1));
                sum = f2_add(sum, p);
                f2_unpack(f2_mul(p, f2_pack(vv[j], vv[j + 1])), x[k + j], x[k + j + 1]);
                if constexpr (!WHOLE) {  // the scale of a key that is not seen may be anything
                    if (!((bits >> (k + j)) & 1u)) x[k + j] = 0.f;
                    if (!((bits >> (k + j + 1)) & 1u)) x[k + j + 1] = 0.f;
                }
            }
        }
        store_weights(r.at + k0, x);
    }
    float a, b;
    f2_unpack(sum, a, b);
    return a + b;
}
// The same with scales of very different size: relative to the row's largest product
// 2^(x2 - mu) 2^e, e the scales' exponents.  WEIGHTS = false: that product's exponent in the half,
// true: the weights times 2^(kShift - top), and the sum.
template <bool CAP, bool WEIGHTS>
__device__ __forceinline__ float far_softmax(const RowTile r, const float* vs, float mu, float top) {
    auto power = [](float v) -> float { return (float)((int)((__float_as_uint(v) >> 23) & 255u) - 127); };
    const float mul = CAP ? 1.f : r.rf;
    float sum = 0.f;
#pragma unroll 1
    for (int c = 0; c < kHalf; c += 16) {
        float x[16];
        tmem_ld16(r.at + c, x);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float v = vs[c + i], e = power(v), y = x[i] * mul - mu;
            if constexpr (!WEIGHTS) {
                top = fmaxf(top, y + e);
            } else {
                const float part = v * (e > 0.f ? exp2f(-e) : exp2f(-e - 1.f) * 2.f);  // the scale's mantissa; 0 stays 0
                sum += fast_exp2(y);
                x[i] = (r.see >> (c + i)) & 1u ? fast_exp2(y + (e - top)) * part * (float)(1 << kShift) : 0.f;
            }
        }
        if constexpr (WEIGHTS) store_weights(r.at + c, x);
    }
    return WEIGHTS ? sum : top;
}

// 16 lanes x 8 columns of tensor memory: lane l holds columns 2 (l % 4) and the next of rows l / 4
// (v[0], v[1]) and l / 4 + 8.
__device__ __forceinline__ void tmem_st_16x8(uint32_t at, const uint32_t (&v)[4]) {
    asm volatile("tcgen05.st.sync.aligned.16x256b.x1.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]));
}
// The queries of the piece that tile t begins, a warp's 32 virtual rows of its block: to tensor memory
// as hi and lo, times qk_mul and a power of two that brings the row's largest element to
// [2^13, 2^14); `back` gets what that takes back.  Four lanes share a row, so that a load touches 8
// lines: with a row a lane, 32 lines, large trees took 412 us where this took 405, chunks 210 and 203.
template <int D>
__device__ __forceinline__ void row_queries(const PagedDesc& a, const Tile& t, int w, int lane, uint32_t at_hi, uint32_t at_lo,
                                            float* back) {
    const Q8Req rq = q8_load_req(a, t.b);
    const int quad = lane & 3;
#pragma unroll 1
    for (int half = 0; half < 32; half += 16) {
        const float* q[2];
        float sc[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = 32 * w + half + (lane >> 2) + 8 * h, v = t.rb * kM + i, row = v / a.G;
            q[h] = v < rq.T * a.G
                       ? a.q + (((int64_t)rq.row0 + row) * a.H + (int64_t)t.hk * a.G + (v - row * a.G)) * D + 4 * quad
                       : nullptr;
        }
        auto load4 = [&](int h, int d) -> float4 {
            if (!q[h]) return make_float4(0.f, 0.f, 0.f, 0.f);
            const float4 y = __ldg(reinterpret_cast<const float4*>(q[h] + d));
            return make_float4(y.x * a.qk_mul, y.y * a.qk_mul, y.z * a.qk_mul, y.w * a.qk_mul);
        };
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float top = 0.f;
#pragma unroll 8
            for (int d = 0; d < D; d += 16) top = q8_abs_top(top, load4(h, d));
            top = q8_nan_max(top, __shfl_xor_sync(FULL, top, 1));
            top = q8_nan_max(top, __shfl_xor_sync(FULL, top, 2));
            sc[h] = mma_row_scale(top, 13);
            if (quad == 0) back[32 * w + half + (lane >> 2) + 8 * h] = 1.f / sc[h];
        }
#pragma unroll 2
        for (int d = 0; d < D; d += 16) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float4 y = load4(h, d);
                mma_split(y.x * sc[h], y.y * sc[h], hi[2 * h], lo[2 * h]);
                mma_split(y.z * sc[h], y.w * sc[h], hi[2 * h + 1], lo[2 * h + 1]);
            }
            tmem_st_16x8(at_hi + ((uint32_t)half << 16) + d / 2, hi);
            tmem_st_16x8(at_lo + ((uint32_t)half << 16) + d / 2, lo);
        }
    }
    tmem_wait_st();
}

template <int D, int FORM, bool CAP>
__global__ void __launch_bounds__(kThreads, 1) 
    q8_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                 const __grid_constant__ TcArgs g) {
    using C = Cfg<D>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* tiles = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    unsigned char* ktiles = tiles;
    unsigned char* vtiles = tiles + kSlots * C::kTile;
    unsigned char* codes = vtiles + kSlots * C::kTile;  // stages of K, stages of V
    long long* prefix = reinterpret_cast<long long*>(codes + (size_t)kStages * 2 * C::kCodes);
    __shared__ __align__(8) uint64_t staged[2][kStages], unstaged[2][kStages], ranged[kRingV], k_ready[kSlots], k_free[kSlots],
        v_ready[kSlots], v_free[kSlots], q_full, q_free, s_full[kScores], p_full[kScores], met[4], o_full, o_free;
    __shared__ uint32_t tmem_base_s;
    __shared__ long long scan_s[kThreads / 32];
    __shared__ __align__(16) float k_scale[kRing][kKT], v_scale[kRingV][kKT], v_norm[kRingV][kKT];
    __shared__ float v_back[kRingV];             // 2^(E - kShift); 0: the scales differ too much
    __shared__ __align__(16) Tile tile_s[kTiles];
    __shared__ float q_back[4][kM];              // by piece: what the queries' power of two takes back
    __shared__ float stat[kStats][4][kM];        // by tile: m, l of either half, factor of its output
    __shared__ float meet[2][2][kM];             // what the halves of a row tell one another
    __shared__ __align__(16) float ones[kHalf];  // scales of keys whose scores have theirs
    __shared__ int piece_end[4];                 // by piece: the tile after it
    __shared__ int v_rows[kRingV];               // of a tile that there are, as V's producer knows; -1: the end

    const PagedDesc& a = g.a;
    const int warp = __shfl_sync(FULL, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            for (int kv = 0; kv < 2; ++kv) {
                mbar_init(&staged[kv][i], 33);  // bytes, and every lane's scales
                mbar_init(&unstaged[kv][i], kConverters + kv);  // and the warp that takes the range of V's scales
            }
        }
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&k_ready[i], kConverters);
            mbar_init(&k_free[i], 1);
            mbar_init(&v_ready[i], kConverters);
            mbar_init(&v_free[i], 1);
        }
        for (int i = 0; i < kScores; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 8);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&met[i], 2);
        for (int i = 0; i < kRingV; ++i) mbar_init(&ranged[i], 1);
        mbar_init(&o_full, 1);
        mbar_init(&o_free, 4);
        mbar_init(&q_free, 2);  // the MMAs' commit, and an arrival that publishes piece_end
        mbar_init(&q_full, 4);
        fence_barrier_init();
    }
    if (threadIdx.x < kHalf) ones[threadIdx.x] = 1.f;
    if (warp == 1) tmem_alloc(&tmem_base_s, 512);
    // The requests' tiles and their running sum.
    long long carry = 0;
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        long long v = 0;
        if (b < a.B) {
            const Q8Req r = q8_load_req(a, b);
            v = ((long long)r.T * a.G + kM - 1) / kM * a.Hk * q8_units(a, r, kKT).nt;
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
    auto part_row = [&](int slot, int i) -> int64_t { return (int64_t)(2 * blockIdx.x + slot) * kM + i; };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 0 || warp == 2) {
            // ---- producers: K and V ---------------------------------------------------------
            const bool values = warp == 2;
            Walk walk;
            walk.start(a, prefix);
            auto empty = [&](int slot) {
                if (slot < 0 || values) return;
                for (int i = lane; i < kM; i += 32) {
                    g.part_m[part_row(slot, i)] = -INFINITY;
                    g.part_l[part_row(slot, i)] = 0.f;
                }
            };
            const float* scales = values ? g.p.v_scale : g.p.k_scale;
            // 32 boxes of a request are looked up at a time, a lane each: the first row of each in the
            // pool, -1 for rows of no page.
            int y_cur = -1, batch = -1, of_piece = -1, n = 0;
            for (bool stop = false; !stop; ++n) {
                Tile t;
                stop = !walk.next(a, prefix, t, empty);
                if (stop) t.flags = kStop;
                const int st = n % kStages;
                if (n >= kStages && !warp_wait(&unstaged[values][st], n / kStages - 1, kErrQ8Free)) break;
                if (lane == 0) {
                    if (values) {
                        v_rows[n % kRingV] = stop ? -1 : max(walk.len - t.key, 0);
                    } else {
                        tile_s[n % kTiles] = t;
                    }
                    mbar_arrive_expect_tx(&staged[values][st], stop ? 0u : C::kCodes);
                }
                __syncwarp();
                if (!stop) {
                    if (t.piece != of_piece) batch = -1;
                    of_piece = t.piece;
                    unsigned char* to = codes + (size_t)(st + (values ? kStages : 0)) * C::kCodes;
                    float* to_scale = values ? v_scale[n % kRingV] : k_scale[n % kRing];
                    const int boxes = kKT >> g.sub_shift, q0 = t.key >> g.sub_shift;
#pragma unroll 1
                    for (int c = 0; c < boxes; c += 32) {
                        if (((q0 + c) >> 5) != batch) {
                            batch = (q0 + c) >> 5;
                            const int row = ((batch << 5) + lane) << g.sub_shift;
                            y_cur = -1;
                            if (row < walk.len) {
                                const int col = g.page_shift >= 0 ? row >> g.page_shift : row / a.page_size;
                                const int page = __ldg(a.block_table + (int64_t)t.b * a.max_pages + col);
                                if ((unsigned)page < (unsigned)a.pages) y_cur = page * a.page_size + (row - col * a.page_size);
                            }
                        }
                        // Rows of no page are out of bounds: zeros.
                        const int y = __shfl_sync(FULL, y_cur, (q0 + lane) & 31);
                        if (lane < boxes)
                            tma_load_2d(to + ((c + lane) << g.sub_shift) * D, values ? &tm_v : &tm_k, t.hk * D,
                                        y < 0 ? (int)(a.pages * a.page_size) : y, &staged[values][st]);
                        const int keys = min(kKT, 32 << g.sub_shift);  // of these boxes
                        for (int k = (c << g.sub_shift) + lane; k < (c << g.sub_shift) + keys; k += 32) {
                            const int key = t.key + k;
                            const int first = __shfl_sync(FULL, y_cur, (key >> g.sub_shift) & 31);
                            const bool there = first >= 0 && key < walk.len;
                            const int64_t at = there ? (int64_t)(first + (key & ((1 << g.sub_shift) - 1))) * a.Hk + t.hk : 0;
                            cp_async4(to_scale + k, scales + at, there ? 4 : 0);
                        }
                    }
                }
                cp_async_arrive(&staged[values][st]);
            }
            drain(staged[values], n);
            if (!values && lane == 0) {
                g.head[2 * blockIdx.x] = walk.starts;
                g.head[2 * blockIdx.x + 1] = make_int4(walk.starts_head, 0, 0, 0);
            }
        } else if (warp == 3) {
            // ---- the range of a tile's value scales ----------------------------------------
            for (int n = 0;; ++n) {
                const int st = n % kStages, rg = n % kRingV;
                if (!warp_wait(&staged[1][st], n / kStages, kErrQ8Load)) break;
                const bool stop = v_rows[rg] < 0;
                const float* vs = v_scale[rg];
                if (stop) break;
                float v[4];
                uint32_t most = 0, least = ~0u;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[i] = vs[lane + 32 * i];
                    const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;
                    most = max(most, b);
                    least = min(least, b ? b : ~0u);
                }
                most = __reduce_max_sync(FULL, most);
                least = __reduce_min_sync(FULL, least);
                // E, where 2^(kShift - E) and its inverse are normal numbers (a tile whose scales are all below
                // 2^-110 keeps 23 bits of its largest weight).
                int e = (int)(most >> 23) - 127;
                const bool far = e > 110 || (most > least && most - least > (uint32_t)kFar << 23);
                e = e < -110 ? -110 : e > 110 ? 110 : e;
                const float up = __uint_as_float((uint32_t)(127 + kShift - e) << 23);
#pragma unroll
                for (int i = 0; i < 4; ++i) v_norm[rg][lane + 32 * i] = v[i] * up;
                if (lane == 0) v_back[rg] = far ? 0.f : __uint_as_float((uint32_t)(127 - kShift + e) << 23);
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&ranged[rg]);
                    mbar_arrive(&unstaged[1][st]);
                }
            }
        } else if (warp == 1) {
            // ---- MMAs ---------------------------------------------------------------------
            constexpr uint32_t id_s = idesc_f16(kM, kKT, false), id_o = idesc_f16(kM, D, true);
            const uint64_t k0 = smem_desc(ktiles, 16), v0 = smem_desc(vtiles, kBlock);
            const uint32_t k_lo = (uint32_t)k0, k_hi = (uint32_t)(k0 >> 32), v_lo = (uint32_t)v0, v_hi = (uint32_t)(v0 >> 32);
            // S goes first where its keys and queries are there; what it is, is looked up before the wait for
            // the weights of O.
            int sn = 0, vn = 0, flags = 0, piece = 0;
            bool end = false, k_ok = false, q_ok = false;
            for (;;) {
                const int sl = sn % kSlots;
                const bool must = sn == vn;
                if (!end && !k_ok) {
                    k_ok = __all_sync(FULL, mbar_test(&k_ready[sl], (uint32_t)((sn / kSlots) & 1)));
                    if (!k_ok && must) {
                        k_ok = warp_wait(&k_ready[sl], sn / kSlots, kErrQ8Mma);
                        if (!k_ok) break;
                    }
                    if (k_ok) {
                        flags = tile_s[sn % kTiles].flags;
                        piece = tile_s[sn % kTiles].piece;
                        end = flags & kStop;
                        q_ok = !(flags & kFirst);
                    }
                }
                if (!end && k_ok && !q_ok) {
                    q_ok = __all_sync(FULL, mbar_test(&q_full, (uint32_t)(piece & 1)));
                    if (!q_ok && must) {
                        q_ok = warp_wait(&q_full, piece, kErrQ8Mma);
                        if (!q_ok) break;
                    }
                }
                if (!end && k_ok && q_ok && sn - vn < kScores) {
                    tc_fence_after();
                    const uint32_t d = tmem + C::kColS + (sn % kScores) * kKT;
                    const uint32_t k = k_lo + sl * (C::kTile >> 4);
                    if (elect_one()) {
                        // Unrolled, with little but the MMA itself to an issue: the warp has a sixth of its
                        // scheduler.  950 cycles; with loops and 64-bit sums half of these took 1500.
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            const uint32_t at = k + (i >> 2) * (kBlock >> 4) + 2 * (i & 3);
                            if (i == 0) mma_f16_ts<false>(d, tmem + C::kColQlo, at, k_hi, id_s);
                            else mma_f16_ts<true>(d, tmem + C::kColQlo + 8 * i, at, k_hi, id_s);
                        }
#pragma unroll
                        for (int i = 0; i < D / 16; ++i)
                            mma_f16_ts<true>(d, tmem + C::kColQhi + 8 * i, k + (i >> 2) * (kBlock >> 4) + 2 * (i & 3), k_hi, id_s);
                        mma_commit(&k_free[sl]);
                        mma_commit(&s_full[sn % kScores]);
                        if (flags & kLast) {
                            piece_end[piece & 3] = sn + 1;
                            mma_commit(&q_free);
                            mbar_arrive(&q_free);  // publishes piece_end
                        }
                    }
                    __syncwarp();
                    ++sn;
                    k_ok = false;
                    continue;
                }
                if (vn < sn) {  // O(vn) = P(vn) V(vn)
                    const int bf = vn % kScores, st = vn % kSlots;
                    // o_free's phases begin with a tile's O: the one before the first is over.
                    if (!warp_wait3(&p_full[bf], vn / kScores, &v_ready[st], vn / kSlots, &o_free, vn - 1, kErrQ8Mma)) break;
                    tc_fence_after();
                    const uint32_t d = tmem + C::kColO, p = tmem + C::kColS + bf * kKT;
                    const uint32_t v = v_lo + st * (C::kTile >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < kKT / 16; ++k) {
                            if (k == 0) mma_f16_ts<false>(d, p + 8, v, v_hi, id_o);
                            else mma_f16_ts<true>(d, p + 16 * k + 8, v + (2048 >> 4) * k, v_hi, id_o);
                        }
#pragma unroll
                        for (int k = 0; k < kKT / 16; ++k) mma_f16_ts<true>(d, p + 16 * k, v + (2048 >> 4) * k, v_hi, id_o);
                        mma_commit(&v_free[st]);
                        mma_commit(&o_full);
                    }
                    __syncwarp();
                    ++vn;
                    continue;
                }
                // The end: the others learn of it in turn, once they have taken their last tiles.
                if (vn > 0 && !warp_wait(&o_free, vn - 1, kErrQ8Mma)) break;
                if (lane == 0) {
                    mbar_arrive(&s_full[sn % kScores]);
                    mbar_arrive(&o_full);
                }
                break;
            }
        }
    } else if (warp < 8) {
        // ---- queries and fold: thread = virtual row --------------------------------------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        const int w = warp & 3, i = 32 * w + lane;
        const uint32_t lanes = (uint32_t)(32 * w) << 16;
        // The queries of the piece that tile j begins.  False at the list's end.
        auto load_queries = [&](int j) -> bool {
            const Tile t = tile_s[j % kTiles];
            if (t.flags & kStop) return false;
            row_queries<D>(a, t, w, lane, tmem + lanes + C::kColQhi, tmem + lanes + C::kColQlo, q_back[t.piece & 3]);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full);
            return true;
        };
        bool more = warp_wait(&k_ready[0], 0, kErrQ8Mma) && load_queries(0);
        int loaded = 0;     // pieces after the first whose queries are in; -1: there are no more
        int folded = 0;     // pieces that are done: tile n is one of the next piece's
        float acc[D], M = -INFINITY, L = 0.f, down = 1.f;  // down: of acc
#pragma unroll
        for (int d = 0; d < D; ++d) acc[d] = 0.f;
        for (int n = 0; more; ++n) {
            // The next piece's queries go in once this one's scores are done and its first tile is
            // known: the scores run ahead of O, so a look a tile mostly finds that in time.
            if (loaded >= 0) {
                const bool must = loaded < folded;
                bool free = __all_sync(FULL, mbar_test(&q_free, (uint32_t)(loaded & 1)));
                if (must && !free && !(free = warp_wait(&q_free, loaded, kErrQ8Mma))) break;
                if (free) {
                    const int e = piece_end[loaded & 3];
                    bool known = __all_sync(FULL, mbar_test(&k_ready[e % kSlots], (uint32_t)((e / kSlots) & 1)));
                    if (must && !known && !(known = warp_wait(&k_ready[e % kSlots], e / kSlots, kErrQ8Mma))) break;
                    if (known) {
                        tc_fence_after();
                        loaded = load_queries(e) ? loaded + 1 : -1;
                    }
                }
            }
            if (!warp_wait(&o_full, n, kErrQ8Mma)) break;
            tc_fence_after();
            const Tile t = tile_s[n % kTiles];
            if (t.flags & kStop) break;
            const float* st = &stat[n % kStats][0][i];
            const float mt = st[0], lt = st[kM] + st[2 * kM];
            const float Mn = fmaxf(M, mt), mu = Mn == -INFINITY ? 0.f : Mn;
            const float alpha = fast_exp2(M - mu), beta = fast_exp2(mt - mu);
            M = Mn;
            L = fmaf(L, alpha, lt * beta);
            const float factor = beta * st[3 * kM];
            if (__any_sync(FULL, alpha != 1.f || factor >= kHugeFactor)) {  // a maximum moved, or a factor is huge
                float by = alpha;
                if (factor >= kHugeFactor && down == 1.f) {
                    by *= 0x1p-32f;
                    down = 0x1p-32f;
                }
                const uint64_t al = f2_pack(by, by);
#pragma unroll
                for (int d = 0; d < D; d += 2) f2_unpack(f2_mul(f2_pack(acc[d], acc[d + 1]), al), acc[d], acc[d + 1]);
            }
            const float bo = factor * down;
            const uint64_t be = f2_pack(bo, bo);
            const uint32_t at = tmem + lanes + C::kColO;
#pragma unroll
            for (int c0 = 0; c0 < D; c0 += 16) {
                float x[16];
                tmem_ld16(at + c0, x);
                tmem_wait_ld();
                if (c0 == D - 16) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&o_free);
                }
#pragma unroll
                for (int d = 0; d < 16; d += 2)
                    f2_unpack(f2_fma(f2_pack(x[d], x[d + 1]), be, f2_pack(acc[c0 + d], acc[c0 + d + 1])), acc[c0 + d],
                              acc[c0 + d + 1]);
            }
            if (t.flags & kLast) {
                const int slot = ((t.flags >> kSlotShift) & 3) - 1, v = t.rb * kM + i;
                const Q8Req rq = q8_load_req(a, t.b);
                float inv = L != 0.f ? 1.f / L / down : 0.f;
                if (a.tree) pdl_wait();  // the drafted rows' part
                if (v < rq.T * a.G) {
                    float* to;
                    Q8Share share{1.f, -0.f};
                    if (slot < 0) {
                        const int64_t row = ((int64_t)rq.row0 + v / a.G) * a.H + (int64_t)t.hk * a.G + v % a.G;
                        to = a.out + row * D;
                        if (a.tree) share = q8_share(M, L, __ldcg(g.draft + row));
                    } else {
                        to = g.part_o + part_row(slot, i) * D;
                        g.part_m[part_row(slot, i)] = M;
                        g.part_l[part_row(slot, i)] = L;
                    }
                    inv *= share.own;
#pragma unroll
                    for (int d = 0; d < D; d += 4) {
                        float4 y = make_float4(acc[d] * inv, acc[d + 1] * inv, acc[d + 2] * inv, acc[d + 3] * inv);
                        if (!q8_nothing(share.draft)) {
                            const float4 z = __ldcg(reinterpret_cast<const float4*>(to + d));
                            y = make_float4(fmaf(share.draft, z.x, y.x), fmaf(share.draft, z.y, y.y), fmaf(share.draft, z.z, y.z),
                                            fmaf(share.draft, z.w, y.w));
                        }
                        *reinterpret_cast<float4*>(to + d) = y;
                    }
                }
                __syncwarp();
                ++folded;
                M = -INFINITY;
                L = 0.f;
                down = 1.f;
#pragma unroll
                for (int d = 0; d < D; ++d) acc[d] = 0.f;
            }
        }
    } else if (warp < 16) {
        // ---- softmax: thread = virtual row, one half of every tile ------------------------------------
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        const int half = (warp - 8) >> 2, i = 32 * (warp & 3) + lane;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        int piece = -1, hi = 0, lo = 0, sinks = 0;
        bool alive = false;
        int meets = 0;
        // The larger of a row's two halves, by a slot each, two meetings in turn.
        auto larger = [&](float x, bool& ok) -> float {
            meet[meets & 1][half][i] = x;
            __syncwarp();
            if (lane == 0) mbar_arrive(&met[warp & 3]);
            ok = warp_wait(&met[warp & 3], meets, kErrQ8Mma);
            const float y = meet[meets & 1][half ^ 1][i];
            ++meets;
            return fmaxf(x, y);
        };
        for (int n = 0;; ++n) {
            if (!warp_wait(&s_full[n % kScores], n / kScores, kErrQ8Mma)) break;
            const Tile t = tile_s[n % kTiles];
            RowTile rt;
            rt.at = tmem + lanes + C::kColS + (n % kScores) * kKT + kHalf * half;
            rt.ks = k_scale[n % kRing] + kHalf * half;
            rt.rf = q_back[t.piece & 3][i];
            if (t.flags & (kStop | kFarKeys)) {
                if (t.flags & kStop) break;
                tc_fence_after();
                far_scores(rt.at, rt.ks, rt.rf);
                rt.ks = ones;
                rt.rf = 1.f;
            }
            if (t.piece != piece) {
                piece = t.piece;
                const Q8Req rq = q8_load_req(a, t.b);
                const int v = t.rb * kM + i, row = v / a.G;
                alive = v < rq.T * a.G;
                int p = a.tree ? rq.len : rq.len - rq.n + row;
                if (a.tree && a.window > 0 && alive) p = __ldg(a.positions + rq.row0 + row);
                // Keys of the cache that the row sees: [lo, hi], and those before `sinks`.
                hi = a.tree ? rq.len - 1 : min(p, rq.len - 1);
                lo = a.window > 0 ? (int)max((int64_t)p - a.window + 1, (int64_t)0) : 0;
                sinks = (int)min(a.sinks, (int64_t)rq.len);
            }
            tc_fence_after();
            const int key = t.key + kHalf * half;
            const bool all = !alive || (hi - key >= kHalf - 1 && lo <= key);
            const bool whole = __all_sync(FULL, all);
            rt.see = ~0ull;
            rt.cap = a.cap_log2;
            if (!all) {
                auto below = [](int c) -> uint64_t { return c <= 0 ? 0ull : c >= 64 ? ~0ull : (1ull << c) - 1; };
                rt.see = below(hi - key + 1) & (~below(lo - key) | below(sinks - key));
            }
            bool ok;
            const float m = larger(whole ? row_max<CAP, true>(rt) : row_max<CAP, false>(rt), ok);
            const float mu = m == -INFINITY ? 0.f : m;
            if (!ok || !warp_wait(&ranged[n % kRingV], n / kRingV, kErrQ8Load)) break;
            float factor = v_back[n % kRingV], l;
            if (factor == 0.f) {  // rare
                const float* vs = v_scale[n % kRingV] + kHalf * half;
                const float top = ceilf(fminf(larger(far_softmax<CAP, false>(rt, vs, mu, -300.f), ok), 126.f));
                if (!ok) break;
                l = far_softmax<CAP, true>(rt, vs, mu, top);
                factor = exp2f(top - (float)kShift);
            } else {
                const float* vn = v_norm[n % kRingV] + kHalf * half;
                l = whole ? row_weights<CAP, true>(rt, vn, mu) : row_weights<CAP, false>(rt, vn, mu);
            }
            stat[n % kStats][1 + half][i] = l;
            if (half == 0) {
                stat[n % kStats][0][i] = m;
                stat[n % kStats][3][i] = factor;
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[n % kScores]);
        }
    } else {
        // ---- codes to f16 ------------------------------------------------------------------
        asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        // Four warps for K, four for V, so that K does not wait for an earlier O with V (eight for
        // both, K first, in halves of a tile: 519 us).
        const int kv = warp >= 20, w = warp & 3;
        uint64_t *ready = kv ? v_ready : k_ready, *freed = kv ? v_free : k_free;
        for (int n = 0;; ++n) {
            const int st = n % kStages, sl = n % kSlots;
            if (!warp_wait(&staged[kv][st], n / kStages, kErrQ8Load)) break;
            const int rows = kv ? v_rows[n % kRingV] : tile_s[n % kTiles].flags & kStop ? -1 : kKT;
            if (n >= kSlots && !warp_wait(&freed[sl], n / kSlots - 1, kErrQ8Free)) break;
            if (rows < 0) {
                if (lane == 0) mbar_arrive(&ready[sl]);
                break;
            }
            unsigned char* from = codes + (size_t)(st + kv * kStages) * C::kCodes;
            unsigned char* to = (kv ? vtiles : ktiles) + sl * C::kTile;
            if (!kv) {
                const bool far = k_scale[n % kRing][32 * w + lane] >= kFarKey;
                if (__any_sync(FULL, far) && lane == 0) atomicOr(&tile_s[n % kTiles].flags, (int)kFarKeys);
            }
            if (FORM == kFormE4m3 && rows < kKT) clear_rows<D>(from, rows, w, lane);
            convert<D, FORM>(from, to, w, lane);
            asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");  // generic writes -> MMA
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&unstaged[kv][st]);
                mbar_arrive(&ready[sl]);
            }
        }
    }

    pdl_wait();  // this grid may not be done before the one that it overlaps
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the partials of the unit that CTA blockIdx.x starts, always in the same order: a warp per
// virtual row.
template <int D>
__global__ void __launch_bounds__(256) q8_tc_merge_kernel(const __grid_constant__ TcArgs g) {
    constexpr int kPer = D / 32;
    pdl_wait();
    const PagedDesc& a = g.a;
    const int4 h = __ldcg(&g.head[2 * blockIdx.x]);
    const int hk = __ldcg(&g.head[2 * blockIdx.x + 1].x);
    const int lane = threadIdx.x & 31, i = blockIdx.y * 8 + (threadIdx.x >> 5), v = h.y + i;
    if (h.x < 0 || v >= h.z) return;
    const int count = h.x - blockIdx.x + 1;
    auto row = [&](int k) -> int64_t { return (int64_t)(2 * (blockIdx.x + k) + (k == 0 ? 1 : 0)) * kM + i; };
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
            if (q8_nothing(f)) continue;
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

PFN_cuTensorMapEncodeTiled_v12000 q8_encoder() {
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
// Boxes of `sub` rows of one head out of row-major codes [rows, cols].
template <int D>
bool encode_rows(CUtensorMap* map, const uint8_t* p, int64_t rows, int64_t cols, int sub) {
    return cached_tensor_map(map, p, rows, cols, D, sub, 8, [&](CUtensorMap* m) {
        auto fn = q8_encoder();
        if (!fn) return false;
        const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)cols};
        const cuuint32_t box[2] = {(cuuint32_t)D, (cuuint32_t)sub}, ones[2] = {1, 1};
        return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(p), dims, strides, box, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    });
}

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

struct Scratch {
    size_t m, l, o, head, draft, total;
};
Scratch scratch_of(int D, int64_t draft_rows) {
    const size_t rows = (size_t)2 * kPagedMaxCtas * kM;
    Scratch s;
    s.m = kWorkspaceHeader;
    s.l = s.m + up256(rows * 4);
    s.o = s.l + up256(rows * 4);
    s.head = s.o + up256(rows * D * 4);
    s.draft = s.head + up256((size_t)2 * kPagedMaxCtas * sizeof(int4));
    s.total = s.draft + up256((size_t)draft_rows * sizeof(float2));
    return s;
}

template <int D, int FORM>
cudaError_t launch_form(const PagedDesc& a, const Q8Pools& p, int num_sms, void* workspace, cudaStream_t stream) {
    TcArgs g;
    std::memset(&g, 0, sizeof(g));
    g.a = a;
    g.p = p;
    g.page_shift = -1;
    for (int i = 0; i < 31; ++i)
        if (a.page_size == 1 << i) g.page_shift = i;
    const Scratch s = scratch_of(D, 0);
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    g.part_m = reinterpret_cast<float*>(ws + s.m);
    g.part_l = reinterpret_cast<float*>(ws + s.l);
    g.part_o = reinterpret_cast<float*>(ws + s.o);
    g.head = reinterpret_cast<int4*>(ws + s.head);
    float2* draft = reinterpret_cast<float2*>(ws + s.draft);
    g.draft = draft;
    while ((1 << g.sub_shift) < 64 && a.page_size % (2 << g.sub_shift) == 0) ++g.sub_shift;
    const int sub = 1 << g.sub_shift;
    CUtensorMap tk, tv;
    if (!encode_rows<D>(&tk, p.k, a.pages * a.page_size, (int64_t)a.Hk * D, sub) ||
        !encode_rows<D>(&tv, p.v, a.pages * a.page_size, (int64_t)a.Hk * D, sub))
        return cudaErrorInvalidValue;
    const int ctas = num_sms < kPagedMaxCtas ? num_sms : kPagedMaxCtas;
    auto kern = a.softcap_on ? q8_tc_kernel<D, FORM, true> : q8_tc_kernel<D, FORM, false>;
    cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kern), (int)Cfg<D>::kSmem);
    if (e != cudaSuccess) return e;
    if (a.tree) {  // the cached part runs beside the drafted one and waits for it at the end
        e = launch_paged_q8_draft(a, draft, stream);
        if (e == cudaSuccess) e = launch_pdl(kern, dim3(ctas), dim3(kThreads), Cfg<D>::kSmem, stream, tk, tv, g);
    } else {
        kern<<<ctas, kThreads, Cfg<D>::kSmem, stream>>>(tk, tv, g);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) return e;
    const int64_t most = (int64_t)a.max_rows * a.G;
    return launch_pdl(q8_tc_merge_kernel<D>, dim3((unsigned)ctas, (unsigned)((most < kM ? most : kM) + 7) / 8), dim3(256), 0,
                      stream, g);
}

}  // namespace

size_t paged_q8_tc_workspace(const PagedDesc& a) { return scratch_of(a.D, a.tree ? a.rows * a.H : 0).total; }

cudaError_t launch_paged_q8_tc(const PagedDesc& a, const Q8Pools& p, int num_sms, void* workspace, cudaStream_t stream) {
    if (a.D == 128)
        return p.form == kFormInt8 ? launch_form<128, kFormInt8>(a, p, num_sms, workspace, stream)
                                   : launch_form<128, kFormE4m3>(a, p, num_sms, workspace, stream);
    return p.form == kFormInt8 ? launch_form<64, kFormInt8>(a, p, num_sms, workspace, stream)
                               : launch_form<64, kFormE4m3>(a, p, num_sms, workspace, stream);
}

unsigned int paged_q8_tc_take_device_error() {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_q8_tc_device_error, sizeof(v)) != cudaSuccess) return 0;
    if (v) {
        const unsigned int zero = 0;
        cudaMemcpyToSymbol(g_q8_tc_device_error, &zero, sizeof(zero));
    }
    return v;
}

}  // namespace vtmu
