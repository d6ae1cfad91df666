// paged_q8_draft.cu -- the drafted rows of a tree beside an 8-bit cache: every row's
// attention over the (at most 64, f32) drafted rows of its request that its mask names.
// The cache's kernels join it with theirs.
//
// A CTA for up to 128 virtual rows (row x head of the group) of a KV head, a warp for 8.  K, V, q and
// the weights are f16 pairs hi + lo after a power of two per row (22 bits), three products each with
// f32 sums; all scores of a row are in registers, so its maximum is known before the first
// weight.  A drafted row with an element that is not finite counts as NaN, as it would in
// the cache.  The drafted rows are split once for the CTA, in shared memory, where a lane finds
// the operands of its products side by side: 8 trees of 64 rows and 32 heads took 49 us when every
// warp read and split them for itself (most of it waiting for L2), and take 19 now (each alone, caches cold).
#include <algorithm>

#include "attn_common.cuh"
#include "launch_cache.h"
#include "paged_q8_list.cuh"
#include "paged_q8_mma.cuh"
#include "pdl.cuh"

namespace vtmu {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int kMostWarps = 16, kRows = kTreeMaxRows;

// Shared memory: K rows hi, lo ([row][D] halves), V row pairs hi, lo ([pair][D] of (row 2 p, row 2 p + 1)),
// 16 bytes between rows so that a quarter of a warp meets no bank twice (V at headDim 64: twice);
// the powers of two of K and V rows (0: a row that is not finite).
template <int D>
struct DraftSmem {
    static constexpr int kPitchK = 2 * D + 16, kPitchV = 4 * D + 16;
    static constexpr int kHiK = 0, kLoK = kRows * kPitchK, kHiV = 2 * kLoK, kLoV = kHiV + kRows / 2 * kPitchV;
    static constexpr int kScale = kLoV + kRows / 2 * kPitchV, kBytes = kScale + 2 * kRows * 4;
};

template <int D>
__global__ void __launch_bounds__(32 * kMostWarps) q8_draft_kernel(const __grid_constant__ PagedDesc a, float2* ml) {
    constexpr int KC = D / 64, MT = D / 16;
    using S = DraftSmem<D>;
    extern __shared__ __align__(16) unsigned char smem[];
    float* kinv = reinterpret_cast<float*>(smem + S::kScale);
    float* vinv_s = kinv + kRows;
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, t4 = lane & 3;
    const int b = blockIdx.z, hk = blockIdx.y, v0 = 8 * (blockIdx.x * warps + warp);
    pdl_launch_dependents();
    const Q8Req rq = q8_load_req(a, b);
    if (8 * blockIdx.x * warps >= rq.T * a.G) return;

    // Queries, as in the cache's kernel: lane row gr is the virtual row.
    uint32_t qf[KC][4][4];
    float rf[2];
    {
        const int v = v0 + gr, t = v / a.G;
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
                y[c][s] = make_float4(x.x * a.qk_mul, x.y * a.qk_mul, x.z * a.qk_mul, x.w * a.qk_mul);
                top = q8_abs_top(top, y[c][s]);
            }
        top = fmaxf(top, __shfl_xor_sync(FULL, top, 1));
        top = fmaxf(top, __shfl_xor_sync(FULL, top, 2));
        const float sc = mma_row_scale(top, 13);
#pragma unroll
        for (int c = 0; c < KC; ++c)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                mma_split(y[c][s].x * sc, y[c][s].y * sc, qf[c][s][0], qf[c][s][2]);
                mma_split(y[c][s].z * sc, y[c][s].w * sc, qf[c][s][1], qf[c][s][3]);
            }
#pragma unroll
        for (int e = 0; e < 2; ++e) rf[e] = __shfl_sync(FULL, 1.f / sc, 4 * (2 * t4 + e));
    }

    // The drafted rows, split: a pair of rows of K or of V a job, D / 4 lanes a row, four channels a lane.
    const int blocks = (rq.T + 15) / 16;
    constexpr int L = D / 4;  // lanes of a row
    for (int job = warp * (32 / L) + lane / L; job < 16 * blocks; job += warps * (32 / L)) {
        const bool values = job >= 8 * blocks;
        const int pair = job - (values ? 8 * blocks : 0), l = lane % L;
        float4 y[2];
        float inv[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = 2 * pair + h;
            y[h] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (row < rq.T)
                y[h] = __ldg(reinterpret_cast<const float4*>((values ? a.v_new : a.k_new) +
                                                             ((int64_t)(rq.row0 + row) * a.Hk + hk) * D + 4 * l));
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float top = q8_abs_top(0.f, y[h]);
#pragma unroll
            for (int off = 1; off < L; off <<= 1) top = q8_nan_max(top, __shfl_xor_sync(FULL, top, off));
            inv[h] = top < INFINITY ? mma_row_scale(top, 8) : 0.f;
            if (l == 0) (values ? vinv_s : kinv)[2 * pair + h] = inv[h];
            if (inv[h] == 0.f) y[h] = make_float4(0.f, 0.f, 0.f, 0.f);
            y[h] = make_float4(y[h].x * inv[h], y[h].y * inv[h], y[h].z * inv[h], y[h].w * inv[h]);
        }
        uint4 hi, lo;
        if (values) {
            mma_split(y[0].x, y[1].x, hi.x, lo.x);
            mma_split(y[0].y, y[1].y, hi.y, lo.y);
            mma_split(y[0].z, y[1].z, hi.z, lo.z);
            mma_split(y[0].w, y[1].w, hi.w, lo.w);
            *reinterpret_cast<uint4*>(smem + S::kHiV + pair * S::kPitchV + 16 * l) = hi;
            *reinterpret_cast<uint4*>(smem + S::kLoV + pair * S::kPitchV + 16 * l) = lo;
        } else {
            mma_split(y[0].x, y[0].y, hi.x, lo.x);
            mma_split(y[0].z, y[0].w, hi.y, lo.y);
            mma_split(y[1].x, y[1].y, hi.z, lo.z);
            mma_split(y[1].z, y[1].w, hi.w, lo.w);
            unsigned char* to = smem + 2 * pair * S::kPitchK + 8 * l;
            *reinterpret_cast<uint2*>(to + S::kHiK) = make_uint2(hi.x, hi.y);
            *reinterpret_cast<uint2*>(to + S::kLoK) = make_uint2(lo.x, lo.y);
            *reinterpret_cast<uint2*>(to + S::kHiK + S::kPitchK) = make_uint2(hi.z, hi.w);
            *reinterpret_cast<uint2*>(to + S::kLoK + S::kPitchK) = make_uint2(lo.z, lo.w);
        }
    }
    __syncthreads();
    if (v0 >= rq.T * a.G) return;

    // Scores: block k holds drafted rows 16 k + gr (elements 0, 1) and + 8 (2, 3).
    float x[4][4], vinv[4][2];  // vinv: of value rows 16 k + gr + 8 h, 0 for a row that is not finite
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[k][e] = 0.f;
        if (k >= blocks) {
            vinv[k][0] = vinv[k][1] = 0.f;
            continue;
        }
        float ks[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float inv = kinv[16 * k + gr + 8 * h];
            ks[h] = inv != 0.f ? 1.f / inv : __int_as_float(0x7fc00000);
            vinv[k][h] = vinv_s[16 * k + gr + 8 * h];
        }
        // A lane's 16 channels of 64 are its channels of four steps, four each.
        const unsigned char* from = smem + (16 * k + gr) * S::kPitchK + 32 * t4;
#pragma unroll
        for (int c = 0; c < KC; ++c)
#pragma unroll
            for (int s2 = 0; s2 < 2; ++s2) {
                const uint4 h0 = *reinterpret_cast<const uint4*>(from + S::kHiK + 128 * c + 16 * s2);
                const uint4 h1 = *reinterpret_cast<const uint4*>(from + S::kHiK + 8 * S::kPitchK + 128 * c + 16 * s2);
                const uint4 l0 = *reinterpret_cast<const uint4*>(from + S::kLoK + 128 * c + 16 * s2);
                const uint4 l1 = *reinterpret_cast<const uint4*>(from + S::kLoK + 8 * S::kPitchK + 128 * c + 16 * s2);
                const uint32_t fh[2][4] = {{h0.x, h1.x, h0.y, h1.y}, {h0.z, h1.z, h0.w, h1.w}};
                const uint32_t fl[2][4] = {{l0.x, l1.x, l0.y, l1.y}, {l0.z, l1.z, l0.w, l1.w}};
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int s = 2 * s2 + i;
                    mma_16816(x[k], fh[i], qf[c][s][2], qf[c][s][3]);
                    mma_16816(x[k], fl[i], qf[c][s][0], qf[c][s][1]);
                    mma_16816(x[k], fh[i], qf[c][s][0], qf[c][s][1]);
                }
            }
#pragma unroll
        for (int e = 0; e < 4; ++e) x[k][e] *= q8_score_unit(ks[e >> 1], rf[e & 1]);
    }
    if (a.softcap_on) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[k][e] = a.cap_log2 * softcap_tanh(x[k][e]);
    }

    // Masks, maximum, and the largest product of weight and value scale, as a power of two.
    uint32_t see = 0;
    float m[2], l[2] = {0.f, 0.f}, r[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int v = v0 + 2 * t4 + e, t = v / a.G;
        uint64_t mask = 0;
        int64_t p = 0;
        if (v < rq.T * a.G) {
            mask = __ldg(reinterpret_cast<const unsigned long long*>(a.masks) + rq.row0 + t);
            if (a.window > 0) p = __ldg(a.positions + rq.row0 + t);
        }
        m[e] = -INFINITY;
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int j = 16 * k + gr + 8 * h;
                bool on = j < rq.T && ((mask >> j) & 1);
                if (on && a.window > 0) on = __ldg(a.positions + rq.row0 + j) > p - a.window;
                if (on) see |= 1u << (4 * k + 2 * h + e);
                if (on) m[e] = fmaxf(m[e], x[k][2 * h + e]);
            }
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) m[e] = fmaxf(m[e], __shfl_xor_sync(FULL, m[e], off));
    }
    // A value row is v = (v vinv) / vinv, vinv = 2^-E.
    auto power = [&](int k, int h) -> float {
        return vinv[k][h] == 0.f ? 0.f : (float)(127 - (int)(__float_as_uint(vinv[k][h]) >> 23));
    };
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const float mu = m[e] == -INFINITY ? 0.f : m[e];
        r[e] = -200.f;
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if ((see >> (4 * k + 2 * h + e)) & 1) r[e] = fmaxf(r[e], (x[k][2 * h + e] - mu) + power(k, h));
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) r[e] = fmaxf(r[e], __shfl_xor_sync(FULL, r[e], off));
        r[e] = ceilf(r[e]);
    }
    // Weights, at most 1 of the largest product, times 2^14 in f16.
    uint32_t ph[4][2], pl[4][2];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float mu = m[e & 1] == -INFINITY ? 0.f : m[e & 1], y = x[k][e] - mu;
            const bool on = (see >> (4 * k + e)) & 1, odd = vinv[k][e >> 1] == 0.f;
            const float p = on ? exp2f(y) : 0.f;
            l[e & 1] += p;
            w[e] = !on ? 0.f : odd ? __int_as_float(0x7fc00000) : exp2f(y + (power(k, e >> 1) - r[e & 1]) + 14.f);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            mma_split(w[2 * h], w[2 * h + 1], ph[k][h], pl[k][h]);
            ph[k][h] = mma_transpose(ph[k][h]);
            pl[k][h] = mma_transpose(pl[k][h]);
        }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l[e] += __shfl_xor_sync(FULL, l[e], off);

    float o[MT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (k >= blocks) break;
        // Pairs 8 k + t4 and + 4, channels (D / 8) gr + 2 i and the next for product i.
        const unsigned char* from = smem + (8 * k + t4) * S::kPitchV + D / 2 * gr;
#pragma unroll
        for (int i = 0; i < MT; i += 2) {
            const uint4 h0 = *reinterpret_cast<const uint4*>(from + S::kHiV + 8 * i);
            const uint4 h1 = *reinterpret_cast<const uint4*>(from + S::kHiV + 4 * S::kPitchV + 8 * i);
            const uint4 l0 = *reinterpret_cast<const uint4*>(from + S::kLoV + 8 * i);
            const uint4 l1 = *reinterpret_cast<const uint4*>(from + S::kLoV + 4 * S::kPitchV + 8 * i);
            const uint32_t fh[2][4] = {{h0.x, h0.y, h1.x, h1.y}, {h0.z, h0.w, h1.z, h1.w}};
            const uint32_t fl[2][4] = {{l0.x, l0.y, l1.x, l1.y}, {l0.z, l0.w, l1.z, l1.w}};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                mma_16816(o[i + j], fh[j], pl[k][0], pl[k][1]);
                mma_16816(o[i + j], fl[j], ph[k][0], ph[k][1]);
                mma_16816(o[i + j], fh[j], ph[k][0], ph[k][1]);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int v = v0 + 2 * t4 + e, t = v / a.G;
        if (v >= rq.T * a.G) continue;
        // 2^(r - 14) in two steps, each a whole power of two and a normal number.
        const float inv = l[e] != 0.f ? 1.f / l[e] : 0.f, half = floorf(0.5f * (r[e] - 14.f));
        const float p0 = exp2f(half), p1 = exp2f((r[e] - 14.f) - half);
        const int64_t row = ((int64_t)rq.row0 + t) * a.H + (int64_t)hk * a.G + (v - t * a.G);
        float* to = a.out + row * D + (D / 8) * gr;
#pragma unroll
        for (int i = 0; i < MT; i += 2)
            *reinterpret_cast<float4*>(to + 2 * i) =
                make_float4(o[i][e] * inv * p0 * p1, o[i][2 + e] * inv * p0 * p1, o[i + 1][e] * inv * p0 * p1,
                            o[i + 1][2 + e] * inv * p0 * p1);
        if (gr == 0) ml[row] = make_float2(m[e], l[e]);
    }
}

template <int D>
cudaError_t launch_d(const PagedDesc& a, float2* ml, cudaStream_t stream) {
    const cudaError_t e = set_smem_once(reinterpret_cast<const void*>(q8_draft_kernel<D>), DraftSmem<D>::kBytes);
    if (e != cudaSuccess) return e;
    // Eight warps at least, to split the rows.
    const int64_t eights = ((int64_t)a.max_rows * a.G + 7) / 8;
    const int warps = (int)std::min<int64_t>(std::max<int64_t>(eights, 8), kMostWarps);
    const dim3 grid((unsigned)((eights + warps - 1) / warps), (unsigned)a.Hk, (unsigned)a.B);
    q8_draft_kernel<D><<<grid, 32 * warps, DraftSmem<D>::kBytes, stream>>>(a, ml);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_q8_draft(const PagedDesc& a, float2* ml, cudaStream_t stream) {
    return a.D == 128 ? launch_d<128>(a, ml, stream) : launch_d<64>(a, ml, stream);
}

}  // namespace vtmu
