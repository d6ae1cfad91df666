// paged_q8_draft.cu -- the drafted rows of a tree beside an 8-bit cache: every row's
// attention over the (at most 64, f32) drafted rows of its request that its mask names.
// The cache's kernels join it with theirs.
//
// A warp for 8 virtual rows (row x head of the group) of a KV head.  K, V, q and the weights
// are f16 pairs hi + lo after a power of two per row (22 bits), three products each with f32
// sums; all scores of a row are in registers, so its maximum is known before the first
// weight.  A drafted row with an element that is not finite counts as NaN, as it would in
// the cache.  Bound by the latency of one pass: 8 trees of 64 rows and 32 heads are
// 1024 warps and 17 MB.
#include "attn_common.cuh"
#include "paged_q8_list.cuh"
#include "paged_q8_mma.cuh"
#include "pdl.cuh"

namespace vtmu {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int kWarps = 4;

template <int D>
__global__ void __launch_bounds__(32 * kWarps) q8_draft_kernel(const __grid_constant__ PagedDesc a, float2* ml) {
    constexpr int KC = D / 64, MT = D / 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, t4 = lane & 3;
    const int b = blockIdx.z, hk = blockIdx.y, v0 = 8 * (blockIdx.x * kWarps + warp);
    pdl_launch_dependents();
    const Q8Req rq = q8_load_req(a, b);
    if (v0 >= rq.T * a.G) return;

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

    // Scores: block k holds drafted rows 16 k + gr (elements 0, 1) and + 8 (2, 3).
    const int blocks = (rq.T + 15) / 16;
    float x[4][4], vinv[4][2];  // vinv: of value rows 16 k + gr + 8 h, 0 for a row that is not finite
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[k][e] = 0.f;
        if (k >= blocks) {
            vinv[k][0] = vinv[k][1] = 0.f;
            continue;
        }
        const float* kr[2];
        float inv[2], ks[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t at = ((int64_t)(rq.row0 + min(16 * k + gr + 8 * h, rq.T - 1)) * a.Hk + hk) * D;
            kr[h] = a.k_new + at;
            float top[2] = {0.f, 0.f};
            for (int d = 4 * t4; d < D; d += 16) {
                top[0] = q8_abs_top(top[0], __ldg(reinterpret_cast<const float4*>(kr[h] + d)));
                top[1] = q8_abs_top(top[1], __ldg(reinterpret_cast<const float4*>(a.v_new + at + d)));
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                top[i] = q8_nan_max(top[i], __shfl_xor_sync(FULL, top[i], 1));
                top[i] = q8_nan_max(top[i], __shfl_xor_sync(FULL, top[i], 2));
            }
            inv[h] = top[0] < INFINITY ? mma_row_scale(top[0], 8) : 0.f;
            ks[h] = inv[h] != 0.f ? 1.f / inv[h] : __int_as_float(0x7fc00000);
            vinv[k][h] = top[1] < INFINITY ? mma_row_scale(top[1], 8) : 0.f;
        }
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
                mma_16816(x[k], fh, qf[c][s][2], qf[c][s][3]);
                mma_16816(x[k], fl, qf[c][s][0], qf[c][s][1]);
                mma_16816(x[k], fh, qf[c][s][0], qf[c][s][1]);
            }
#pragma unroll
        for (int e = 0; e < 4; ++e) x[k][e] *= ks[e >> 1] * rf[e & 1];
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
        const float* vr[4];
        float vi[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // rows 2 t4, + 1, + 8, + 9: what lanes of row gr = 2 t4 (+ 1) found
            vi[j] = __shfl_sync(FULL, vinv[k][j >> 1], 4 * (2 * t4 + (j & 1)));
            vr[j] = a.v_new + ((int64_t)(rq.row0 + min(16 * k + 2 * t4 + (j & 1) + 8 * (j >> 1), rq.T - 1)) * a.Hk + hk) * D +
                    (D / 8) * gr;
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            uint32_t fh[4], fl[4];
            float2 y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                y[j] = __ldg(reinterpret_cast<const float2*>(vr[j] + 2 * i));
                y[j] = vi[j] == 0.f ? make_float2(0.f, 0.f) : make_float2(y[j].x * vi[j], y[j].y * vi[j]);
            }
            mma_split(y[0].x, y[1].x, fh[0], fl[0]);
            mma_split(y[0].y, y[1].y, fh[1], fl[1]);
            mma_split(y[2].x, y[3].x, fh[2], fl[2]);
            mma_split(y[2].y, y[3].y, fh[3], fl[3]);
            mma_16816(o[i], fh, pl[k][0], pl[k][1]);
            mma_16816(o[i], fl, ph[k][0], ph[k][1]);
            mma_16816(o[i], fh, ph[k][0], ph[k][1]);
        }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int v = v0 + 2 * t4 + e, t = v / a.G;
        if (v >= rq.T * a.G) continue;
        const float inv = l[e] != 0.f ? 1.f / l[e] : 0.f, half = exp2f(0.5f * (r[e] - 14.f));  // 2^(r - 14), in two steps
        const int64_t row = ((int64_t)rq.row0 + t) * a.H + (int64_t)hk * a.G + (v - t * a.G);
        float* to = a.out + row * D + (D / 8) * gr;
#pragma unroll
        for (int i = 0; i < MT; i += 2)
            *reinterpret_cast<float4*>(to + 2 * i) =
                make_float4(o[i][e] * inv * half * half, o[i][2 + e] * inv * half * half, o[i + 1][e] * inv * half * half,
                            o[i + 1][2 + e] * inv * half * half);
        if (gr == 0) ml[row] = make_float2(m[e], l[e]);
    }
}

}  // namespace

cudaError_t launch_paged_q8_draft(const PagedDesc& a, float2* ml, cudaStream_t stream) {
    const int64_t blocks = ((int64_t)a.max_rows * a.G + 8 * kWarps - 1) / (8 * kWarps);
    const dim3 grid((unsigned)blocks, (unsigned)a.Hk, (unsigned)a.B);
    if (a.D == 128)
        q8_draft_kernel<128><<<grid, 32 * kWarps, 0, stream>>>(a, ml);
    else
        q8_draft_kernel<64><<<grid, 32 * kWarps, 0, stream>>>(a, ml);
    return cudaGetLastError();
}

}  // namespace vtmu
