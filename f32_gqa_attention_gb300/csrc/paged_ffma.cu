// paged_ffma.cu -- attention of a ragged batch over a paged cache on the CUDA
// cores: any headDim to 256, any page size, f32 throughout.  It serves the
// shapes that the tensor-core kernel does not cover.
//
// For request b, query row t and head h, with virtual row v = t G + h % G of
// KV head h / G:  x2_s = log2 e * softcap(scale q.k_s), p_s = 2^(x2_s - m),
// out = sum p_s v_s / sum p_s over the keys that row t sees.
// One CTA per (tile of kR virtual rows, KV head, request); its eight warps take
// the chunks of 32 keys in turn and are joined at the end by the log-sum-exp
// rule.  Scores: lane = key, the lane reads its whole key row (served by L1
// after the first touch of a line) against the kR queries in shared memory.
// Values: lane = dims, one coalesced row per key; a key that no row sees is not
// read, and does not enter a row that does not see it: its probability there is -0,
// which exp2f never gives (one that is seen counts, were its weight +0: 0 x inf).  The keys of one request are not split over CTAs: lengths
// are known to the device alone, and this kernel needs no workspace.  Where both
// kernels cover a call the tensor cores win at every size measured: one token
// of a chat of 211 rows 36.9 us here and 28 there, small trees 99 and 32, one row
// for each of 32 requests of up to 8111 rows 2134 and 255, trees of 64 rows on 8
// requests of up to 32704 72.9 ms and 0.60.  Bound by the lanes' scattered reads of
// key rows and by the few CTAs of a small batch.
#include "attn_common.cuh"
#include "paged.cuh"
#include "paged_kernels.h"

namespace vtmu {
namespace {

constexpr int kR = 4;       // virtual rows per CTA
constexpr int kWarps = 8;
constexpr int kMaxD = 256;
constexpr int kPer = kMaxD / 32;
constexpr unsigned FULL = 0xffffffffu;
constexpr unsigned kUnseen = 0x80000000u;  // -0

__device__ __forceinline__ float apply_cap(const PagedDesc& a, float dot) {
    return a.softcap_on ? a.cap_log2 * softcap_tanh(dot * a.qk_mul) : dot * a.qk_mul;
}

template <bool VEC4>
__global__ void __launch_bounds__(32 * kWarps) paged_ffma_kernel(const PagedDesc a) {
    __shared__ __align__(16) float sq[kR][kMaxD];
    __shared__ float so[kWarps][kR][kMaxD];
    __shared__ float sm[kWarps][kR], sl[kWarps][kR];
    const int b = blockIdx.z, hk = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const PackedRows pr = packed_rows(a.cu_rows, b, a.B, a.rows);
    const int64_t nt = min(pr.n, (int64_t)a.max_rows);
    const int64_t v0 = (int64_t)blockIdx.x * kR, nv = nt * a.G;
    if (v0 >= nv) return;
    const int D = a.D;
    const int64_t len = clamp64(__ldg(a.lens + b), 0, (int64_t)a.max_pages * a.page_size);
    const int64_t total = a.tree ? len + nt : len;  // keys: the cache's rows, then the drafted ones

    for (int i = threadIdx.x; i < kR * D; i += blockDim.x) {
        const int r = i / D, d = i % D;
        const int64_t v = v0 + r;
        sq[r][d] = v < nv ? __ldg(a.q + ((pr.row0 + v / a.G) * a.H + (int64_t)hk * a.G + v % a.G) * D + d) : 0.f;
    }
    __syncthreads();

    int64_t pos[kR];
    uint64_t mask[kR];
    bool alive[kR];
    int64_t lo = total, hi = 0;  // the range of cache rows that some row of the tile sees
#pragma unroll
    for (int r = 0; r < kR; ++r) {
        const int64_t v = v0 + r, t = v < nv ? v / a.G : 0;
        alive[r] = v < nv;
        mask[r] = a.tree && alive[r] ? __ldg(reinterpret_cast<const unsigned long long*>(a.masks) + pr.row0 + t) : 0;
        pos[r] = !a.tree ? len - pr.n + t : a.window > 0 ? (int64_t)__ldg(a.positions + pr.row0 + t) : len;
        if (!alive[r]) continue;
        const int64_t rlo = a.window > 0 ? max(pos[r] - a.window + 1, (int64_t)0) : 0;
        const int64_t rhi = a.tree ? len : min(pos[r] + 1, len);
        lo = min(lo, rlo);
        hi = max(hi, rhi);
    }
    const int64_t sink_end = min(a.sinks, hi);

    float m[kR], l[kR], o[kR][kPer];
#pragma unroll
    for (int r = 0; r < kR; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) o[r][i] = 0.f;
    }

    for (int64_t c0 = (int64_t)warp * 32; c0 < total; c0 += 32 * kWarps) {
        // Chunks that lie wholly outside what the tile sees are passed over.
        if (c0 + 32 <= len && c0 >= sink_end && (c0 + 32 <= lo || c0 >= hi)) continue;
        const int64_t s = c0 + lane;
        const float* krow = nullptr;  // null: rows of zeros (a page id outside the pool)
        const float* vrow = nullptr;
        const bool drafted = s >= len;
        if (s < total) {
            if (drafted) {
                const int64_t r = pr.row0 + (s - len);
                krow = a.k_new + (r * a.Hk + hk) * D;
                vrow = a.v_new + (r * a.Hk + hk) * D;
            } else {
                const int64_t page = __ldg(a.block_table + (int64_t)b * a.max_pages + s / a.page_size);
                if (page >= 0 && page < a.pages) {
                    const int64_t r = page * a.page_size + s % a.page_size;
                    krow = a.k_pool + (r * a.Hk + hk) * D;
                    vrow = a.v_pool + (r * a.Hk + hk) * D;
                }
            }
        }
        const int64_t kpos = !drafted ? s : a.window > 0 && s < total ? (int64_t)__ldg(a.positions + pr.row0 + (s - len)) : s;
        bool see[kR], any = false;
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            bool v = alive[r] && s < total;
            if (drafted)
                v = v && ((mask[r] >> ((s - len) & 63)) & 1);
            else
                v = v && (a.tree || s <= pos[r]);
            if (a.window > 0) v = v && (kpos > pos[r] - a.window || (!drafted && s < a.sinks));
            see[r] = v;
            any = any || v;
        }
        if (!__any_sync(FULL, any)) continue;
        float x[kR];
#pragma unroll
        for (int r = 0; r < kR; ++r) x[r] = 0.f;
        if (any && krow) {
            if constexpr (VEC4) {
                for (int d = 0; d < D; d += 4) {
                    const float4 kv = __ldg(reinterpret_cast<const float4*>(krow + d));
#pragma unroll
                    for (int r = 0; r < kR; ++r) {
                        const float4 qv = *reinterpret_cast<const float4*>(&sq[r][d]);
                        x[r] = fmaf(qv.x, kv.x, fmaf(qv.y, kv.y, fmaf(qv.z, kv.z, fmaf(qv.w, kv.w, x[r]))));
                    }
                }
            } else {
                for (int d = 0; d < D; ++d) {
                    const float kv = __ldg(krow + d);
#pragma unroll
                    for (int r = 0; r < kR; ++r) x[r] = fmaf(sq[r][d], kv, x[r]);
                }
            }
        }
        float p[kR];
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            const float x2 = see[r] ? apply_cap(a, x[r]) : -INFINITY;
            float mt = x2;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) mt = fmaxf(mt, __shfl_xor_sync(FULL, mt, off));
            const float mn = fmaxf(m[r], mt), mu = mn == -INFINITY ? 0.f : mn;
            const float alpha = exp2f(m[r] - mu);
            p[r] = see[r] ? exp2f(x2 - mu) : -0.f;
            m[r] = mn;
            l[r] = fmaf(l[r], alpha, p[r]);  // this lane's keys
            if (alpha != 1.f) {
#pragma unroll
                for (int i = 0; i < kPer; ++i) o[r][i] *= alpha;
            }
        }
        for (int kk = 0; kk < 32; ++kk) {
            float w[kR];
            bool need = false;
#pragma unroll
            for (int r = 0; r < kR; ++r) {
                w[r] = __shfl_sync(FULL, p[r], kk);
                need = need || __float_as_uint(w[r]) != kUnseen;
            }
            const float* vr = reinterpret_cast<const float*>(
                __shfl_sync(FULL, reinterpret_cast<unsigned long long>(vrow), kk));
            if (!need || !vr) continue;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int d = lane + 32 * i;
                if (d < D) {
                    const float vv = __ldg(vr + d);
#pragma unroll
                    for (int r = 0; r < kR; ++r)
                        if (__float_as_uint(w[r]) != kUnseen) o[r][i] = fmaf(w[r], vv, o[r][i]);
                }
            }
        }
    }

#pragma unroll
    for (int r = 0; r < kR; ++r) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) l[r] += __shfl_xor_sync(FULL, l[r], off);
        if (lane == 0) {
            sm[warp][r] = m[r];
            sl[warp][r] = l[r];
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (lane + 32 * i < D) so[warp][r][lane + 32 * i] = o[r][i];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kR * D; i += blockDim.x) {
        const int r = i / D, d = i % D;
        const int64_t v = v0 + r;
        if (v >= nv) continue;
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sm[w][r]);
        float den = 0.f, acc = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (sl[w][r] == 0.f) continue;  // nothing seen; NaN scores leave the maximum at -inf, but not l at 0
            const float f = exp2f(sm[w][r] - mx);
            den = fmaf(sl[w][r], f, den);
            acc = fmaf(so[w][r][d], f, acc);
        }
        a.out[((pr.row0 + v / a.G) * a.H + (int64_t)hk * a.G + v % a.G) * D + d] = den != 0.f ? acc / den : 0.f;
    }
}

}  // namespace

cudaError_t launch_paged_ffma(const PagedDesc& a, cudaStream_t stream) {
    const int64_t tiles = ((int64_t)a.max_rows * a.G + kR - 1) / kR;
    const dim3 grid((unsigned)tiles, (unsigned)a.Hk, (unsigned)a.B);
    const uintptr_t mis = reinterpret_cast<uintptr_t>(a.k_pool) | reinterpret_cast<uintptr_t>(a.v_pool) |
                          reinterpret_cast<uintptr_t>(a.k_new) | reinterpret_cast<uintptr_t>(a.v_new);
    if (a.D % 4 == 0 && (mis & 15u) == 0)
        paged_ffma_kernel<true><<<grid, 32 * kWarps, 0, stream>>>(a);
    else
        paged_ffma_kernel<false><<<grid, 32 * kWarps, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace vtmu
