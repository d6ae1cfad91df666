// norm_rope.cu -- an RMS norm of every head of a step's queries and keys and
// op "rope" at given positions (op catalog, vtmu.mpakt.dev/api/ops) in one pass
// over them.
//
// Mathematics, head by head: y = x / sqrt(mean x^2 + eps) (w + offset), then pair j of y
// turns by positions[axis(j)][t] inv_freq[j] as in rope.cu (angle in double).  The norm
// needs the whole head before its first output, so a head stays in the registers of
// L lanes: eight elements each, the two quads of four pairs, so that the rotation
// needs no exchange; a lane past the rotated channels holds eight that pass through.
// Memory-bound: 8 bytes an element.  A CTA per row; it asks for the first heads' elements
// before it forms the row's (cos, sin) table, which hides one behind the other.
#include "norm_rope.h"
#include "rope.cuh"

namespace vtmu {
namespace {

constexpr int64_t kWave = 152 * 8;  // CTAs of 256 threads that are resident at once
constexpr unsigned FULL = 0xffffffffu;

// Sums of squares that leave f32's range (elements from about 2^63 on), or its precision
// (below about 2^-36, with no eps to speak of), are taken once more of the elements times a
// power of two, `pre`, which the elements then keep: kDown or kUp.  Both ends' squares fit, 256
// of them too.
constexpr float kDown = 0x1p-96f, kUp = 0x1p90f;
__device__ __forceinline__ float pre_of(float ss, const NormRopeArgs& a) {
    if (!(ss <= 3.0e38f)) return kDown;
    return ss / (float)a.D < 0x1p-80f && a.eps < 0x1p-80f ? kUp : 1.f;
}
__device__ __forceinline__ float factor_of(float ss, float pre, const NormRopeArgs& a) {
    const float eps = pre == 1.f ? a.eps : pre == kUp ? a.eps * kUp * kUp : 0.f;
    return rsqrtf(fmaf(ss, 1.f / (float)a.D, eps));
}

__device__ __forceinline__ float sq4(const float4& x, float f) {
    const float a = x.x * f, b = x.y * f, c = x.z * f, d = x.w * f;
    return fmaf(a, a, fmaf(b, b, fmaf(c, c, d * d)));
}
__device__ __forceinline__ float4 scale4(const float4& x, float f, const float4& w) {
    return make_float4(x.x * f * w.x, x.y * f * w.y, x.z * f * w.z, x.w * f * w.w);
}

// L lanes to a head (D <= 8 L), all of a warp's groups in step.
__global__ void __launch_bounds__(256) norm_rope_fast(const __grid_constant__ NormRopeArgs a, int L) {
    __shared__ __align__(16) float2 cs[kRopeMaxPairs];
    const int half = a.r.half, D = a.D, heads = a.H + a.Hk, groups = 256 / L;
    const int group = threadIdx.x / L, lane = threadIdx.x % L;
    // This lane's two quads: channels ia .. ia + 3 and ib .. ib + 3.
    const bool turns = 4 * lane < half, on = 8 * lane < D;
    int ia, ib;
    if (turns) {
        ia = a.r.interleaved ? 8 * lane : 4 * lane;
        ib = a.r.interleaved ? 8 * lane + 4 : 4 * lane + half;
    } else {
        ia = 8 * lane;  // behind 2 half channels, which are 8 a lane too
        ib = ia + 4;
    }
    const int rounds = (heads + groups - 1) / groups;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        bool skip = false;
        for (int i = 0; i < a.axes; ++i) skip = skip || __ldg(a.positions + i * a.T + t) < 0;
        if (skip) continue;  // the same for every thread of the CTA
        float4 u = make_float4(0.f, 0.f, 0.f, 0.f), v = u;
        auto load = [&](int h) {
            if (h >= heads || !on) return;
            const float* x = h < a.H ? a.q + (t * a.H + h) * D : a.k + (t * a.Hk + (h - a.H)) * D;
            u = *reinterpret_cast<const float4*>(x + ia);
            v = *reinterpret_cast<const float4*>(x + ib);
        };
        load(group);
        __syncthreads();  // the previous row's table is no longer read
        for (int j = threadIdx.x; j < half; j += 256)
            cs[j] = rope_cos_sin(a.r, __ldg(a.positions + a.axis[j] * a.T + t), j);
        __syncthreads();
        for (int i = 0, h = group; i < rounds; ++i, h += groups) {
            if (i > 0) load(h);
            const bool live = h < heads && on;
            const bool query = h < a.H;
            float4 p = u, q = v;
            if (a.norm) {
                auto sum = [&](float f) {
                    float ss = live ? sq4(u, f) + sq4(v, f) : 0.f;
                    for (int off = L / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(FULL, ss, off);
                    return ss;
                };
                // The rare second sum is taken by every group of the warp where one wants it.
                float ss = sum(1.f);
                const float pre = pre_of(ss, a);
                if (__any_sync(FULL, pre != 1.f)) {
                    ss = sum(pre);
                    u = make_float4(u.x * pre, u.y * pre, u.z * pre, u.w * pre);
                    v = make_float4(v.x * pre, v.y * pre, v.z * pre, v.w * pre);
                }
                const float f = factor_of(ss, pre, a);
                const float* w = query ? a.qw : a.kw;
                float4 w0 = make_float4(1.f, 1.f, 1.f, 1.f), w1 = w0;
                if (w && live) {
                    const float o = a.weight_offset;
                    w0 = __ldg(reinterpret_cast<const float4*>(w + ia));
                    w1 = __ldg(reinterpret_cast<const float4*>(w + ib));
                    w0 = make_float4(w0.x + o, w0.y + o, w0.z + o, w0.w + o);
                    w1 = make_float4(w1.x + o, w1.y + o, w1.z + o, w1.w + o);
                }
                p = scale4(u, f, w0);
                q = scale4(v, f, w1);
            }
            if (!live) continue;
            if (turns) {
                const int j = 4 * lane;
                const float4 c01 = *reinterpret_cast<const float4*>(&cs[j]), c23 = *reinterpret_cast<const float4*>(&cs[j + 2]);
                const float2 c0 = make_float2(c01.x, c01.y), c1 = make_float2(c01.z, c01.w), c2 = make_float2(c23.x, c23.y),
                             c3 = make_float2(c23.z, c23.w);
                const float4 y = p, z = q;
                if (a.r.interleaved) {
                    p = make_float4(rope_channel(y.x, y.y, true, c0), rope_channel(y.y, y.x, false, c0),
                                    rope_channel(y.z, y.w, true, c1), rope_channel(y.w, y.z, false, c1));
                    q = make_float4(rope_channel(z.x, z.y, true, c2), rope_channel(z.y, z.x, false, c2),
                                    rope_channel(z.z, z.w, true, c3), rope_channel(z.w, z.z, false, c3));
                } else {
                    p = make_float4(rope_channel(y.x, z.x, true, c0), rope_channel(y.y, z.y, true, c1),
                                    rope_channel(y.z, z.z, true, c2), rope_channel(y.w, z.w, true, c3));
                    q = make_float4(rope_channel(z.x, y.x, false, c0), rope_channel(z.y, y.y, false, c1),
                                    rope_channel(z.z, y.z, false, c2), rope_channel(z.w, y.w, false, c3));
                }
            }
            float* o = query ? a.q_out + (t * a.H + h) * D : a.k_out + (t * a.Hk + (h - a.H)) * D;
            *reinterpret_cast<float4*>(o + ia) = p;
            *reinterpret_cast<float4*>(o + ib) = q;
        }
    }
}

// Any width and alignment: a warp per head, which it reads twice.
__global__ void __launch_bounds__(256) norm_rope_any(const __grid_constant__ NormRopeArgs a) {
    __shared__ float2 cs[kRopeMaxPairs];
    const int half = a.r.half, D = a.D, heads = a.H + a.Hk;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        bool skip = false;
        for (int i = 0; i < a.axes; ++i) skip = skip || __ldg(a.positions + i * a.T + t) < 0;
        if (skip) continue;
        __syncthreads();
        for (int j = threadIdx.x; j < half; j += 256)
            cs[j] = rope_cos_sin(a.r, __ldg(a.positions + a.axis[j] * a.T + t), j);
        __syncthreads();
        for (int h = warp; h < heads; h += 8) {
            const bool query = h < a.H;
            const float* x = query ? a.q + (t * a.H + h) * D : a.k + (t * a.Hk + (h - a.H)) * D;
            float* o = query ? a.q_out + (t * a.H + h) * D : a.k_out + (t * a.Hk + (h - a.H)) * D;
            const float* w = query ? a.qw : a.kw;
            float f = 1.f, pre = 1.f;
            if (a.norm) {
                auto sum = [&](float m) {
                    float ss = 0.f;
                    for (int d = lane; d < D; d += 32) ss = fmaf(x[d] * m, x[d] * m, ss);
                    for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(FULL, ss, off);
                    return ss;
                };
                float ss = sum(1.f);
                pre = pre_of(ss, a);
                if (pre != 1.f) ss = sum(pre);
                f = factor_of(ss, pre, a);
            }
            __syncwarp();  // in place: every lane has read the head before one writes it
            auto normed = [&](int d) { return a.norm ? x[d] * pre * f * (w ? __ldg(w + d) + a.weight_offset : 1.f) : x[d]; };
            for (int j = lane; j < half; j += 32) {
                const int ia = a.r.interleaved ? 2 * j : j, ib = a.r.interleaved ? 2 * j + 1 : j + half;
                const float y = normed(ia), z = normed(ib);
                o[ia] = rope_channel(y, z, true, cs[j]);
                o[ib] = rope_channel(z, y, false, cs[j]);
            }
            for (int d = 2 * half + lane; d < D; d += 32) o[d] = normed(d);
        }
    }
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, cudaStream_t stream) {
    if (a.T == 0) return cudaSuccess;
    const unsigned blocks = (unsigned)(a.T < kWave ? a.T : kWave);
    const uintptr_t mis = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k) |
                          reinterpret_cast<uintptr_t>(a.qw) | reinterpret_cast<uintptr_t>(a.kw) |
                          reinterpret_cast<uintptr_t>(a.q_out) | reinterpret_cast<uintptr_t>(a.k_out);
    // Quads of four pairs and 16-byte accesses; other widths turn a pair at a time.
    if ((mis & 15u) == 0 && a.D % 8 == 0 && a.D <= 256 && a.r.half % 4 == 0) {
        int L = 1;
        while (8 * L < a.D) L *= 2;
        norm_rope_fast<<<blocks, 256, 0, stream>>>(a, L);
    } else {
        norm_rope_any<<<blocks, 256, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace vtmu
