// norm_rope.cu -- an RMS norm of every head of a step's queries and keys and
// op "rope" at given positions (op catalog, vtmu.mpakt.dev/api/ops) in one pass
// over them.
//
// Mathematics, head by head: y = x / sqrt(mean x^2 + eps) (w + offset), then pair j of y
// turns by positions[axis(j)][t] inv_freq[j] as in rope.cu.  The norm
// needs the whole head before its first output, so a head stays in the registers of
// L lanes: eight elements each, the two quads of four pairs, so that the rotation
// needs no exchange; a lane past the rotated channels holds eight that pass through.
// Memory-bound: 8 bytes an element.  8111 rows of 32 + 8 heads of 128 (332 MB) take 61 us, 5.4 TB/s
// (81 % of the copy rate); without the streaming accesses 67, with a CTA per row and a table of
// sines in shared memory 74 to 100.  A few rows: 3.2 us in a replayed graph.
#include "norm_rope.h"
#include "rope.cuh"

namespace vtmu {
namespace {

constexpr int64_t kWave = 152 * 8;  // CTAs of 256 threads that are resident at once
constexpr unsigned FULL = 0xffffffffu;

// A pair's angle: position x turn, whole turns drop out of 64-bit arithmetic by themselves, so
// that the rest is exact to 2^-64 x position of a turn; then sine and cosine of it in f32.  No
// double: this GPU's are slow, and a table of 64 angles was most of a row's time.  (So were
// 64 different words of the parameters, read one after the other; a thread now reads its own once.)
struct Pair {
    uint64_t turn;
    int axis;
};
__device__ __forceinline__ Pair pair_of(const NormRopeArgs& a, unsigned j) {
    Pair p{0, 0};
    if (j < (unsigned)a.half) p = Pair{a.turn[j], a.axis[j]};
    return p;
}
__device__ __forceinline__ float2 cos_sin(const NormRopeArgs& a, const Pair& p, int64_t t) {
    const int64_t pos = __ldg(a.positions + p.axis * a.T + t);
    const int32_t part = (int32_t)(((uint64_t)pos * p.turn + 0x80000000ull) >> 32);  // of 2^32 to a turn, in [-1/2, 1/2)
    float s, c;
    // 2 pi / 2^32.  The angle's roundings (part, the factor, the product) come to 3.0e-7 at most, and __sincosf is
    // off by 2^-21.41 (sine) and 2^-21.19 (cosine) on [-pi, pi]: 7.2e-7 in all, below 2^-20.4.
    __sincosf((float)part * 1.4629180792671596e-9f, &s, &c);
    return make_float2(c * a.attn, s * a.attn);
}

// Sums of squares that leave f32's range (elements from about 2^63 on, or beside an eps like that), or its precision
// (all below 2^-40, with no eps to speak of), are taken once more of the elements times a
// power of two, `pre`: kDown or kUp.  Both ends' squares fit, 4096
// of them too.
constexpr float kDown = 0x1p-96f, kUp = 0x1p90f;
__device__ __forceinline__ float pre_of(float ss, const NormRopeArgs& a) {
    if (!(ss + a.eps <= 3.0e38f)) return kDown;
    return ss < 0x1p-80f && a.eps < 0x1p-80f ? kUp : 1.f;
}
// What an element is multiplied by, one after the other: `pre` first on the way up; on the way down last, where
// small elements keep their bits (x first is at most 64 2^96).
__device__ __forceinline__ float2 factors_of(float ss, float pre, const NormRopeArgs& a) {
    const float eps = a.eps * pre * pre;  // below 2^100, and 0 where it says nothing beside the squares
    const float f = rsqrtf(fmaf(ss, a.inv_d, eps));
    return pre == kDown ? make_float2(f, pre) : make_float2(pre, f);
}

__device__ __forceinline__ float sq4(const float4& x, float f) {
    const float a = x.x * f, b = x.y * f, c = x.z * f, d = x.w * f;
    return fmaf(a, a, fmaf(b, b, fmaf(c, c, d * d)));
}
__device__ __forceinline__ float4 scale4(const float4& x, float f, const float4& w) {
    return make_float4(x.x * f * w.x, x.y * f * w.y, x.z * f * w.z, x.w * f * w.w);
}

// A warp's job is IT turns of 32 / L heads of a row (D <= 8 L), all of whose elements are asked for
// before the first is used; warps share nothing and wait for nobody.  A lane's four pairs are the
// same in every job, so their turns stay in registers (64 different words of the
// parameters are read one after the other), and their sines and cosines serve all heads of
// the job.
template <int IT>
__global__ void __launch_bounds__(128, 6) norm_rope_fast(const __grid_constant__ NormRopeArgs a, int log_l, unsigned chunks) {
    const int half = a.half, D = a.D, heads = a.H + a.Hk, L = 1 << log_l, side = 32 >> log_l;
    const int lane = threadIdx.x & (L - 1), group = (threadIdx.x & 31) >> log_l;
    // This lane's two quads: channels ia .. ia + 3 and ib .. ib + 3.
    const bool turns = 4 * lane < half, on = 8 * lane < D;
    int ia = 8 * lane, ib = ia + 4;  // interleaved pairs; or behind 2 half channels, which are 8 a lane too
    if (turns && !a.interleaved) {
        ia = 4 * lane;
        ib = 4 * lane + half;
    }
    Pair pair[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) pair[k] = pair_of(a, 4 * lane + k);

    // Weights of q and of k, with their offset; ones without.
    float4 wq[2], wk[2];
    auto weights = [&](const float* w, float4 (&r)[2]) {
        r[0] = r[1] = make_float4(1.f, 1.f, 1.f, 1.f);
        if (!w || !on) return;
        const float o = a.weight_offset;
        const float4 x = __ldg(reinterpret_cast<const float4*>(w + ia)), y = __ldg(reinterpret_cast<const float4*>(w + ib));
        r[0] = make_float4(x.x + o, x.y + o, x.z + o, x.w + o);
        r[1] = make_float4(y.x + o, y.y + o, y.z + o, y.w + o);
    };
    weights(a.qw, wq);
    weights(a.kw, wk);
    const unsigned jobs = (unsigned)a.T * chunks, step = gridDim.x * 4;
    for (unsigned job = blockIdx.x * 4 + (threadIdx.x >> 5); job < jobs; job += step) {
        const int64_t t = job / chunks;
        const int h0 = (int)(job - (unsigned)t * chunks) * (IT * side) + group;
        const int64_t q_row = t * a.H * D, k_row = (t * a.Hk - a.H) * D;  // + h D: heads of k come after q's
        float4 u[IT], v[IT];
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int h = h0 + i * side;
            u[i] = v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (h < heads && on) {
                const float* x = (h < a.H ? a.q + q_row : a.k + k_row) + h * D;
                u[i] = __ldcs(reinterpret_cast<const float4*>(x + ia));
                v[i] = __ldcs(reinterpret_cast<const float4*>(x + ib));
            }
        }
        bool skip = false;
        for (int i = 0; i < a.axes; ++i) skip = skip || __ldg(a.positions + i * a.T + t) < 0;
        if (skip) continue;  // the same for the whole warp
        float2 cs[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) cs[k] = turns ? cos_sin(a, pair[k], t) : make_float2(1.f, 0.f);
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int h = h0 + i * side;
            const bool live = h < heads && on, query = h < a.H;
            float4 p = u[i], q = v[i];
            if (a.norm) {
                auto sum = [&](float f) {
                    float ss = live ? sq4(u[i], f) + sq4(v[i], f) : 0.f;
                    for (int off = L / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(FULL, ss, off);
                    return ss;
                };
                // The rare second sum is taken by every group of the warp where one wants it.
                float ss = sum(1.f);
                const float pre = pre_of(ss, a);
                const bool far = __any_sync(FULL, pre != 1.f);
                if (far) ss = sum(pre);
                const float2 f = factors_of(ss, pre, a);
                if (far) {
                    p = make_float4(p.x * f.x, p.y * f.x, p.z * f.x, p.w * f.x);
                    q = make_float4(q.x * f.x, q.y * f.x, q.z * f.x, q.w * f.x);
                }
                p = scale4(p, f.y, query ? wq[0] : wk[0]);
                q = scale4(q, f.y, query ? wq[1] : wk[1]);
            }
            if (!live) continue;
            if (turns) {
                const float4 y = p, z = q;
                if (a.interleaved) {
                    p = make_float4(rope_channel(y.x, y.y, true, cs[0]), rope_channel(y.y, y.x, false, cs[0]),
                                    rope_channel(y.z, y.w, true, cs[1]), rope_channel(y.w, y.z, false, cs[1]));
                    q = make_float4(rope_channel(z.x, z.y, true, cs[2]), rope_channel(z.y, z.x, false, cs[2]),
                                    rope_channel(z.z, z.w, true, cs[3]), rope_channel(z.w, z.z, false, cs[3]));
                } else {
                    p = make_float4(rope_channel(y.x, z.x, true, cs[0]), rope_channel(y.y, z.y, true, cs[1]),
                                    rope_channel(y.z, z.z, true, cs[2]), rope_channel(y.w, z.w, true, cs[3]));
                    q = make_float4(rope_channel(z.x, y.x, false, cs[0]), rope_channel(z.y, y.y, false, cs[1]),
                                    rope_channel(z.z, y.z, false, cs[2]), rope_channel(z.w, y.w, false, cs[3]));
                }
            }
            float* o = (query ? a.q_out + q_row : a.k_out + k_row) + h * D;
            __stcs(reinterpret_cast<float4*>(o + ia), p);
            __stcs(reinterpret_cast<float4*>(o + ib), q);
        }
    }
}

// Any width and alignment: a warp per head, which it reads twice.
__global__ void __launch_bounds__(256) norm_rope_any(const __grid_constant__ NormRopeArgs a) {
    __shared__ float2 cs[kRopeMaxPairs];
    const int half = a.half, D = a.D, heads = a.H + a.Hk;
    const Pair mine = pair_of(a, threadIdx.x);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        bool skip = false;
        for (int i = 0; i < a.axes; ++i) skip = skip || __ldg(a.positions + i * a.T + t) < 0;
        if (skip) continue;
        __syncthreads();
        if (threadIdx.x < half) cs[threadIdx.x] = cos_sin(a, mine, t);
        __syncthreads();
        for (int h = warp; h < heads; h += 8) {
            const bool query = h < a.H;
            const float* x = query ? a.q + (t * a.H + h) * D : a.k + (t * a.Hk + (h - a.H)) * D;
            float* o = query ? a.q_out + (t * a.H + h) * D : a.k_out + (t * a.Hk + (h - a.H)) * D;
            const float* w = query ? a.qw : a.kw;
            float2 f = make_float2(1.f, 1.f);
            if (a.norm) {
                auto sum = [&](float m) {
                    float ss = 0.f;
                    for (int d = lane; d < D; d += 32) ss = fmaf(x[d] * m, x[d] * m, ss);
                    for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(FULL, ss, off);
                    return ss;
                };
                float ss = sum(1.f);
                const float pre = pre_of(ss, a);
                if (pre != 1.f) ss = sum(pre);
                f = factors_of(ss, pre, a);
            }
            __syncwarp();  // in place: every lane has read the head before one writes it
            auto normed = [&](int d) { return a.norm ? x[d] * f.x * f.y * (w ? __ldg(w + d) + a.weight_offset : 1.f) : x[d]; };
            for (int j = lane; j < half; j += 32) {
                const int ia = a.interleaved ? 2 * j : j, ib = a.interleaved ? 2 * j + 1 : j + half;
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
    const uintptr_t mis = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k) |
                          reinterpret_cast<uintptr_t>(a.qw) | reinterpret_cast<uintptr_t>(a.kw) |
                          reinterpret_cast<uintptr_t>(a.q_out) | reinterpret_cast<uintptr_t>(a.k_out);
    int log_l = 0;
    while (8 << log_l < a.D) ++log_l;
    const int64_t heads = (int64_t)a.H + a.Hk, side = 32 >> (log_l < 5 ? log_l : 5);
    // Quads of four pairs and 16-byte accesses; other widths turn a pair at a time.
    if ((mis & 15u) == 0 && a.D % 8 == 0 && a.D <= 256 && a.half % 4 == 0 && a.T * heads < ((int64_t)1 << 31)) {
        // Few rows: a turn a job, for the latency.
        const bool few = a.T * heads < 16 * kWave * side;
        const int64_t each = (few ? 1 : 4) * side, chunks = (heads + each - 1) / each, ctas = (a.T * chunks + 3) / 4;
        const unsigned grid = (unsigned)(ctas < 6 * 152 ? ctas : 6 * 152);  // resident at once
        if (few)
            norm_rope_fast<1><<<grid, 128, 0, stream>>>(a, log_l, (unsigned)chunks);
        else
            norm_rope_fast<4><<<grid, 128, 0, stream>>>(a, log_l, (unsigned)chunks);
    } else {
        const unsigned blocks = (unsigned)(a.T < kWave ? a.T : kWave);
        norm_rope_any<<<blocks, 256, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace vtmu
