// paged_q8.cu -- writes into an 8-bit paged cache and reads out of it: op
// "cache_write" through a slot map (op catalog, vtmu.mpakt.dev/api/ops) whose
// rows are quantised on the way, and its inverse.
//
// The unit is a KV head of a row: D elements x share a scale s.
//   int8:  s = max |x| / 127 rounded to f32, code = nearest integer to x / s;
//   e4m3:  s = 2^k, the least with max |x| <= 448 s, code = nearest e4m3 to x / s.
// Ties go to even, s is at least 2^-126 (rows of zeros and subnormal ones), and a
// unit with an element that is not finite has s = NaN and codes 0, so that nothing
// of it passes for a number.  A power of two costs e4m3 nothing (its relative
// step is the same at every size) and makes x / s and code x s exact; int8, whose
// steps are even, would lose up to one bit to it.
#include "paged_q8.cuh"

namespace vtmu {
namespace {

// ---- write -----------------------------------------------------------------------
// Memory-bound: 5 bytes an element and log2 L shuffles.  L lanes hold a unit, eight elements
// each as two 16-byte loads D / 2 apart (so that each load of the group is one run of D / 2
// elements); any D to 256 that is a multiple of 8.  A CTA takes ROWS rows and asks for the
// slots and then the elements of all of them before it forms a code.  32003 rows of 8 heads of 128
// (323 MB) take 51 us as e4m3, 95 % of the copy rate; a row at a time 63.  As int8 64 us, 76 %: q8_nearest is
// several instructions an element where e4m3 has half a conversion.
template <int FORM, int ROWS>
__global__ void __launch_bounds__(256) paged_write_q8_fast(const Q8WriteArgs a, int log_l) {
    const int lane = threadIdx.x & ((1 << log_l) - 1), group = threadIdx.x >> log_l, groups = 256 >> log_l;
    const int D = a.D, parts = 2 * a.Hk;
    const int64_t r0 = (int64_t)blockIdx.x * ROWS;
    int64_t slot[ROWS];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
        slot[k] = r0 + k < a.rows ? (int64_t)__ldg(a.slots + r0 + k) : -1;
        if (slot[k] >= a.pool_rows) slot[k] = -1;
    }
    const bool on = 8 * lane < D;
    // All of a warp's groups in step, for the shuffles.
    for (int p0 = 0; p0 < parts; p0 += groups) {
        const int part = p0 + group;
        const bool values = part >= a.Hk;
        const int head = part - (values ? a.Hk : 0);
        const bool mine = part < parts && on;
        const float* x = (values ? a.v_new : a.k_new) + (r0 * a.Hk + head) * D + 4 * lane;
        const int64_t pitch = (int64_t)a.Hk * D;
        float4 u[ROWS], v[ROWS];
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            u[k] = v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (mine && slot[k] >= 0) {
                u[k] = __ldcs(reinterpret_cast<const float4*>(x + k * pitch));
                v[k] = __ldcs(reinterpret_cast<const float4*>(x + k * pitch + D / 2));
            }
        }
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            float top = q8_abs_top(q8_abs_top(0.f, u[k]), v[k]);
            for (int off = 1 << log_l >> 1; off > 0; off >>= 1) top = q8_nan_max(top, __shfl_xor_sync(0xffffffffu, top, off));
            const Q8Scale s = q8_scale<FORM>(top);
            if (!mine || slot[k] < 0) continue;
            const int64_t unit = slot[k] * a.Hk + head;
            uint8_t* to = (values ? a.v_pool : a.k_pool) + unit * D;
            reinterpret_cast<uint32_t*>(to)[lane] = q8_codes4<FORM>(u[k], s);
            reinterpret_cast<uint32_t*>(to + D / 2)[lane] = q8_codes4<FORM>(v[k], s);
            if (lane == 0) (values ? a.v_scale : a.k_scale)[unit] = s.scale;
        }
    }
}
// Any width and alignment: a warp walks a unit twice.
template <int FORM>
__global__ void __launch_bounds__(256) paged_write_q8_any(const Q8WriteArgs a) {
    const int lane = threadIdx.x & 31, D = a.D;
    const int64_t r = blockIdx.x;
    const int64_t slot = __ldg(a.slots + r);
    if (slot < 0 || slot >= a.pool_rows) return;
    for (int part = threadIdx.x >> 5; part < 2 * a.Hk; part += 8) {
        const bool values = part >= a.Hk;
        const int head = part - (values ? a.Hk : 0);
        const float* x = (values ? a.v_new : a.k_new) + (r * a.Hk + head) * D;
        float top = 0.f;
        for (int d = lane; d < D; d += 32) top = q8_nan_max(top, fabsf(__ldg(x + d)));
        for (int off = 16; off > 0; off >>= 1) top = q8_nan_max(top, __shfl_xor_sync(0xffffffffu, top, off));
        const Q8Scale s = q8_scale<FORM>(top);
        const int64_t unit = slot * a.Hk + head;
        uint8_t* to = (values ? a.v_pool : a.k_pool) + unit * D;
        for (int d = lane; d < D; d += 32) to[d] = q8_code<FORM>(__ldg(x + d), s);
        if (lane == 0) (values ? a.v_scale : a.k_scale)[unit] = s.scale;
    }
}

// ---- read ------------------------------------------------------------------------
// Memory-bound, four fifths of it the f32 rows written.  A thread keeps its column (four
// codes, or one: N) and takes ROWS rows of it, all of whose slots, codes and scales are
// asked for before the first is written.  Rows of no slot are zeros.  31999 rows of 8 heads of 128 (330 MB)
// take 63 us, 78 % of the copy rate; a row at a time 133.
template <int FORM, int N, int ROWS>
__global__ void __launch_bounds__(256) paged_read_q8_kernel(const Q8ReadArgs a) {
    const int per_row = a.Hk * a.D / N, w = per_row < 256 ? per_row : 256, step = 256 / w;  // step: rows side by side
    const int t = threadIdx.x;
    if (t >= w * step) return;
    const float* scales = blockIdx.y ? a.p.v_scale : a.p.k_scale;
    const uint8_t* pool = blockIdx.y ? a.p.v : a.p.k;
    float* out = blockIdx.y ? a.v_out : a.k_out;
    const int64_t r0 = (int64_t)blockIdx.x * ROWS * step + t / w;
    int64_t slot[ROWS];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
        slot[k] = r0 + k * step < a.rows ? (int64_t)__ldg(a.slots + r0 + k * step) : -1;
        if (slot[k] >= a.pool_rows) slot[k] = -1;
    }
    for (int c = t % w; c < per_row; c += 256) {
        const int head = c * N / a.D;
        float s[ROWS];
        uint32_t code[ROWS];
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            s[k] = 0.f;
            code[k] = 0;
            if (slot[k] >= 0) {
                if constexpr (N == 4)
                    code[k] = __ldcs(reinterpret_cast<const uint32_t*>(pool) + slot[k] * per_row + c);
                else
                    code[k] = __ldg(pool + slot[k] * per_row + c);
                s[k] = __ldg(scales + slot[k] * a.Hk + head);
            }
        }
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            const int64_t r = r0 + k * step;
            if (r >= a.rows) break;
            if constexpr (N == 4) {
                const float4 y = slot[k] >= 0 ? q8_values4<FORM>(code[k], s[k]) : make_float4(0.f, 0.f, 0.f, 0.f);
                __stcs(reinterpret_cast<float4*>(out) + r * per_row + c, y);
            } else {
                out[r * per_row + c] = slot[k] >= 0 ? q8_value<FORM>((uint8_t)code[k]) * s[k] : 0.f;
            }
        }
    }
}

constexpr int64_t kWave = 152 * 8;  // CTAs of 256 threads that are resident at once

template <int FORM>
cudaError_t write_form(const Q8WriteArgs& a, cudaStream_t stream) {
    const uintptr_t mis = reinterpret_cast<uintptr_t>(a.k_new) | reinterpret_cast<uintptr_t>(a.v_new),
                    mis4 = reinterpret_cast<uintptr_t>(a.k_pool) | reinterpret_cast<uintptr_t>(a.v_pool);
    if (a.D % 8 == 0 && a.D <= 256 && (mis & 15u) == 0 && (mis4 & 3u) == 0) {
        int log_l = 0;
        while (8 << log_l < a.D) ++log_l;
        // Few rows: one a CTA, for the latency.
        if (a.rows <= 2 * kWave)
            paged_write_q8_fast<FORM, 1><<<(unsigned)a.rows, 256, 0, stream>>>(a, log_l);
        else
            paged_write_q8_fast<FORM, 2><<<(unsigned)((a.rows + 1) / 2), 256, 0, stream>>>(a, log_l);
    } else {
        paged_write_q8_any<FORM><<<(unsigned)a.rows, 256, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

template <int FORM, int N>
cudaError_t read_n(const Q8ReadArgs& a, cudaStream_t stream) {
    const int64_t per_row = (int64_t)a.Hk * a.D / N, step = per_row < 256 ? 256 / per_row : 1;
    if (a.rows <= kWave * step) {
        paged_read_q8_kernel<FORM, N, 1><<<dim3((unsigned)((a.rows + step - 1) / step), 2), 256, 0, stream>>>(a);
    } else {
        paged_read_q8_kernel<FORM, N, 4><<<dim3((unsigned)((a.rows + 4 * step - 1) / (4 * step)), 2), 256, 0, stream>>>(a);
    }
    return cudaGetLastError();
}
template <int FORM>
cudaError_t read_form(const Q8ReadArgs& a, cudaStream_t stream) {
    const uintptr_t mis = reinterpret_cast<uintptr_t>(a.k_out) | reinterpret_cast<uintptr_t>(a.v_out),
                    mis4 = reinterpret_cast<uintptr_t>(a.p.k) | reinterpret_cast<uintptr_t>(a.p.v);
    return a.D % 4 == 0 && (mis & 15u) == 0 && (mis4 & 3u) == 0 ? read_n<FORM, 4>(a, stream) : read_n<FORM, 1>(a, stream);
}

}  // namespace

cudaError_t launch_paged_write_q8(const Q8WriteArgs& a, cudaStream_t stream) {
    if (a.rows == 0) return cudaSuccess;
    return a.form == kFormInt8 ? write_form<kFormInt8>(a, stream) : write_form<kFormE4m3>(a, stream);
}

cudaError_t launch_paged_read_q8(const Q8ReadArgs& a, cudaStream_t stream) {
    if (a.rows == 0) return cudaSuccess;
    return a.p.form == kFormInt8 ? read_form<kFormInt8>(a, stream) : read_form<kFormE4m3>(a, stream);
}

}  // namespace vtmu
