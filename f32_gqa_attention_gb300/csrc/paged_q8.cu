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

// Lanes that share a unit in the fast kernels: D / 8, rounded up to a power of two.
int lanes_of(int D) {
    int l = 1;
    while (8 * l < D) l *= 2;
    return l;
}

// ---- write -----------------------------------------------------------------------
// Memory-bound: 5 bytes an element and two reductions of log2 L shuffles.  FAST: L
// lanes hold a unit, eight elements each as two 16-byte loads D / 2 apart (so that each
// load of the group is one run of D / 2 elements); any D to 256 that is a multiple of 8.
// Otherwise a warp walks a unit twice.
template <int FORM, bool FAST>
__global__ void __launch_bounds__(256) paged_write_q8_kernel(const Q8WriteArgs a, int L) {
    const int group = FAST ? L : 32;
    const int64_t unit = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / group;
    const int lane = threadIdx.x & (group - 1), per_row = 2 * a.Hk, D = a.D;
    // Every lane of a warp takes part in the shuffles, also behind the last unit.
    const int64_t r = unit / per_row;
    const int part = (int)(unit - r * per_row), head = part % a.Hk;
    const bool values = part >= a.Hk;
    int64_t slot = r < a.rows ? (int64_t)__ldg(a.slots + r) : -1;
    if (slot >= a.pool_rows) slot = -1;
    const float* x = (values ? a.v_new : a.k_new) + (r * a.Hk + head) * D;
    uint8_t* to = (values ? a.v_pool : a.k_pool) + (slot * a.Hk + head) * D;
    float top = 0.f;
    if constexpr (FAST) {
        float4 u = make_float4(0.f, 0.f, 0.f, 0.f), v = u;
        const bool live = slot >= 0 && 8 * lane < D;
        if (live) {
            u = __ldcs(reinterpret_cast<const float4*>(x) + lane);
            v = __ldcs(reinterpret_cast<const float4*>(x + D / 2) + lane);
        }
        top = q8_abs_top(q8_abs_top(0.f, u), v);
        for (int off = L / 2; off > 0; off >>= 1) top = q8_nan_max(top, __shfl_xor_sync(0xffffffffu, top, off));
        const Q8Scale s = q8_scale<FORM>(top);
        if (live) {
            reinterpret_cast<uint32_t*>(to)[lane] = q8_codes4<FORM>(u, s);
            reinterpret_cast<uint32_t*>(to + D / 2)[lane] = q8_codes4<FORM>(v, s);
        }
        if (slot >= 0 && lane == 0) (values ? a.v_scale : a.k_scale)[slot * a.Hk + head] = s.scale;
    } else {
        if (slot >= 0)
            for (int d = lane; d < D; d += 32) top = q8_nan_max(top, fabsf(__ldg(x + d)));
        for (int off = 16; off > 0; off >>= 1) top = q8_nan_max(top, __shfl_xor_sync(0xffffffffu, top, off));
        const Q8Scale s = q8_scale<FORM>(top);
        if (slot < 0) return;
        for (int d = lane; d < D; d += 32) to[d] = q8_code<FORM>(__ldg(x + d), s);
        if (lane == 0) (values ? a.v_scale : a.k_scale)[slot * a.Hk + head] = s.scale;
    }
}

// ---- read ------------------------------------------------------------------------
// Memory-bound, four fifths of it the f32 rows written: a thread takes four codes (VEC:
// D a multiple of four, aligned buffers) or one.  Rows of no slot are zeros.
template <int FORM, bool VEC>
__global__ void __launch_bounds__(256) paged_read_q8_kernel(const Q8ReadArgs a) {
    constexpr int N = VEC ? 4 : 1;
    const int64_t per_row = (int64_t)a.Hk * a.D / N;
    const float* scales = blockIdx.y ? a.p.v_scale : a.p.k_scale;
    const uint8_t* pool = blockIdx.y ? a.p.v : a.p.k;
    float* out = blockIdx.y ? a.v_out : a.k_out;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const int64_t slot = __ldg(a.slots + r);
        const bool live = slot >= 0 && slot < a.pool_rows;
        for (int64_t i = threadIdx.x; i < per_row; i += blockDim.x) {
            const int head = (int)(i * N / a.D);
            const float s = live ? __ldg(scales + slot * a.Hk + head) : 0.f;
            if constexpr (VEC) {
                float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
                if (live) y = q8_values4<FORM>(__ldg(reinterpret_cast<const uint32_t*>(pool) + slot * per_row + i), s);
                __stcs(reinterpret_cast<float4*>(out) + r * per_row + i, y);
            } else {
                out[r * per_row + i] = live ? q8_value<FORM>(__ldg(pool + slot * per_row + i)) * s : 0.f;
            }
        }
    }
}

template <int FORM>
cudaError_t write_form(const Q8WriteArgs& a, cudaStream_t stream) {
    const uintptr_t mis = reinterpret_cast<uintptr_t>(a.k_new) | reinterpret_cast<uintptr_t>(a.v_new),
                    mis4 = reinterpret_cast<uintptr_t>(a.k_pool) | reinterpret_cast<uintptr_t>(a.v_pool);
    const bool fast = a.D % 8 == 0 && a.D <= 256 && (mis & 15u) == 0 && (mis4 & 3u) == 0;
    const int L = fast ? lanes_of(a.D) : 32;
    const int64_t blocks = (a.rows * 2 * a.Hk * L + 255) / 256;
    if (fast)
        paged_write_q8_kernel<FORM, true><<<(unsigned)blocks, 256, 0, stream>>>(a, L);
    else
        paged_write_q8_kernel<FORM, false><<<(unsigned)blocks, 256, 0, stream>>>(a, L);
    return cudaGetLastError();
}

template <int FORM>
cudaError_t read_form(const Q8ReadArgs& a, cudaStream_t stream) {
    const uintptr_t mis = reinterpret_cast<uintptr_t>(a.k_out) | reinterpret_cast<uintptr_t>(a.v_out),
                    mis4 = reinterpret_cast<uintptr_t>(a.p.k) | reinterpret_cast<uintptr_t>(a.p.v);
    const bool vec = a.D % 4 == 0 && (mis & 15u) == 0 && (mis4 & 3u) == 0;
    const dim3 grid((unsigned)(a.rows < (1 << 20) ? a.rows : (1 << 20)), 2);
    if (vec)
        paged_read_q8_kernel<FORM, true><<<grid, 256, 0, stream>>>(a);
    else
        paged_read_q8_kernel<FORM, false><<<grid, 256, 0, stream>>>(a);
    return cudaGetLastError();
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
