// paged_q8_mma.cuh -- f16 fragments of the 8-bit cache's attention: codes to
// halves, f32 to pairs of halves, and the warp-wide product (PTX ISA, mma.m16n8k16).
#pragma once

#include <cstdint>

#include "attn_common.cuh"
#include "paged_q8.cuh"

namespace vtmu {

// One of the arrivals that `bar` counts, once this thread's earlier cp.async have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];\n" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;\n" ::: "memory"); }

// The power of two that brings a row's largest |element| to [2^bits, 2^(bits + 1)), or, where that is
// above 2^126, 2^126: it and its inverse are normal numbers.  With bits 8 and 13 that leaves normal elements
// at 1 and more, whose 22 bits f16 pairs hold (they end at 2^-24).
__device__ __forceinline__ float mma_row_scale(float top, int bits) {
    int e = (int)(__float_as_uint(top) >> 23) - 127;
    e = e < bits - 126 ? bits - 126 : e > 127 ? 127 : e;
    return __uint_as_float((uint32_t)(bits - e + 127) << 23);
}

// A pair of f32 as pairs of halves hi + lo.
__device__ __forceinline__ void mma_split(float x, float y, uint32_t& hi, uint32_t& lo) {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = *reinterpret_cast<const uint32_t*>(&l);
}

// Signed bytes as halves: 1024 + (code + 128) is the half with the byte as its last
// bits; 1152 comes off exactly.
__device__ __forceinline__ uint32_t int8_off(uint32_t h) {
    const uint32_t k = 0x64806480u;
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&h), *reinterpret_cast<const __half2*>(&k));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
    return r;
}
// Four codes as halves: bytes 0, 1 and bytes 2, 3.
template <int FORM>
__device__ __forceinline__ void q8_halves(uint32_t w, uint32_t& h01, uint32_t& h23) {
    if constexpr (FORM == kFormInt8) {
        const uint32_t u = w ^ 0x80808080u;
        h01 = int8_off(__byte_perm(u, 0x64646464u, 0x4140));
        h23 = int8_off(__byte_perm(u, 0x64646464u, 0x4342));
    } else {
        h01 = e4m3_pair(w);
        h23 = e4m3_pair(w >> 16);
    }
}
// Four codes each of two rows: byte i of both, as a pair.
template <int FORM>
__device__ __forceinline__ void q8_halves2(uint32_t wa, uint32_t wb, uint32_t& h0, uint32_t& h1, uint32_t& h2, uint32_t& h3) {
    q8_halves<FORM>(__byte_perm(wa, wb, 0x5140), h0, h1);
    q8_halves<FORM>(__byte_perm(wa, wb, 0x7362), h2, h3);
}

// An 8 x 8 block of halves, row lane / 4, columns 2 (lane % 4) and the next: its transpose.
__device__ __forceinline__ uint32_t mma_transpose(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// c += a b, 16 x 16 by 16 x 8, f32 sums.
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

}  // namespace vtmu
