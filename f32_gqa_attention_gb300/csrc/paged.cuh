// paged.cuh -- what the paged kernels share: the packed rows and lengths of a
// request as the device arrays give them, brought into range.
#pragma once

#include <cstdint>

#include "paged_kernels.h"

namespace vtmu {

__device__ __forceinline__ int64_t clamp64(int64_t x, int64_t lo, int64_t hi) { return x < lo ? lo : x > hi ? hi : x; }

// Packed rows [row0, row0 + n) of request b: cu_rows clamped to the buffers,
// a decreasing pair holds none.
struct PackedRows {
    int64_t row0;
    int64_t n;
};
__device__ __forceinline__ PackedRows packed_rows(const int32_t* cu_rows, int b, int64_t rows) {
    PackedRows r;
    r.row0 = clamp64(__ldg(cu_rows + b), 0, rows);
    r.n = clamp64(__ldg(cu_rows + b + 1), r.row0, rows) - r.row0;
    return r;
}

}  // namespace vtmu
