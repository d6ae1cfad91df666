// paged.cuh -- what the paged kernels share: the packed rows and lengths of a
// request as the device arrays give them, brought into range.
#pragma once

#include <cstdint>

#include "paged_kernels.h"

namespace vtmu {

__device__ __forceinline__ int64_t clamp64(int64_t x, int64_t lo, int64_t hi) { return x < lo ? lo : x > hi ? hi : x; }

// The rows of all requests, [first, last): cu_rows[0] .. cu_rows[requests] clamped to the
// buffers.  Rows outside belong to none, whatever lies between these two.
struct RowRange {
    int64_t first, last;
};
__device__ __forceinline__ RowRange rows_of_all(const int32_t* cu_rows, int requests, int64_t rows) {
    return {clamp64(__ldg(cu_rows), 0, rows), clamp64(__ldg(cu_rows + requests), 0, rows)};
}

// Packed rows [row0, row0 + n) of request b: its pair of cu_rows inside that range, a
// decreasing pair holds none.
struct PackedRows {
    int64_t row0;
    int64_t n;
};
__device__ __forceinline__ PackedRows packed_rows(const int32_t* cu_rows, int b, const RowRange& all, int64_t rows) {
    PackedRows r;
    r.row0 = max(clamp64(__ldg(cu_rows + b), 0, rows), all.first);
    r.n = max(min((int64_t)__ldg(cu_rows + b + 1), all.last) - r.row0, (int64_t)0);
    return r;
}
__device__ __forceinline__ PackedRows packed_rows(const int32_t* cu_rows, int b, int requests, int64_t rows) {
    return packed_rows(cu_rows, b, rows_of_all(cu_rows, requests, rows), rows);
}

}  // namespace vtmu
