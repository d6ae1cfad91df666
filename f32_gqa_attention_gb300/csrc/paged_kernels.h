// paged_kernels.h -- launchers of the paged-cache kernels: page maps, drafted
// trees, rope at positions, paged writes and paged attention.  Beside kernels.h, so
// that the other kernels' sources, which their profiles record, do not change with it.
#pragma once

#include "kernels.h"

namespace vtmu {

struct PageMapArgs {
    const int32_t* lens;
    const int32_t* cu_rows;
    const uint64_t* accept;     // nullptr: every packed row is added
    int32_t* block_table;
    const int32_t* free_pages;
    const int32_t* n_free;
    int32_t* slots;
    int32_t* positions;         // nullptr: not wanted
    int32_t* new_lens;
    int32_t* n_free_out;
    int64_t free_capacity, rows;
    int32_t requests, page_size, max_pages;
};
cudaError_t launch_page_map(const PageMapArgs& a, cudaStream_t stream);
cudaError_t launch_tree_plan(const int32_t* parents, const int32_t* cu_rows, const int32_t* lens, uint64_t* masks,
                             int32_t* positions, int32_t requests, int64_t rows, cudaStream_t stream);
// out = rope(x), row t at positions[t]; rows at negative positions are left as they were.
cudaError_t launch_rope_at(const float* x, float* out, int64_t T, int H, int D, const int32_t* positions,
                           const RopeDev& r, cudaStream_t stream);
cudaError_t launch_paged_write(float* k_pool, float* v_pool, int64_t pool_rows, int64_t k_width, int64_t v_width,
                               const float* k_new, const float* v_new, const int32_t* slots, int64_t rows,
                               cudaStream_t stream);

constexpr int kPagedMaxRequests = 1024;
constexpr int kTreeMaxRows = 64;
struct PagedDesc {
    const float* q;
    const float* k_pool;
    const float* v_pool;
    const int32_t* block_table;
    const int32_t* lens;
    const int32_t* cu_rows;
    const float* k_new;       // tree: the drafted rows
    const float* v_new;
    const uint64_t* masks;
    const int32_t* positions;
    float* out;
    int64_t rows, pages;
    int64_t window, sinks;    // sinks: 0 without a window
    int32_t B, H, Hk, G, D;
    int32_t page_size, max_pages, max_rows, tree;
    int32_t softcap_on;
    // As in AttnDesc: without softcap x2 = dot * qk_mul, with it x2 =
    // cap_log2 * tanh(dot * qk_mul).
    float qk_mul, cap_log2;
};
cudaError_t launch_paged_ffma(const PagedDesc& a, cudaStream_t stream);
// The tensor-core kernel: headDim 64 or 128, pages of a multiple of 64 or of 8,
// 16 or 32 rows; 16-byte aligned pools and new rows are checked at launch.
constexpr int kPagedMaxCtas = 160;  // the workspace holds two partials for each
bool paged_tc_supported(const PagedDesc& a);
size_t paged_tc_workspace(const PagedDesc& a);
cudaError_t launch_paged_tc(const PagedDesc& a, int num_sms, void* workspace, cudaStream_t stream);
unsigned int paged_take_device_error();

}  // namespace vtmu
