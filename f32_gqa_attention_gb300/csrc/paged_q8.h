// paged_q8.h -- the 8-bit paged cache: its formats and the launchers of the
// kernels that write it, read it back and attend over it.
#pragma once

#include "paged_kernels.h"

namespace vtmu {

// An element is code x scale, one scale per pool row and KV head (the values
// are vtmu_kv_format's).
enum KvForm : int32_t { kFormF32 = 0, kFormInt8 = 1, kFormE4m3 = 2 };

// The pools of one call: codes [pool rows, Hk * D], scales [pool rows, Hk].
struct Q8Pools {
    const uint8_t* k;
    const uint8_t* v;
    const float* k_scale;
    const float* v_scale;
    int32_t form;
};

struct Q8WriteArgs {
    uint8_t* k_pool;
    uint8_t* v_pool;
    float* k_scale;
    float* v_scale;
    const float* k_new;
    const float* v_new;
    const int32_t* slots;
    int64_t pool_rows, rows;
    int32_t Hk, D, form;
};
cudaError_t launch_paged_write_q8(const Q8WriteArgs& a, cudaStream_t stream);

struct Q8ReadArgs {
    Q8Pools p;
    const int32_t* slots;
    float* k_out;
    float* v_out;
    int64_t pool_rows, rows;
    int32_t Hk, D;
};
cudaError_t launch_paged_read_q8(const Q8ReadArgs& a, cudaStream_t stream);

// a.k_pool and a.v_pool are not read.
cudaError_t launch_paged_q8_ffma(const PagedDesc& a, const Q8Pools& p, cudaStream_t stream);
// Warp-wide f16 products: headDim 64 or 128; q, out, pools and new rows 16-byte aligned.
bool paged_q8_mma_supported(const PagedDesc& a);
size_t paged_q8_mma_workspace(const PagedDesc& a);
cudaError_t launch_paged_q8_mma(const PagedDesc& a, const Q8Pools& p, int num_sms, void* workspace, cudaStream_t stream);
// tcgen05 products of 128-row blocks, for the same calls.
size_t paged_q8_tc_workspace(const PagedDesc& a);
cudaError_t launch_paged_q8_tc(const PagedDesc& a, const Q8Pools& p, int num_sms, void* workspace, cudaStream_t stream);
unsigned int paged_q8_tc_take_device_error();
// Which of the two: virtual rows (rows of a request x heads of a group) above kQ8FewRows take the
// blocks of 128; its boxes of 64-byte rows want pages of an even size, and the box behind the
// pool, which stands for bad pages, coordinates below 2^31.
// 32 requests of 517 to 8111 rows, 4 heads a group: 16 virtual rows take 132 us with few rows' kernel,
// 20 to 32 take 218 to 230 there and 193 to 202 in blocks, 64 take 408 and 210 (8 heads a group: 129 us at
// 16, 196 at 24, 208 at 64).
constexpr int kQ8FewRows = 16;
inline bool paged_q8_few_rows(const PagedDesc& a) {
    return (int64_t)a.max_rows * a.G <= kQ8FewRows || (a.D == 64 && a.page_size % 2 != 0) ||
           a.pages * a.page_size >= ((int64_t)1 << 31) - 256;
}
// The drafted rows' part of every row: its output to a.out, its maximum and sum to ml [rows][H].
cudaError_t launch_paged_q8_draft(const PagedDesc& a, float2* ml, cudaStream_t stream);
unsigned int paged_q8_take_device_error();

}  // namespace vtmu
