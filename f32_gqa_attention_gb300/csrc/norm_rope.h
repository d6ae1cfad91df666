// norm_rope.h -- launcher of the fused norm and rotation of queries and keys.
#pragma once

#include <cuda_runtime.h>

#include "attn_desc.h"

namespace vtmu {

constexpr int kMaxAxes = 4;

struct NormRopeArgs {
    const float* q;
    const float* k;
    const float* qw;           // nullptr: weights of one (without weight_offset)
    const float* kw;
    float* q_out;
    float* k_out;
    const int32_t* positions;  // [axes, T]
    int64_t T;
    int32_t H, Hk, D, axes, norm;
    float eps, weight_offset, inv_d;  // inv_d: 1 / D
    int32_t half, interleaved;    // as RopeDev's
    float attn;
    uint8_t axis[kRopeMaxPairs];  // of each pair
    uint64_t turn[kRopeMaxPairs]; // inv_freq / (2 pi) less its whole part, times 2^64
};
cudaError_t launch_norm_rope(const NormRopeArgs& a, cudaStream_t stream);

}  // namespace vtmu
