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
    float eps, weight_offset;
    uint8_t axis[kRopeMaxPairs];  // of each pair
    RopeDev r;
};
cudaError_t launch_norm_rope(const NormRopeArgs& a, cudaStream_t stream);

}  // namespace vtmu
