// ssm_common.cuh -- device helpers shared by the selective scan's kernels.
#pragma once

#include "../common.cuh"
#include "ssm.h"

namespace ramnet {

// Step size of one token and head: softplus(dt + bias) (or dt + bias), clamped.
__device__ __forceinline__ float step_size(float dt, float bias, int softplus, float lo, float hi)
{
    float v = dt + bias;
    if (softplus) v = fmaxf(v, 0.0f) + log1pf(expf(-fabsf(v)));
    return fminf(fmaxf(v, lo), hi);
}

// Tokens [first, last) of segment `seg` of a sequence of `len` tokens.
struct SegRange {
    int first, last;
};
__device__ __forceinline__ SegRange seg_range(int len, int seg, int seg_len)
{
    const int64_t f = static_cast<int64_t>(seg) * seg_len;
    SegRange r;
    r.first = static_cast<int>(f < len ? f : len);
    r.last = static_cast<int>(f + seg_len < len ? f + seg_len : len);
    return r;
}

__device__ __forceinline__ int seq_len(const int32_t* lengths, int b, int T)
{
    return lengths ? min(max(lengths[b], 0), T) : T;
}

}  // namespace ramnet
