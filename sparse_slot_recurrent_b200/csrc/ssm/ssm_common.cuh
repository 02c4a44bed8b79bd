// ssm_common.cuh -- device helpers shared by the selective scan's kernels.
#pragma once

#include "../common.cuh"
#include "ssm.h"

namespace ramnet {

// The scan's launches follow one another as programmatic dependents: a launch may start, and set itself up, while the
// one before still runs; after_before() waits for all of that one's memory, let_next() allows the next to start.
__device__ __forceinline__ void after_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <class... Args>
cudaError_t launch_dependent(void (*kern)(Args...), dim3 grid, unsigned threads, size_t smem, cudaStream_t s, Args... args)
{
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Step size of one token and head: softplus(dt + bias) (or dt + bias), clamped; what is no number stays none (fminf and
// fmaxf alone would make a limit of it).
__device__ __forceinline__ float step_size(float dt, float bias, int softplus, float lo, float hi)
{
    float v = dt + bias;
    if (softplus) v = fmaxf(v, 0.0f) + log1pf(expf(-fabsf(v)));
    return v != v ? v : fminf(fmaxf(v, lo), hi);
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

// Whether a range lies within its sequence, and its state among the workspace's (outputs by segment, else by piece).
__device__ __forceinline__ bool segment_fits(const SsmParams& p, const SegRange& r, int seg, bool outputs)
{
    const int at = outputs ? seg * p.split.sub : seg;
    return 0 <= r.first && r.first <= r.last && r.last <= p.T && at < p.split.slots() && seg < (outputs ? p.split.nseg : p.split.pieces());
}

// 2^x, rounded once: a bias of the hardware's exp2, a fraction of an ulp, would add up over the hundreds of
// chunks that a slowly decaying state remembers.  Taylor series of 2^f, |f| <= 1/2, in 64 bits (error below 1e-11).
__device__ __forceinline__ float exp2_of(double x)
{
    if (x != x) return static_cast<float>(x);
    x = fmin(fmax(x, -160.0), 160.0);
    const double n = rint(x), f = (x - n) * 0.69314718055994530942;
    double r = 1.0 / 362880;
    const double inv[9] = {1.0 / 40320, 1.0 / 5040, 1.0 / 720, 1.0 / 120, 1.0 / 24, 1.0 / 6, 0.5, 1.0, 1.0};
#pragma unroll
    for (int i = 0; i < 9; ++i) r = fma(r, f, inv[i]);
    return ldexpf(static_cast<float>(r), static_cast<int>(n));
}

__device__ __forceinline__ int seq_len(const int32_t* lengths, int b, int T)
{
    return lengths ? min(max(lengths[b], 0), T) : T;
}

}  // namespace ramnet
