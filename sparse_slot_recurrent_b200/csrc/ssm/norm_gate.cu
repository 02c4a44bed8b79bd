// norm_gate.cu -- RMSNorm of rows in groups of channels, with a SiLU output gate before or
// behind the norm:
//   gate first:  u = x silu(z),  y = u / sqrt(mean_group(u^2) + eps) * w
//   norm first:  y = x / sqrt(mean_group(x^2) + eps) * w * silu(z)
// without z the gate is left out.  Sums in fp32, in a fixed order.
//
// Bound: HBM, x and z read once and y written once.  A block (or one warp, for short groups)
// owns one group of one row and keeps it in registers between the sum and the scaling.
#include "../common.cuh"
#include "ssm.h"

namespace ramnet {
namespace {

template <bool BF, int V>
__device__ __forceinline__ void load_vec(const void* base, int64_t i, float (&v)[V])
{
    if constexpr (V == 1) {
        v[0] = load_in(base, static_cast<size_t>(i), BF);
    } else if constexpr (BF) {
        const uint4 r = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(base) + i);
        const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(u[j] << 16);
            v[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
        }
    } else {
        load_row_g<V>(reinterpret_cast<const float*>(base) + i, v);
    }
}

template <bool BF, int V>
__device__ __forceinline__ void store_vec(void* base, int64_t i, const float (&v)[V])
{
    if constexpr (V == 1) {
        store_out(base, static_cast<size_t>(i), v[0], BF);
    } else if constexpr (BF) {
        uint32_t u[V / 2];
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
            u[j] = *reinterpret_cast<const uint32_t*>(&b);
        }
        uint32_t* p = reinterpret_cast<uint32_t*>(reinterpret_cast<__nv_bfloat16*>(base) + i);
        if constexpr (V == 8) *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
        else *reinterpret_cast<uint2*>(p) = make_uint2(u[0], u[1]);
    } else {
        store_row_g<V>(reinterpret_cast<float*>(base) + i, v);
    }
}

// as in the convolution: the hardware's exp2 and reciprocal where the result is bf16
template <bool FAST>
__device__ __forceinline__ float silu(float v)
{
    if constexpr (FAST) return __fdividef(v, 1.0f + __expf(-v));
    else return v / (1.0f + expf(-v));
}

constexpr int kThreads = 256;

// One group of one row per block; each thread keeps up to NV vectors of V channels, a longer
// group is read a second time (from L2) for the scaling.
template <int V, int NV, bool IB, bool OB>
__global__ void __launch_bounds__(kThreads) k_norm_gate(NormParams p)
{
    __shared__ float part[kThreads / 32];
    const int64_t row = blockIdx.x / p.groups;
    const int g = static_cast<int>(blockIdx.x % p.groups);
    const int width = p.D / p.groups;
    const int64_t xo = row * p.sx + static_cast<int64_t>(g) * width;
    const int64_t zo = row * p.sz + static_cast<int64_t>(g) * width;
    const int nv = width / V;
    float u[NV][V], gate[NV][V];

    auto fetch = [&](int i, float (&uu)[V], float (&gg)[V]) {
        load_vec<IB, V>(p.x, xo + static_cast<int64_t>(i) * V, uu);
        if (p.z) {
            load_vec<IB, V>(p.z, zo + static_cast<int64_t>(i) * V, gg);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                gg[v] = silu<OB>(gg[v]);
                if (p.gate_first) uu[v] *= gg[v];
            }
        }
    };
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int i = threadIdx.x + k * kThreads;
        if (i < nv) {
            fetch(i, u[k], gate[k]);
#pragma unroll
            for (int v = 0; v < V; ++v) sum = fmaf(u[k][v], u[k][v], sum);
        }
    }
    for (int i = threadIdx.x + NV * kThreads; i < nv; i += kThreads) {
        float uu[V], gg[V];
        fetch(i, uu, gg);
#pragma unroll
        for (int v = 0; v < V; ++v) sum = fmaf(uu[v], uu[v], sum);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
    __syncthreads();
    sum = part[0];
#pragma unroll
    for (int i = 1; i < kThreads / 32; ++i) sum += part[i];
    const float inv = 1.0f / sqrtf(sum / static_cast<float>(width) + p.eps);

    auto finish = [&](int i, float (&uu)[V], float (&gg)[V]) {
        const int d = g * width + i * V;
        float wv[V];
        if (p.w) load_vec<false, V == 8 ? 8 : V>(p.w, d, wv);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            uu[v] *= inv;
            if (p.w) uu[v] *= wv[v];
            if (p.z && !p.gate_first) uu[v] *= gg[v];
        }
        store_vec<OB, V>(p.y, row * p.D + d, uu);
    };
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int i = threadIdx.x + k * kThreads;
        if (i < nv) finish(i, u[k], gate[k]);
    }
    for (int i = threadIdx.x + NV * kThreads; i < nv; i += kThreads) {
        float uu[V], gg[V];
        fetch(i, uu, gg);
        finish(i, uu, gg);
    }
}

bool al(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <int V, int NV, bool IB>
cudaError_t go(const NormParams& p, cudaStream_t s)
{
    const unsigned grid = static_cast<unsigned>(p.R * p.groups);
    if (p.out_bf16) k_norm_gate<V, NV, IB, true><<<grid, kThreads, 0, s>>>(p);
    else k_norm_gate<V, NV, IB, false><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_gate(const NormParams& p, cudaStream_t s)
{
    const int v = p.in_bf16 ? 8 : 4;
    const int width = p.D / p.groups;
    const bool vec = width % v == 0 && p.sx % v == 0 && al(p.x, 16) && (!p.z || (p.sz % v == 0 && al(p.z, 16)));
    if (p.in_bf16) return vec ? go<8, 2, true>(p, s) : go<1, 4, true>(p, s);
    return vec ? go<4, 2, false>(p, s) : go<1, 4, false>(p, s);
}

}  // namespace ramnet
