// conv.cu -- short causal convolution along the sequence, one filter per channel, for prompts
// (k_conv) and for single tokens (k_conv_step):
//   y[t,c] = act(bias[c] + sum_k w[c,k] x[t-W+1+k,c]),  act = SiLU or none,
// with the W-1 inputs before the first token taken from a carried state.  Sums in fp32.
//
// Bound: HBM, one read of x and one write of y (2 W flops per element).  A thread owns V
// neighbouring channels (16 bytes where addresses allow) over a run of tokens and slides a
// window of W-1 inputs in registers, so each input is read once but for W-1 rows per run.
#include "../common.cuh"
#include "ssm.h"

namespace ramnet {
namespace {

constexpr int kConvRun = 32;  // tokens per thread

template <bool BF>
using InT = typename std::conditional<BF, __nv_bfloat16, float>::type;

// V elements at p (V * element size aligned) as fp32, and back.
template <bool BF, int V>
__device__ __forceinline__ void load_vec(const void* base, int64_t i, float (&v)[V])
{
    const InT<BF>* p = reinterpret_cast<const InT<BF>*>(base) + i;
    if constexpr (V == 1) {
        if constexpr (BF) v[0] = __bfloat162float(p[0]);
        else v[0] = p[0];
    } else if constexpr (BF) {
        static_assert(V == 8, "16 bytes");
        const uint4 r = *reinterpret_cast<const uint4*>(p);
        const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(u[j] << 16);
            v[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
        }
    } else {
        static_assert(V == 4, "16 bytes");
        const float4 r = *reinterpret_cast<const float4*>(p);
        v[0] = r.x;
        v[1] = r.y;
        v[2] = r.z;
        v[3] = r.w;
    }
}

template <bool BF, int V>
__device__ __forceinline__ void store_vec(void* base, int64_t i, const float (&v)[V])
{
    InT<BF>* p = reinterpret_cast<InT<BF>*>(base) + i;
    if constexpr (V == 1) {
        if constexpr (BF) p[0] = __float2bfloat16_rn(v[0]);
        else p[0] = v[0];
    } else if constexpr (BF) {
        uint32_t u[V / 2];
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
            u[j] = *reinterpret_cast<const uint32_t*>(&b);
        }
        if constexpr (V == 8) *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
        else *reinterpret_cast<uint2*>(p) = make_uint2(u[0], u[1]);
    } else {
#pragma unroll
        for (int j = 0; j < V; j += 4) *reinterpret_cast<float4*>(p + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
    }
}

// SiLU.  For a bf16 result the hardware's exp2 and reciprocal are enough (their relative error
// of about 2^-21 is far below bf16's 2^-9); an fp32 result takes the accurate forms.
template <bool FAST>
__device__ __forceinline__ float silu(float v)
{
    if constexpr (FAST) return __fdividef(v, 1.0f + __expf(-v));
    else return v / (1.0f + expf(-v));
}

template <int W, int V, bool IB, bool OB>
__global__ void __launch_bounds__(128) k_conv(ConvParams p, int ncv, int64_t work)
{
    const int64_t id = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
    if (id >= work) return;
    const int cv = static_cast<int>(id % ncv);
    const int64_t run = id / ncv;
    const int runs = (p.T + kConvRun - 1) / kConvRun;
    const int b = static_cast<int>(run / runs);
    const int t0 = static_cast<int>(run % runs) * kConvRun;
    const int c = cv * V;
    int len = p.T;
    if (p.lengths) len = min(max(p.lengths[b], 0), p.T);
    if (t0 >= len && t0 > 0) return;
    const int t1 = min(t0 + kConvRun, len);

    float wt[V][W], bias[V], win[W][V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int k = 0; k < W; ++k) wt[v][k] = p.w[static_cast<int64_t>(c + v) * W + k];
        bias[v] = p.bias ? p.bias[c + v] : 0.0f;
    }
    const int64_t xb = static_cast<int64_t>(b) * p.sb + c;
    const int64_t sbase = static_cast<int64_t>(b) * (W - 1) * p.C + c;
    float old[W - 1][V];  // the carried state, kept by the first run (it also writes state_out)
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        const int t = t0 - (W - 1) + k;
        if (t >= 0) {
            load_vec<IB, V>(p.x, xb + static_cast<int64_t>(t) * p.st, win[k]);
        } else if (p.state_in) {
            load_vec<IB, V>(p.state_in, sbase + static_cast<int64_t>(t + W - 1) * p.C, win[k]);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) win[k][v] = 0.0f;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) old[k][v] = win[k][v];
    }
#pragma unroll 4
    for (int t = t0; t < t1; ++t) {
        load_vec<IB, V>(p.x, xb + static_cast<int64_t>(t) * p.st, win[W - 1]);
        float acc[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            acc[v] = bias[v];
#pragma unroll
            for (int k = 0; k < W; ++k) acc[v] = fmaf(wt[v][k], win[k][v], acc[v]);
            if (p.silu) acc[v] = silu<OB>(acc[v]);
        }
        store_vec<OB, V>(p.y, (static_cast<int64_t>(b) * p.T + t) * p.C + c, acc);
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) win[k][v] = win[k + 1][v];
    }
    // The last W-1 inputs: from x, or from the old state where the sequence is shorter.  Only
    // the first run touches the state, after it has read all of it, so it may be in place.
    if (t0 == 0 && p.state_out) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            const int t = len - (W - 1) + k;
            float v8[V];
            if (t >= 0) {
                load_vec<IB, V>(p.x, xb + static_cast<int64_t>(t) * p.st, v8);
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) v8[v] = 0.0f;
#pragma unroll
                for (int q = 0; q < W - 1; ++q)
                    if (q == t + W - 1) {
#pragma unroll
                        for (int v = 0; v < V; ++v) v8[v] = old[q][v];
                    }
            }
            store_vec<IB, V>(p.state_out, sbase + static_cast<int64_t>(k) * p.C, v8);
        }
    }
}

template <int W, int V, bool IB, bool OB>
__global__ void __launch_bounds__(128) k_conv_step(ConvStepParams p, int ncv, int64_t work)
{
    const int64_t id = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
    if (id >= work) return;
    const int c = static_cast<int>(id % ncv) * V;
    const int64_t b = id / ncv;
    const int64_t sbase = b * (W - 1) * p.C + c;
    float win[W][V], acc[V];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) load_vec<IB, V>(p.state, sbase + static_cast<int64_t>(k) * p.C, win[k]);
    load_vec<IB, V>(p.x, b * p.sb + c, win[W - 1]);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        acc[v] = p.bias ? p.bias[c + v] : 0.0f;
#pragma unroll
        for (int k = 0; k < W; ++k) acc[v] = fmaf(p.w[static_cast<int64_t>(c + v) * W + k], win[k][v], acc[v]);
        if (p.silu) acc[v] = silu<OB>(acc[v]);
    }
    store_vec<OB, V>(p.y, b * p.C + c, acc);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) store_vec<IB, V>(p.state, sbase + static_cast<int64_t>(k) * p.C, win[k + 1]);
}

bool al(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <int W, int V, bool IB, bool OB>
cudaError_t go(const ConvParams& p, cudaStream_t s)
{
    const int ncv = p.C / V;
    const int64_t work = static_cast<int64_t>(ncv) * p.B * ((p.T + kConvRun - 1) / kConvRun);
    k_conv<W, V, IB, OB><<<static_cast<unsigned>((work + 127) / 128), 128, 0, s>>>(p, ncv, work);
    return cudaGetLastError();
}

template <int W, int V, bool IB, bool OB>
cudaError_t go(const ConvStepParams& p, cudaStream_t s)
{
    const int ncv = p.C / V;
    const int64_t work = static_cast<int64_t>(ncv) * p.B;
    k_conv_step<W, V, IB, OB><<<static_cast<unsigned>((work + 127) / 128), 128, 0, s>>>(p, ncv, work);
    return cudaGetLastError();
}

template <int W, bool IB, class P>
cudaError_t pick_v(const P& p, bool vec, cudaStream_t s)
{
    constexpr int V = IB ? 8 : 4;
    if (vec) return p.out_bf16 ? go<W, V, IB, true>(p, s) : go<W, V, IB, false>(p, s);
    return p.out_bf16 ? go<W, 1, IB, true>(p, s) : go<W, 1, IB, false>(p, s);
}

template <int W, class P>
cudaError_t pick_in(const P& p, bool vec, cudaStream_t s)
{
    return p.in_bf16 ? pick_v<W, true>(p, vec, s) : pick_v<W, false>(p, vec, s);
}

template <class P>
cudaError_t pick_w(const P& p, bool vec, cudaStream_t s)
{
    switch (p.W) {
        case 2: return pick_in<2>(p, vec, s);
        case 3: return pick_in<3>(p, vec, s);
        case 4: return pick_in<4>(p, vec, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_conv(const ConvParams& p, cudaStream_t s)
{
    // 16-byte accesses need every row of x, y and the states to start on a 16-byte boundary
    const int v = p.in_bf16 ? 8 : 4;
    const bool vec = p.C % v == 0 && p.sb % v == 0 && p.st % v == 0 && al(p.x, 16);
    return pick_w(p, vec, s);
}

cudaError_t launch_conv_step(const ConvStepParams& p, cudaStream_t s)
{
    const int v = p.in_bf16 ? 8 : 4;
    const bool vec = p.C % v == 0 && p.sb % v == 0 && al(p.x, 16);
    return pick_w(p, vec, s);
}

}  // namespace ramnet
