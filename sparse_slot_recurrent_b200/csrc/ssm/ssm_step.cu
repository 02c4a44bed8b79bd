// ssm_step.cu -- selective scan, one token per sequence against the state in HBM:
//   S <- exp(d A) S + d B (x) x,   y = C . S + D x     per (b,h), S [N,P] fp32.
//
// Bound: HBM, the state read and written once (8 N P bytes per head against 5 N P flops).  A
// block owns one (b,h): consecutive threads take consecutive 16-byte pieces of a state row, and
// the rows of a block are spread over its warps, kRows of them in flight per thread.
#include "ssm_common.cuh"

namespace ramnet {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 8;

__global__ void __launch_bounds__(kThreads) k_ssm_step(SsmStepParams p)
{
    __shared__ float bc[2][256];
    __shared__ float4 part[kThreads];
    const int h = static_cast<int>(blockIdx.x % p.H);
    const int64_t b = blockIdx.x / p.H;
    const int g = h / (p.H / p.G);
    const int N = p.N, P = p.P, lp = P / 4;  // threads per state row
    const int nrow = kThreads / lp;          // rows per pass of the block
    const int c = threadIdx.x % lp, r0 = threadIdx.x / lp;
    float* S = p.S + (b * p.H + h) * static_cast<int64_t>(N) * P;

    for (int i = threadIdx.x; i < N; i += kThreads) {
        bc[0][i] = load_in(p.Bm, static_cast<size_t>(b * p.bs.b + g * p.bs.h + i), p.in_bf16);
        bc[1][i] = load_in(p.Cm, static_cast<size_t>(b * p.cs.b + g * p.cs.h + i), p.in_bf16);
    }
    const float d = step_size(load_in(p.dt, static_cast<size_t>(b * p.dts.b + h * p.dts.h), p.in_bf16),
                              p.dt_bias ? p.dt_bias[h] : 0.0f, p.softplus, p.dt_min, p.dt_max);
    const float a = expf(d * p.A[h]);
    float x[4], u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[j] = load_in(p.x, static_cast<size_t>(b * p.xs.b + h * p.xs.h + c * 4 + j), p.in_bf16);
        u[j] = d * x[j];
    }
    __syncthreads();
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int n0 = r0; n0 < N; n0 += nrow * kRows) {
        float4 s[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int n = n0 + k * nrow;
            if (n < N) s[k] = *reinterpret_cast<const float4*>(S + static_cast<int64_t>(n) * P + c * 4);
        }
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int n = n0 + k * nrow;
            if (n < N) {
                const float bn = bc[0][n], cn = bc[1][n];
                s[k].x = fmaf(bn, u[0], a * s[k].x);
                s[k].y = fmaf(bn, u[1], a * s[k].y);
                s[k].z = fmaf(bn, u[2], a * s[k].z);
                s[k].w = fmaf(bn, u[3], a * s[k].w);
                acc.x = fmaf(cn, s[k].x, acc.x);
                acc.y = fmaf(cn, s[k].y, acc.y);
                acc.z = fmaf(cn, s[k].z, acc.z);
                acc.w = fmaf(cn, s[k].w, acc.w);
                *reinterpret_cast<float4*>(S + static_cast<int64_t>(n) * P + c * 4) = s[k];
            }
        }
    }
    part[threadIdx.x] = acc;
    __syncthreads();
    if (threadIdx.x < P) {
        const float* f = reinterpret_cast<const float*>(part);
        float y = 0.0f;
        for (int r = 0; r < nrow; ++r) y += f[r * P + threadIdx.x];
        const float xv = load_in(p.x, static_cast<size_t>(b * p.xs.b + h * p.xs.h + threadIdx.x), p.in_bf16);
        if (p.D) y = fmaf(p.D[h], xv, y);
        store_out(p.y, static_cast<size_t>((b * p.H + h) * P + threadIdx.x), y, p.out_bf16);
    }
}

}  // namespace

cudaError_t launch_ssm_step(const SsmStepParams& p, cudaStream_t s)
{
    k_ssm_step<<<static_cast<unsigned>(static_cast<int64_t>(p.B) * p.H), kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace ramnet
