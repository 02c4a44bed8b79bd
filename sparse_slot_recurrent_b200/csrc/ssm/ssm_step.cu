// ssm_step.cu -- selective scan, one token per sequence against the state in HBM:
//   S <- exp(d A) S + d B (x) x,   y = C . S + D x     per (b,h), S [N,P] fp32.
//
// Bound: HBM, the state read and written once (8 N P bytes per head against 5 N P flops): 85 us for
// 256 sequences x 16 heads of 128 x 128 values, 96% of the copy bandwidth.  A block owns one (b,h):
// consecutive threads take consecutive 16-byte pieces of a state row, rows are spread over its warps,
// kRows pieces in flight per thread, asked for before the token's operands are worked out.
// The decay is rounded once from 64 bits, as in the prompt form: a bias of expf would add up over the
// thousands of tokens that a slowly decaying state remembers.
#include "ssm_common.cuh"

namespace ramnet {
namespace {

constexpr int kRows = 8;

template <int TH>
__global__ void __launch_bounds__(TH) k_ssm_step(SsmStepParams p)
{
    __shared__ float bc[2][256], decay;
    __shared__ float4 part[TH];
    const int h = static_cast<int>(blockIdx.x % p.H);
    const int64_t b = blockIdx.x / p.H;
    const int g = h / (p.H / p.G);
    const int N = p.N, P = p.P, lp = P / 4;  // threads per state row
    const int nrow = TH / lp;                // rows per pass of the block
    const int c = threadIdx.x % lp, r0 = threadIdx.x / lp;
    if (!dcheck(b < p.B && g < p.G && N <= 256 && lp * nrow == TH && nrow > 0, p.status)) return;
    float* S = p.S + (b * p.H + h) * static_cast<int64_t>(N) * P;

    float4 s[kRows];
    auto fetch = [&](int n0) {
#pragma unroll
        for (int k = 0; k < kRows; ++k)
            if (n0 + k * nrow < N) s[k] = *reinterpret_cast<const float4*>(S + static_cast<int64_t>(n0 + k * nrow) * P + c * 4);
    };
    fetch(r0);  // on its way while the token's operands are worked out
    for (int i = threadIdx.x; i < N; i += TH) {
        bc[0][i] = load_in(p.Bm, static_cast<size_t>(b * p.bs.b + g * p.bs.h + i), p.in_bf16);
        bc[1][i] = load_in(p.Cm, static_cast<size_t>(b * p.cs.b + g * p.cs.h + i), p.in_bf16);
    }
    const float d = step_size(load_in(p.dt, static_cast<size_t>(b * p.dts.b + h * p.dts.h), p.in_bf16),
                              p.dt_bias ? p.dt_bias[h] : 0.0f, p.softplus, p.dt_min, p.dt_max);
    if (threadIdx.x == 0) decay = exp2_of(static_cast<double>(d) * p.A[h] * 1.4426950408889634074);  // rounded once, as the prompt's
    float x[4], u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[j] = load_in(p.x, static_cast<size_t>(b * p.xs.b + h * p.xs.h + c * 4 + j), p.in_bf16);
        u[j] = d * x[j];
    }
    __syncthreads();
    const float a = decay;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int n0 = r0; n0 < N; n0 += nrow * kRows) {
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
        fetch(n0 + nrow * kRows);
    }
    part[threadIdx.x] = acc;
    __syncthreads();
    for (int i = threadIdx.x; i < P; i += TH) {
        const float* f = reinterpret_cast<const float*>(part);
        float y = 0.0f;
        for (int r = 0; r < nrow; ++r) y += f[r * P + i];
        const float xv = load_in(p.x, static_cast<size_t>(b * p.xs.b + h * p.xs.h + i), p.in_bf16);
        if (p.D) y = fmaf(p.D[h], xv, y);
        store_out(p.y, static_cast<size_t>((b * p.H + h) * P + i), y, p.out_bf16);
    }
}

}  // namespace

cudaError_t launch_ssm_step(const SsmStepParams& p, cudaStream_t s)
{
    const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(p.B) * p.H);
    // Enough threads for kRows pieces each, so that small heads leave room for more blocks.  (256 for all: 216 us instead of
    // 90 for 2048 x 16 heads of 16 x 128, 130 us instead of 85 for 1024 x 16 of 64 x 64.)
    const int want = p.N * p.P / (4 * kRows);
    if (want >= 256) k_ssm_step<256><<<grid, 256, 0, s>>>(p);
    else if (want >= 128) k_ssm_step<128><<<grid, 128, 0, s>>>(p);
    else if (want >= 64) k_ssm_step<64><<<grid, 64, 0, s>>>(p);
    else k_ssm_step<32><<<grid, 32, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace ramnet
