// ssm_scan.cu -- selective scan over a prompt, token by token in fp32 (any layout the entry
// point allows), and the chaining of segments:
//   d = clamp(softplus(dt + bias)),  S_t = exp(d A) S_{t-1} + d B_t (x) x_t,  y_t = C_t . S_t + D x_t
//
// k_ssm_scan: NS = N/16 neighbouring lanes own one channel p of one head and hold 16 of its N
// state values each in registers; blocks of kTok tokens of B, C, x and the step sizes are staged
// in shared memory.  Per token a thread takes 3 x 16 multiply-adds and a log2(NS)-step lane sum.
// Bound: fp32 issue (3 N P per token-head) and, with few heads, the latency of the token chain.
#include "ssm_common.cuh"

namespace ramnet {
namespace {

constexpr int kTok = 16;

template <int N, bool OUT>
__global__ void __launch_bounds__(128) k_ssm_scan(SsmParams p)
{
    constexpr int NS = N / 16;
    extern __shared__ float sm[];
    const int pt = blockDim.x / NS;  // channels per block
    float* sB = sm;                  // [kTok][N]
    float* sC = sB + kTok * N;       // [kTok][N]
    float* sX = sC + kTok * N;       // [kTok][pt]
    float* sA = sX + kTok * pt;      // [kTok] decay
    float* sD = sA + kTok;           // [kTok] step size
    const int seg = blockIdx.y;
    const int ptiles = p.P / pt;
    const int tile = static_cast<int>(blockIdx.x % ptiles);
    const int64_t bh = blockIdx.x / ptiles;
    const int h = static_cast<int>(bh % p.H);
    const int64_t b = bh / p.H;
    const int g = h / (p.H / p.G);
    const SegRange r = seg_range(seq_len(p.lengths, static_cast<int>(b), p.T), seg, OUT ? p.split.seg_len : p.split.piece_len());
    const int s = threadIdx.x % NS, pl = threadIdx.x / NS;
    const int ch = tile * pt + pl;
    const float A = p.A[h], bias = p.dt_bias ? p.dt_bias[h] : 0.0f, skip = p.D ? p.D[h] : 0.0f;

    // state value k of this thread is n = 4 * (s + NS * (k / 4)) + k % 4
    float S[16];
    const float* start = nullptr;
    if (OUT) {
        if (p.split.nseg > 1) start = p.seg_state + (bh * p.split.slots() + seg * p.split.sub) * static_cast<int64_t>(N) * p.P;
        else if (p.S_in) start = p.S_in + bh * static_cast<int64_t>(N) * p.P;
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const int n = 4 * (s + NS * (k / 4)) + k % 4;
        S[k] = start ? start[static_cast<int64_t>(n) * p.P + ch] : 0.0f;
    }
    double logdecay = 0.0;
    for (int t0 = r.first; t0 < r.last; t0 += kTok) {
        const int nt = min(kTok, r.last - t0);
        __syncthreads();
        for (int i = threadIdx.x; i < nt * N; i += blockDim.x) {
            const int t = i / N, n = i % N;
            sB[i] = load_in(p.Bm, static_cast<size_t>(b * p.bs.b + (t0 + t) * p.bs.t + g * p.bs.h + n), p.in_bf16);
            if (OUT) sC[i] = load_in(p.Cm, static_cast<size_t>(b * p.cs.b + (t0 + t) * p.cs.t + g * p.cs.h + n), p.in_bf16);
        }
        for (int i = threadIdx.x; i < nt * pt; i += blockDim.x) {
            const int t = i / pt, q = i % pt;
            sX[i] = load_in(p.x, static_cast<size_t>(b * p.xs.b + (t0 + t) * p.xs.t + h * p.xs.h + tile * pt + q), p.in_bf16);
        }
        for (int t = threadIdx.x; t < nt; t += blockDim.x) {
            const float d = step_size(load_in(p.dt, static_cast<size_t>(b * p.dts.b + (t0 + t) * p.dts.t + h * p.dts.h), p.in_bf16),
                                      bias, p.softplus, p.dt_min, p.dt_max);
            sD[t] = d;
            // rounded once from 64 bits: a bias of expf, a fraction of an ulp, would add up over
            // the thousands of tokens that a slowly decaying state remembers
            sA[t] = static_cast<float>(exp(static_cast<double>(d) * static_cast<double>(A)));
        }
        __syncthreads();
        if (!OUT && threadIdx.x == 0)
            for (int t = 0; t < nt; ++t) logdecay += static_cast<double>(sD[t]) * static_cast<double>(A);
        for (int t = 0; t < nt; ++t) {
            const float a = sA[t], x = sX[t * pt + pl], u = sD[t] * x;
            float y = 0.0f;
#pragma unroll
            for (int k4 = 0; k4 < 4; ++k4) {
                const float4 bv = *reinterpret_cast<const float4*>(sB + t * N + 4 * (s + NS * k4));
                const float bb[4] = {bv.x, bv.y, bv.z, bv.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) S[4 * k4 + j] = fmaf(bb[j], u, a * S[4 * k4 + j]);
                if (OUT) {
                    const float4 cv = *reinterpret_cast<const float4*>(sC + t * N + 4 * (s + NS * k4));
                    const float cc[4] = {cv.x, cv.y, cv.z, cv.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) y = fmaf(cc[j], S[4 * k4 + j], y);
                }
            }
            if (OUT) {
#pragma unroll
                for (int o = NS / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
                if (s == 0)
                    store_out(p.y, static_cast<size_t>(((b * p.T + t0 + t) * p.H + h) * p.P + ch), fmaf(skip, x, y), p.out_bf16);
            }
        }
    }
    float* end = nullptr;
    if (!OUT) end = p.seg_state + (bh * p.split.slots() + seg) * static_cast<int64_t>(N) * p.P;
    else if (seg == p.split.nseg - 1) end = p.S_out + bh * static_cast<int64_t>(N) * p.P;
    if (end) {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const int n = 4 * (s + NS * (k / 4)) + k % 4;
            end[static_cast<int64_t>(n) * p.P + ch] = S[k];
        }
    }
    if (!OUT && threadIdx.x == 0 && tile == 0)
        p.seg_decay[bh * p.split.pieces() + seg] = static_cast<float>(exp(logdecay));
}

// Turns what the pieces add into the states the segments start from, in token order; four
// neighbouring state values per thread, one (sequence, head) per blockIdx.y.  With chunk totals the
// pieces' decays come from those, else from seg_decay.
__global__ void __launch_bounds__(256) k_ssm_chain(SsmParams p)
{
    __shared__ float decay[256];
    let_next();
    after_before();
    const int np4 = p.N * p.P / 4;
    const int e = blockIdx.x * 256 + threadIdx.x;
    const int64_t bh = blockIdx.y;
    const int n = p.split.pieces(), sub = p.split.sub;
    for (int k = threadIdx.x >> 5; k < n; k += 8) {  // a warp per piece
        if (p.toks) {
            const int chunks = (p.T + kChunk - 1) / kChunk, per = p.split.piece_len() / kChunk;
            const int b = static_cast<int>((bh + p.chain_first) / p.H);
            const int have = (seq_len(p.lengths, b, p.T) + kChunk - 1) / kChunk;  // chunks that the sequence has
            double sum = 0.0;
            for (int i = k * per + (threadIdx.x & 31); i < min((k + 1) * per, have); i += 32) sum += p.toks[bh * chunks + i].total;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if ((threadIdx.x & 31) == 0) decay[k] = exp2_of(sum);
        } else if ((threadIdx.x & 31) == 0) {
            decay[k] = p.seg_decay[bh * n + k];
        }
    }
    __syncthreads();
    if (e >= np4) return;
    float4 s = p.S_in ? reinterpret_cast<const float4*>(p.S_in)[bh * np4 + e] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float4* at = reinterpret_cast<float4*>(p.seg_state) + bh * p.split.slots() * np4 + e;
#pragma unroll 4
    for (int k = 0; k < n; ++k, at += np4) {
        const float4 add = *at;
        const float d = decay[k];
        if (k % sub == 0) *at = s;
        s = make_float4(fmaf(d, s.x, add.x), fmaf(d, s.y, add.y), fmaf(d, s.z, add.z), fmaf(d, s.w, add.w));
    }
    *at = s;
}

template <int N>
cudaError_t go(const SsmParams& p, cudaStream_t s)
{
    constexpr int NS = N / 16;
    const int threads = p.P * NS < 128 ? p.P * NS : 128;
    const int pt = threads / NS;
    const size_t smem = sizeof(float) * (2 * kTok * N + kTok * pt + 2 * kTok);
    const unsigned gx = static_cast<unsigned>(static_cast<int64_t>(p.B) * p.H * (p.P / pt));
    if (p.split.nseg > 1) {
        k_ssm_scan<N, false><<<dim3(gx, p.split.pieces()), threads, smem, s>>>(p);
        const cudaError_t e = launch_ssm_chain(p, s);
        if (e != cudaSuccess) return e;
    }
    k_ssm_scan<N, true><<<dim3(gx, p.split.nseg), threads, smem, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_ssm_chain(const SsmParams& p, cudaStream_t s)
{
    const int64_t bh = static_cast<int64_t>(p.B) * p.H;
    for (int64_t at = 0; at < bh; at += 65535) {  // the grid's limit in y
        SsmParams q = p;
        const int64_t np = static_cast<int64_t>(p.N) * p.P;
        if (p.S_in) q.S_in = p.S_in + at * np;
        q.seg_state = p.seg_state + at * p.split.slots() * np;
        q.seg_decay = p.seg_decay + at * p.split.pieces();
        if (p.toks) q.toks = p.toks + at * ((p.T + kChunk - 1) / kChunk);
        q.chain_first = at;
        const int64_t rows = bh - at < 65535 ? bh - at : 65535;
        const cudaError_t e = launch_dependent(k_ssm_chain, dim3(static_cast<unsigned>((np / 4 + 255) / 256), static_cast<unsigned>(rows)), 256, 0, s, q);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// As many segments as fill 148 SMs with one block of 128 channels each, none shorter than 256
// tokens; and where the segments before the last leave SMs idle in the first launch, pieces of them.
SsmSplit ssm_split(int B, int T, int H, int G, int P)
{
    const int64_t units = static_cast<int64_t>(B) * G * ((static_cast<int64_t>(H / G) * P + 127) / 128);
    int64_t n = 148 / units;
    const int64_t most = T / 256;
    n = n < most ? n : most;
    SsmSplit s{1, T, 1};
    if (n <= 1) return s;
    s.seg_len = static_cast<int>((T + n - 1) / n + 63) / 64 * 64;
    s.nseg = (T + s.seg_len - 1) / s.seg_len;
    if (s.nseg <= 1) return SsmSplit{1, T, 1};
    while (units * (s.nseg - 1) * s.sub * 2 <= 148 && s.seg_len % (128 * s.sub) == 0) s.sub *= 2;
    return s;
}

cudaError_t launch_ssm_plain(const SsmParams& p, cudaStream_t s)
{
    switch (p.N) {
        case 16: return go<16>(p, s);
        case 32: return go<32>(p, s);
        case 64: return go<64>(p, s);
        case 128: return go<128>(p, s);
        case 256: return go<256>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_ssm_scan(const SsmParams& p, cudaStream_t s)
{
    if (ssm_mma_takes(p)) return launch_ssm_mma(p, s);
    SsmParams q = p;
    q.toks = nullptr;
    return launch_ssm_plain(q, s);
}

}  // namespace ramnet
