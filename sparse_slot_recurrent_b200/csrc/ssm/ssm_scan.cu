// ssm_scan.cu -- selective scan over a prompt, token by token in fp32 (any layout the entry
// point allows), and the chaining of segments:
//   d = clamp(softplus(dt + bias)),  S_t = exp(d A) S_{t-1} + d B_t (x) x_t,  y_t = C_t . S_t + D x_t
//
// k_ssm_scan: NS neighbouring lanes own one channel p of one head and hold NR = N/NS of its state values each in
// registers (NR = 16, fewer for small heads, so that a block has 128 threads).  Blocks of kTok tokens of B, C, x and the
// step sizes go through shared memory; while one is worked on, the next is on its way into registers.  Per token a
// thread takes 3 NR multiply-adds and a log2(NS)-step lane sum.
// Bound: fp32 issue (3 N P per token-head) and, with few heads, the latency of the token chain.
#include "ssm_common.cuh"

namespace ramnet {
namespace {

constexpr int kTok = 16;

template <int N, int NR, int PT, bool OUT>
__global__ void __launch_bounds__(PT * (N / NR)) k_ssm_scan(SsmParams p)
{
    constexpr int NS = N / NR, TH = PT * NS;  // lanes per channel, threads
    constexpr int LB = kTok * N / TH, LX = (kTok * PT + TH - 1) / TH;
    static_assert(NS <= 32 && kTok * N % TH == 0, "shape");
    __shared__ __align__(16) float sB[kTok * N], sC[OUT ? kTok * N : 4], sX[kTok * PT], sA[kTok], sD[kTok];
    const int seg = blockIdx.y, tid = threadIdx.x;
    const int ptiles = p.P / PT;
    const int tile = static_cast<int>(blockIdx.x % ptiles);
    const int64_t bh = blockIdx.x / ptiles;
    const int h = static_cast<int>(bh % p.H);
    const int64_t b = bh / p.H;
    const int g = h / (p.H / p.G);
    const SegRange r = seg_range(seq_len(p.lengths, static_cast<int>(b), p.T), seg, OUT ? p.split.seg_len : p.split.piece_len());
    const int s = tid % NS, pl = tid / NS;
    const int ch = tile * PT + pl;
    const float A = p.A[h], bias = p.dt_bias ? p.dt_bias[h] : 0.0f, skip = p.D ? p.D[h] : 0.0f;

    // state value k of this thread is n = 4 * (s + NS * (k / 4)) + k % 4
    float S[NR];
    const float* start = nullptr;
    if (OUT) {
        if (p.split.nseg > 1) start = p.seg_state + (bh * p.split.slots() + seg * p.split.sub) * static_cast<int64_t>(N) * p.P;
        else if (p.S_in) start = p.S_in + bh * static_cast<int64_t>(N) * p.P;
    }
#pragma unroll
    for (int k = 0; k < NR; ++k) {
        const int n = 4 * (s + NS * (k / 4)) + k % 4;
        S[k] = start ? start[static_cast<int64_t>(n) * p.P + ch] : 0.0f;
    }
    // the block of tokens from t0, into registers (tokens that are not there as zeros)
    float vB[LB], vC[LB], vX[LX], vD = 0.0f;
    auto fetch = [&](int t0) {
#pragma unroll
        for (int k = 0; k < LB; ++k) {
            const int i = k * TH + tid, t = t0 + i / N, n = i % N;
            vB[k] = t < r.last ? load_in(p.Bm, static_cast<size_t>(b * p.bs.b + t * p.bs.t + g * p.bs.h + n), p.in_bf16) : 0.0f;
            if (OUT) vC[k] = t < r.last ? load_in(p.Cm, static_cast<size_t>(b * p.cs.b + t * p.cs.t + g * p.cs.h + n), p.in_bf16) : 0.0f;
        }
#pragma unroll
        for (int k = 0; k < LX; ++k) {
            const int i = k * TH + tid, t = t0 + i / PT;
            vX[k] = i < kTok * PT && t < r.last ? load_in(p.x, static_cast<size_t>(b * p.xs.b + t * p.xs.t + h * p.xs.h + tile * PT + i % PT), p.in_bf16) : 0.0f;
        }
        if (tid < kTok && t0 + tid < r.last) vD = load_in(p.dt, static_cast<size_t>(b * p.dts.b + (t0 + tid) * p.dts.t + h * p.dts.h), p.in_bf16);
    };
    double logdecay = 0.0;  // of this thread's tokens (the first kTok threads)
    if (r.first < r.last) fetch(r.first);
    for (int t0 = r.first; t0 < r.last; t0 += kTok) {
        const int nt = min(kTok, r.last - t0);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < LB; ++k) {
            sB[k * TH + tid] = vB[k];
            if (OUT) sC[k * TH + tid] = vC[k];
        }
#pragma unroll
        for (int k = 0; k < LX; ++k)
            if (k * TH + tid < kTok * PT) sX[k * TH + tid] = vX[k];
        if (tid < nt) {
            const float d = step_size(vD, bias, p.softplus, p.dt_min, p.dt_max);
            const double l = static_cast<double>(d) * A;
            sD[tid] = d;
            // rounded once from 64 bits: a bias of expf, a fraction of an ulp, would add up over
            // the thousands of tokens that a slowly decaying state remembers
            sA[tid] = exp2_of(l * 1.4426950408889634074);
            logdecay += l;
        }
        __syncthreads();
        if (t0 + kTok < r.last) fetch(t0 + kTok);
#pragma unroll 2
        for (int t = 0; t < nt; ++t) {
            const float a = sA[t], x = sX[t * PT + pl], u = sD[t] * x;
            float y = 0.0f;
#pragma unroll
            for (int k4 = 0; k4 < NR / 4; ++k4) {
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
        for (int k = 0; k < NR; ++k) {
            const int n = 4 * (s + NS * (k / 4)) + k % 4;
            end[static_cast<int64_t>(n) * p.P + ch] = S[k];
        }
    }
    if (!OUT && tile == 0 && tid < 32) {
        if (tid >= kTok) logdecay = 0.0;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) logdecay += __shfl_xor_sync(0xffffffffu, logdecay, o);
        if (tid == 0) p.seg_decay[bh * p.split.pieces() + seg] = exp2_of(logdecay * 1.4426950408889634074);
    }
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

template <int N, int NR, int PT>
cudaError_t go(const SsmParams& p, cudaStream_t s)
{
    const unsigned gx = static_cast<unsigned>(static_cast<int64_t>(p.B) * p.H * (p.P / PT));
    if (p.split.nseg > 1) {
        k_ssm_scan<N, NR, PT, false><<<dim3(gx, p.split.pieces()), PT * (N / NR), 0, s>>>(p);
        const cudaError_t e = launch_ssm_chain(p, s);
        if (e != cudaSuccess) return e;
    }
    k_ssm_scan<N, NR, PT, true><<<dim3(gx, p.split.nseg), PT * (N / NR), 0, s>>>(p);
    return cudaGetLastError();
}

// 16 state values per thread, and as many channels as make 128 threads; small heads hold fewer values per thread
// instead (64 threads at the least).
template <int N>
cudaError_t shape(const SsmParams& p, cudaStream_t s)
{
    if constexpr (N >= 128) return go<N, 16, 2048 / N>(p, s);
    else if (p.P >= 64) return go<N, 16, 128 * 16 / N < 64 ? 128 * 16 / N : 64>(p, s);
    else if (p.P == 32) return go<N, N == 16 ? 4 : N / 4, 32>(p, s);
    else return go<N, N == 16 ? 4 : N / 8, 16>(p, s);
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
        case 16: return shape<16>(p, s);
        case 32: return shape<32>(p, s);
        case 64: return shape<64>(p, s);
        case 128: return shape<128>(p, s);
        case 256: return shape<256>(p, s);
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
