// ssm_scan.cu -- selective scan over a prompt, token by token in fp32 (any layout the entry
// point allows), and the chaining of segments:
//   d = clamp(softplus(dt + bias)),  S_t = exp(d A) S_{t-1} + d B_t (x) x_t,  y_t = C_t . S_t + D x_t
//
// k_ssm_scan: NS neighbouring lanes own one channel p of one head and hold NR = N/NS of its state values each in
// registers (NR = 16, fewer for small heads, so that a block has 128 threads).  Blocks of kTok tokens of B, C, x and the
// step sizes go through shared memory; while one is worked on, the next is on its way into registers.  Per token a
// thread takes 3 NR multiply-adds and a log2(NS)-step lane sum.
// k_ssm_tile, for heads of at least 64 x 32 values or so: a thread holds 8 state values of 4 channels, so that a token's
// loads from shared memory (5 x 16 bytes) serve 96 multiply-adds, taken in pairs; the lane sum scatters the channels while it
// adds, and y leaves through shared memory.  (k_ssm_scan moves four times the shared memory per value: 9.8 ms for
// B4 T16384 H16 P128 N128 in fp32, against 3.7 ms.)  The lane sums take four tokens at once: one at a time their shuffles
// were each token's latency (5.0 ms).
// The state is rounded to fp32 once per token, as the definition reads: 1.8e-7 off the 64-bit state over 333 tokens, where
// sums over chunks of 64 tokens are 0.7e-7 off.
// Bound: fp32 issue (3 N P per token-head) and, with few heads, the latency of the token chain.
#include "pairs.cuh"
#include "ssm_common.cuh"

namespace ramnet {
namespace {

constexpr int kTok = 16;

// One input value's bits, and the value: kept apart, so that loads that are in flight wait for nothing.
template <bool BF>
__device__ __forceinline__ uint32_t bits_at(const void* p, int64_t i)
{
    if constexpr (BF) return reinterpret_cast<const uint16_t*>(p)[i];
    else return reinterpret_cast<const uint32_t*>(p)[i];
}
template <bool BF>
__device__ __forceinline__ float value_of(uint32_t bits)
{
    return __uint_as_float(BF ? bits << 16 : bits);
}

template <int N, int NR, int PT, bool BF, bool OUT>
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
    if (!dcheck(b < p.B && g < p.G && (tile + 1) * PT <= p.P && segment_fits(p, r, seg, OUT), p.status)) return;
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
    uint32_t vB[LB], vC[LB], vX[LX], vD = 0;
    auto fetch = [&](int t0) {
#pragma unroll
        for (int k = 0; k < LB; ++k) {
            const int i = k * TH + tid, t = t0 + i / N, n = i % N;
            vB[k] = t < r.last ? bits_at<BF>(p.Bm, b * p.bs.b + t * p.bs.t + g * p.bs.h + n) : 0u;
            if (OUT) vC[k] = t < r.last ? bits_at<BF>(p.Cm, b * p.cs.b + t * p.cs.t + g * p.cs.h + n) : 0u;
        }
#pragma unroll
        for (int k = 0; k < LX; ++k) {
            const int i = k * TH + tid, t = t0 + i / PT;
            vX[k] = i < kTok * PT && t < r.last ? bits_at<BF>(p.x, b * p.xs.b + t * p.xs.t + h * p.xs.h + tile * PT + i % PT) : 0u;
        }
        if (tid < kTok && t0 + tid < r.last) vD = bits_at<BF>(p.dt, b * p.dts.b + (t0 + tid) * p.dts.t + h * p.dts.h);
    };
    double logdecay = 0.0;  // of this thread's tokens (the first kTok threads)
    if (r.first < r.last) fetch(r.first);
    for (int t0 = r.first; t0 < r.last; t0 += kTok) {
        const int nt = min(kTok, r.last - t0);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < LB; ++k) {
            sB[k * TH + tid] = value_of<BF>(vB[k]);
            if (OUT) sC[k * TH + tid] = value_of<BF>(vC[k]);
        }
#pragma unroll
        for (int k = 0; k < LX; ++k)
            if (k * TH + tid < kTok * PT) sX[k * TH + tid] = value_of<BF>(vX[k]);
        if (tid < nt) {
            const float d = step_size(value_of<BF>(vD), bias, p.softplus, p.dt_min, p.dt_max);
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

// Threads of k_ssm_tile: N/8 neighbouring lanes for 4 channels, PT channels per block.
template <int N, int PT, bool BF, bool OUT>
__global__ void __launch_bounds__(N / 8 * (PT / 4)) k_ssm_tile(SsmParams p)
{
    constexpr int kTok = N > 128 ? 8 : 16;  // (the next block's registers)
    constexpr int NG = N / 8, TH = NG * (PT / 4);
    constexpr int LB = kTok * N / TH, LX = kTok * PT / TH;
    static_assert(NG <= 32 && LB * TH == kTok * N && LX * TH == kTok * PT, "shape");
    __shared__ __align__(16) float sB[kTok * N], sC[OUT ? kTok * N : 4], sX[kTok * PT], sY[OUT ? kTok * PT : 4];
    __shared__ float2 sA[kTok];  // a token's decay and step size
    const int seg = blockIdx.y, tid = threadIdx.x;
    const int ptiles = p.P / PT;
    const int tile = static_cast<int>(blockIdx.x % ptiles);
    const int64_t bh = blockIdx.x / ptiles;
    const int h = static_cast<int>(bh % p.H);
    const int64_t b = bh / p.H;
    const int g = h / (p.H / p.G);
    const SegRange r = seg_range(seq_len(p.lengths, static_cast<int>(b), p.T), seg, OUT ? p.split.seg_len : p.split.piece_len());
    if (!dcheck(b < p.B && g < p.G && (tile + 1) * PT <= p.P && segment_fits(p, r, seg, OUT), p.status)) return;
    const int s = tid % NG, pl = tid / NG * 4;  // lane's place among the state values; its first channel
    const int64_t np = static_cast<int64_t>(N) * p.P;
    const float A = p.A[h], bias = p.dt_bias ? p.dt_bias[h] : 0.0f, skip = p.D ? p.D[h] : 0.0f;

    // values n = 4 (s + NG (k/2)) + 2 (k%2) and n + 1, for k < 4, of channels pl + q
    F2 S[4][4];
    auto at = [&](int k) { return 4 * (s + NG * (k >> 1)) + 2 * (k & 1); };
    const float* start = nullptr;
    if (OUT) {
        if (p.split.nseg > 1) start = p.seg_state + (bh * p.split.slots() + seg * p.split.sub) * np;
        else if (p.S_in) start = p.S_in + bh * np;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float4 lo = make_float4(0.0f, 0.0f, 0.0f, 0.0f), hi = lo;
        if (start) {
            lo = *reinterpret_cast<const float4*>(start + static_cast<int64_t>(at(k)) * p.P + tile * PT + pl);
            hi = *reinterpret_cast<const float4*>(start + static_cast<int64_t>(at(k) + 1) * p.P + tile * PT + pl);
        }
        S[k][0] = f2(lo.x, hi.x), S[k][1] = f2(lo.y, hi.y), S[k][2] = f2(lo.z, hi.z), S[k][3] = f2(lo.w, hi.w);
    }
    // The block of tokens from t0, into registers (tokens that are not there as zeros).  Value k of a thread lies a fixed
    // number of tokens and columns behind its first.
    uint32_t vB[LB], vC[LB], vX[LX], vD = 0;
    const int64_t oB = b * p.bs.b + g * p.bs.h + tid % N + (r.first + tid / N) * p.bs.t, oC = b * p.cs.b + g * p.cs.h + tid % N + (r.first + tid / N) * p.cs.t;
    const int64_t oX = b * p.xs.b + h * p.xs.h + tile * PT + tid % PT + (r.first + tid / PT) * p.xs.t, oD = b * p.dts.b + h * p.dts.h + (r.first + tid) * p.dts.t;
    auto fetch = [&](int t0) {
        const int64_t on = t0 - r.first;
        const int left = r.last - t0;
        const int64_t fB = oB + on * p.bs.t, fC = oC + on * p.cs.t, fX = oX + on * p.xs.t;
#pragma unroll
        for (int k = 0; k < LB; ++k) {
            const int t = k * TH / N, n = k * TH % N;
            vB[k] = t + tid / N < left ? bits_at<BF>(p.Bm, fB + t * p.bs.t + n) : 0u;
            if (OUT) vC[k] = t + tid / N < left ? bits_at<BF>(p.Cm, fC + t * p.cs.t + n) : 0u;
        }
#pragma unroll
        for (int k = 0; k < LX; ++k) {
            const int t = k * TH / PT, c = k * TH % PT;
            vX[k] = t + tid / PT < left ? bits_at<BF>(p.x, fX + t * p.xs.t + c) : 0u;
        }
        if (tid < kTok && tid < left) vD = bits_at<BF>(p.dt, oD + on * p.dts.t);
    };
    const int64_t yrow = static_cast<int64_t>(p.H) * p.P, oY = (b * p.T + tid / PT) * yrow + static_cast<int64_t>(h) * p.P + tile * PT + tid % PT;
    auto leave = [&](int t0, int nt) {  // y of the block of nt tokens from t0
        const int64_t to = oY + t0 * yrow;
#pragma unroll
        for (int k = 0; k < LX; ++k) {
            const int t = k * TH / PT, c = k * TH % PT;
            if (t + tid / PT < nt) store_out(p.y, static_cast<size_t>(to + t * yrow + c), sY[k * TH + tid], p.out_bf16);
        }
    };
    double logdecay = 0.0;  // of this thread's tokens (the first kTok threads)
    if (r.first < r.last) fetch(r.first);
    for (int t0 = r.first; t0 < r.last; t0 += kTok) {
        const int nt = min(kTok, r.last - t0);
        __syncthreads();
        if (OUT && t0 > r.first) leave(t0 - kTok, kTok);
#pragma unroll
        for (int k = 0; k < LB; ++k) {
            sB[k * TH + tid] = value_of<BF>(vB[k]);
            if (OUT) sC[k * TH + tid] = value_of<BF>(vC[k]);
        }
#pragma unroll
        for (int k = 0; k < LX; ++k) sX[k * TH + tid] = value_of<BF>(vX[k]);
        if (tid < kTok) {
            float2 ad = make_float2(1.0f, 0.0f);  // a token that is not there changes nothing
            if (tid < nt) {
                const float d = step_size(value_of<BF>(vD), bias, p.softplus, p.dt_min, p.dt_max);
                const double l = static_cast<double>(d) * A;
                ad = make_float2(exp2_of(l * 1.4426950408889634074), d);  // rounded once from 64 bits, as in k_ssm_scan
                logdecay += l;
            }
            sA[tid] = ad;
        }
        __syncthreads();
        if (t0 + kTok < r.last) fetch(t0 + kTok);
#pragma unroll 1
        for (int t4 = 0; t4 < nt; t4 += 4) {
            float v[16];  // this lane's part of y: 4 tokens x 4 channels
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = t4 + i;
                const float2 ad = sA[t];
                const float4 xv = *reinterpret_cast<const float4*>(sX + t * PT + pl);
                const F2 a = f2(ad.x, ad.x);
                const F2 u[4] = {f2(ad.y * xv.x, ad.y * xv.x), f2(ad.y * xv.y, ad.y * xv.y), f2(ad.y * xv.z, ad.y * xv.z), f2(ad.y * xv.w, ad.y * xv.w)};
                F2 y[4] = {f2(0.0f, 0.0f), f2(0.0f, 0.0f), f2(0.0f, 0.0f), f2(0.0f, 0.0f)};
#pragma unroll
                for (int k2 = 0; k2 < 2; ++k2) {
                    const float4 bv = *reinterpret_cast<const float4*>(sB + t * N + 4 * (s + NG * k2));
                    const F2 bb[2] = {f2(bv.x, bv.y), f2(bv.z, bv.w)};
                    F2 cc[2];
                    if (OUT) {
                        const float4 cv = *reinterpret_cast<const float4*>(sC + t * N + 4 * (s + NG * k2));
                        cc[0] = f2(cv.x, cv.y), cc[1] = f2(cv.z, cv.w);
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            F2& w = S[2 * k2 + j][q];
                            w = fma2(bb[j], u[q], mul2(a, w));
                            if (OUT) y[q] = fma2(cc[j], w, y[q]);
                        }
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float e, f;
                    un(y[q], e, f);
                    v[4 * i + q] = e + f;
                }
            }
            if (OUT) {
                // sums over the lanes of these channels: of two lanes each hands the other half of its values, then whole sums
                constexpr int kHalvings = NG >= 16 ? 4 : NG == 8 ? 3 : NG == 4 ? 2 : 1;
                int first = 0;  // of this lane's values among the 16
#pragma unroll
                for (int m = 0; m < kHalvings; ++m) {
                    const int half = 8 >> m;
                    const bool up = s & (1 << m);
                    first += up ? half : 0;
#pragma unroll
                    for (int e = 0; e < half; ++e) {
                        const float give = up ? v[e] : v[e + half];
                        v[e] = (up ? v[e + half] : v[e]) + __shfl_xor_sync(0xffffffffu, give, 1 << m);
                    }
                }
#pragma unroll
                for (int o = 16; o < NG; o <<= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
                if (s < 16) {
#pragma unroll
                    for (int e = 0; e < (16 >> kHalvings); ++e) {
                        const int at = (t4 + ((first + e) >> 2)) * PT + pl + ((first + e) & 3);
                        sY[at] = fmaf(skip, sX[at], v[e]);
                    }
                }
            }
        }
    }
    if (OUT && r.first < r.last) {
        __syncthreads();
        const int done = (r.last - r.first - 1) / kTok * kTok;
        leave(r.first + done, r.last - r.first - done);
    }
    float* end = nullptr;
    if (!OUT) end = p.seg_state + (bh * p.split.slots() + seg) * np;
    else if (seg == p.split.nseg - 1) end = p.S_out + bh * np;
    if (end) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float4 lo, hi;
            un(S[k][0], lo.x, hi.x);
            un(S[k][1], lo.y, hi.y);
            un(S[k][2], lo.z, hi.z);
            un(S[k][3], lo.w, hi.w);
            *reinterpret_cast<float4*>(end + static_cast<int64_t>(at(k)) * p.P + tile * PT + pl) = lo;
            *reinterpret_cast<float4*>(end + static_cast<int64_t>(at(k) + 1) * p.P + tile * PT + pl) = hi;
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
// pieces' decays come from those, else from seg_decay.  Bound: latency; the next piece's values are asked for one ahead, the
// first before the decays are summed (B8 T4096 H8 P128 N128: 95 us in all instead of 96).
__global__ void __launch_bounds__(256) k_ssm_chain(SsmParams p)
{
    __shared__ float decay[256];
    let_next();
    after_before();
    const int np4 = p.N * p.P / 4;
    const int e = blockIdx.x * 256 + threadIdx.x;
    const int64_t bh = blockIdx.y;
    const int n = p.split.pieces(), sub = p.split.sub;
    if (!dcheck(bh < static_cast<int64_t>(p.B) * p.H && n <= 256 && sub > 0 && n % sub == 0, p.status)) return;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f), add = s;
    float4* at = reinterpret_cast<float4*>(p.seg_state) + bh * p.split.slots() * np4 + e;
    if (e < np4) {  // on their way while the decays are summed
        if (p.S_in) s = reinterpret_cast<const float4*>(p.S_in)[bh * np4 + e];
        add = *at;
    }
    for (int k = threadIdx.x >> 5; k < n; k += 8) {  // a warp per piece
        if (p.toks) {
            const int chunks = (p.T + kChunk - 1) / kChunk, per = p.split.piece_len() / kChunk;
            const int b = static_cast<int>(bh / p.H);
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
#pragma unroll 4
    for (int k = 0; k < n; ++k, at += np4) {
        float4 next = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (k + 1 < n) next = at[np4];
        const float d = decay[k];
        if (k % sub == 0) *at = s;
        s = make_float4(fmaf(d, s.x, add.x), fmaf(d, s.y, add.y), fmaf(d, s.z, add.z), fmaf(d, s.w, add.w));
        add = next;
    }
    *at = s;
}

template <class K1, class K2>
cudaError_t launches(const SsmParams& p, K1 pieces, K2 outputs, int pt, int threads, cudaStream_t s)
{
    const unsigned gx = static_cast<unsigned>(static_cast<int64_t>(p.B) * p.H * (p.P / pt));
    if (p.split.nseg > 1) {
        pieces<<<dim3(gx, p.split.pieces()), threads, 0, s>>>(p);
        const cudaError_t e = launch_ssm_chain(p, s);
        if (e != cudaSuccess) return e;
    }
    outputs<<<dim3(gx, p.split.nseg), threads, 0, s>>>(p);
    return cudaGetLastError();
}

template <int N, int NR, int PT>
cudaError_t small(const SsmParams& p, cudaStream_t s)
{
    return p.in_bf16 ? launches(p, k_ssm_scan<N, NR, PT, true, false>, k_ssm_scan<N, NR, PT, true, true>, PT, PT * (N / NR), s)
                     : launches(p, k_ssm_scan<N, NR, PT, false, false>, k_ssm_scan<N, NR, PT, false, true>, PT, PT * (N / NR), s);
}

template <int N, int PT>
cudaError_t tiled(const SsmParams& p, cudaStream_t s)
{
    return p.in_bf16 ? launches(p, k_ssm_tile<N, PT, true, false>, k_ssm_tile<N, PT, true, true>, PT, N / 8 * (PT / 4), s)
                     : launches(p, k_ssm_tile<N, PT, false, false>, k_ssm_tile<N, PT, false, true>, PT, N / 8 * (PT / 4), s);
}

// The tiled form where a head makes a block of at least 64 threads of it (128 at most, over 4096/N channels); else 4 to 16
// values per thread so that the head still makes 64 or 128.
template <int N>
cudaError_t shape(const SsmParams& p, cudaStream_t s)
{
    constexpr int most = 4096 / N;
    if (p.P >= most) return tiled<N, most>(p, s);
    if (2 * p.P >= most) return tiled<N, most / 2>(p, s);
    if constexpr (N == 64) return small<N, 8, 16>(p, s);
    if constexpr (N < 64) {
        if (p.P >= 64) return small<N, 16, 64>(p, s);
        return p.P == 32 ? small<N, N / 4, 32>(p, s) : small<N, 4, 16>(p, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

// (Sequences are cut only where they are few: 148 blocks of four heads, or of 64 threads of 512 per SM, at most some hundreds.)
cudaError_t launch_ssm_chain(const SsmParams& p, cudaStream_t s)
{
    const unsigned heads = static_cast<unsigned>(p.B) * p.H;
    return launch_dependent(k_ssm_chain, dim3(static_cast<unsigned>((p.N * p.P / 4 + 255) / 256), heads), 256, 0, s, p);
}

// As many segments as fill 148 SMs with one block of 128 channels each, none shorter than 256 tokens, and none at all
// below 768 tokens, where two more launches cost more than they save.  (H2 P128 N128, whole against cut: T512 25 us and 31,
// T1024 39 and 31, T4096 126 and 32; B1 H32 T4096 130 and 70.)  Where the segments before the last leave SMs idle in
// the first launch, pieces of them run there: halving them saves a chunk's time for every 64 tokens (about a
// microsecond), and the chain takes about a quarter of that per piece more.  (B6 T1021 H24 P64 N64: 44 us with whole
// segments, 38 with halves; but H2 T4096, 16 segments of 256 tokens: 32 us whole, 42 in quarters.)
SsmSplit ssm_split(int B, int T, int H, int G, int P)
{
    const int64_t units = static_cast<int64_t>(B) * G * ((static_cast<int64_t>(H / G) * P + 127) / 128);
    int64_t n = 148 / units;
    const int64_t most = T / 256;
    n = n < most ? n : most;
    SsmSplit s{1, T, 1};
    if (n <= 1 || most <= 2) return s;
    s.seg_len = static_cast<int>((T + n - 1) / n + 63) / 64 * 64;
    s.nseg = (T + s.seg_len - 1) / s.seg_len;
    if (s.nseg <= 1) return SsmSplit{1, T, 1};
    while (units * s.pieces() * 2 <= 148 && s.seg_len % (128 * s.sub) == 0 && s.seg_len / (128 * s.sub) * 4 >= s.pieces()) s.sub *= 2;
    return s;
}

// The same for the token-by-token form, where a token costs a block its latency whatever else runs: segments from 64
// tokens on while there are no more than 512 threads per SM, but none where that leaves only two (the first launch and the
// chain then cost what they save), and 64 at most, for the chain.  Whole against cut, fp32: B2 T333 H5 P32 N16 59 us and
// 28, T2048 341 and 36; B4 T4096 H20 P64 N64 853 and 397; H16 P128 N128 T16384 B1 4.1 ms and 1.2, B4 (in two) 5.0
// and 5.4.  Up to 256 threads: 164 us instead of 111 for B5 T11720 H5 P16 N16; up to 1024: 107 instead of 88 for B5 T276
// H42 P16 N256.  118 segments: 99 us instead of 95 for B5 T7669 H2 P16 N128.
SsmSplit ssm_split_plain(int B, int T, int H, int N, int P)
{
    int most = 4096 / N;
    while (most > P) most /= 2;  // channels per block
    const int threads = N * most > 1024 ? N * most / 32 : 64;
    const int64_t units = static_cast<int64_t>(B) * H * (P / most);
    int64_t n = 148 * 512 / (units * threads);
    n = n < T / 64 ? n : T / 64;
    if (n > 64) n = 64;
    SsmSplit s{1, T, 1};
    if (n <= 2) return s;
    s.seg_len = static_cast<int>((T + n - 1) / n + 15) / 16 * 16;
    s.nseg = (T + s.seg_len - 1) / s.seg_len;
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

// The tensor-core form, but for a few tokens of a few heads: those are through, token by token, before a chunk of 64 is.
// (H16 P128 N128, one launch against two: B4 T16 14 us and 18, T64 27 and 23; but B9 T32 28 and 18, B64 T16 85 and 61.)
cudaError_t launch_ssm_scan(const SsmParams& p, cudaStream_t s)
{
    SsmParams q = p;
    const bool few = p.T <= 16 && static_cast<int64_t>(p.B) * p.H * p.P <= 148 * 128;
    if (!few && ssm_mma_takes(p)) {
        q.split = ssm_split(p.B, p.T, p.H, p.G, p.P);
        return launch_ssm_mma(q, s);
    }
    q.split = ssm_split_plain(p.B, p.T, p.H, p.N, p.P);
    q.toks = nullptr;
    return launch_ssm_plain(q, s);
}

}  // namespace ramnet
