// conv.cu -- short causal convolution along the sequence, one filter per channel, for prompts
// (k_conv) and for single tokens (k_conv_step):
//   y[t,c] = act(bias[c] + sum_k w[c,k] x[t-W+1+k,c]),  act = SiLU or none,
// with the W-1 inputs before the first token taken from a carried state.  Sums in fp32.
//
// Bound: HBM, one read of x and one write of y (2 W flops per element).  A thread owns V
// neighbouring channels (16 bytes, or two or one where addresses allow no more) over a run of tokens and slides a
// window of W-1 inputs in registers, so each input is read once but for W-1 rows per run (which
// the run before has just brought into L2).  Rows come through a ring in shared memory that
// only its own thread fills and reads, up to fourteen in flight.  For 4 x 16384 x 2304 bf16 channels: 273 us with one
// load at a time behind the store before it, 209 us with four in registers, 119 us this way (77% of the copy
// bandwidth); a fifth block per SM would cost the registers of the weights (185 us).  Products and sums run on pairs of channels.
#include "rows.cuh"

namespace ramnet {
namespace {

constexpr int kRunShort = 16, kRunLong = 64;  // tokens per thread

constexpr int kDepth = 8;   // steps of two rows in a thread's ring: seven in flight, one in use
static_assert(kRunShort % 8 == 0 && kRunLong % 8 == 0, "whole steps");

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src)
{
    if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}

template <int W, int V, bool IB, bool OB>
__global__ void __launch_bounds__(128, V > 1 ? 4 : 1) k_conv(ConvParams p, int ncv, int64_t work, int run_len)
{
    const int64_t id = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
    if (id >= work) return;
    const int cv = static_cast<int>(id % ncv);
    const int64_t run = id / ncv;
    const int runs = (p.T + run_len - 1) / run_len;
    const int b = static_cast<int>(run / runs);
    const int t0 = static_cast<int>(run % runs) * run_len;
    const int c = cv * V;
    int len = p.T;
    if (p.lengths) len = min(max(p.lengths[b], 0), p.T);
    if (t0 >= len && t0 > 0) return;
    const int t1 = min(t0 + run_len, len);
    if (!dcheck(b < p.B && c + V <= p.C && t0 >= 0 && t1 <= p.T, p.status)) return;
    constexpr int H = (V + 1) / 2;            // pairs of channels
    constexpr int kBytes = Raw<IB, V>::kBytes;
    constexpr bool kRing = kBytes >= 4;       // what copies itself; a lone bf16 value comes through registers
    constexpr int kBatch = kRing ? 2 : 8;     // rows per step

    Val<V> wt[W][H], bias[H], win[W + kBatch - 1][H];
    {
        float wv[V][W], bv[V];
        const bool wide = W == 4 && (reinterpret_cast<uintptr_t>(p.w) & 15) == 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (wide) {
                const float4 f = *reinterpret_cast<const float4*>(p.w + static_cast<int64_t>(c + v) * 4);
                const float a[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                for (int k = 0; k < W; ++k) wv[v][k] = a[k];
            } else {
#pragma unroll
                for (int k = 0; k < W; ++k) wv[v][k] = p.w[static_cast<int64_t>(c + v) * W + k];
            }
            bv[v] = p.bias ? p.bias[c + v] : 0.0f;
        }
#pragma unroll
        for (int h = 0; h < H; ++h) {
#pragma unroll
            for (int k = 0; k < W; ++k) wt[k][h] = val<V>(wv[2 * h][k], wv[(2 * h + 1) % V][k]);
            bias[h] = val<V>(bv[2 * h], bv[(2 * h + 1) % V]);
        }
    }
    const int64_t xb = static_cast<int64_t>(b) * p.sb + c;
    const int64_t sbase = static_cast<int64_t>(b) * (W - 1) * p.C + c;
    Raw<IB, V> old[W - 1];  // the carried state, kept by the first run (it also writes state_out)
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        const int t = t0 - (W - 1) + k;
        if (t >= 0) old[k].load(p.x, xb + static_cast<int64_t>(t) * p.st);
        else if (p.state_in) old[k].load(p.state_in, sbase + static_cast<int64_t>(t + W - 1) * p.C);
        else old[k].clear();
        old[k].widen(win[k]);
    }
    // each thread's own ring of rows in shared memory, or one step in registers
    __shared__ __align__(16) unsigned char ring[kRing ? kDepth * kBatch * 128 * kBytes : 16];
    const uint32_t mine = smem_addr(ring) + threadIdx.x * kBytes;
    Raw<IB, V> next[kBatch];
    const unsigned char* src = reinterpret_cast<const unsigned char*>(p.x) + (xb + static_cast<int64_t>(t0) * p.st) * (IB ? 2 : 4);
    const int64_t stride = p.st * (IB ? 2 : 4);
    auto fetch = [&](int t) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (t + i < t1) {
                if constexpr (kRing) copy_async<kBytes>(mine + (((t - t0) & (kDepth * kBatch - 1)) + i) * (128 * kBytes), src + (t - t0 + i) * stride);
                else next[i].load(p.x, xb + static_cast<int64_t>(t + i) * p.st);
            }
        if constexpr (kRing) asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int d = 0; d < (kRing ? kDepth - 1 : 1); ++d) fetch(t0 + d * kBatch);
#pragma unroll 1
    for (int t = t0; t < t1; t += kBatch) {
        if constexpr (kRing) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 2) : "memory");
#pragma unroll
            for (int i = 0; i < kBatch; ++i) next[i].take(ring + (((t - t0) & (kDepth * kBatch - 1)) + i) * (128 * kBytes) + threadIdx.x * kBytes);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) next[i].widen(win[W - 1 + i]);
        fetch(t + (kRing ? (kDepth - 1) * kBatch : kBatch));
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            float y[V];
#pragma unroll
            for (int h = 0; h < H; ++h) {
                Val<V> acc = bias[h];
#pragma unroll
                for (int k = 0; k < W; ++k) acc = fma2(wt[k][h], win[i + k][h], acc);
                if (p.silu) acc = silu2<OB>(acc);
                put<V>(acc, h, y);
            }
            if (t + i < t1) store_vec<OB, V>(p.y, (static_cast<int64_t>(b) * p.T + t + i) * p.C + c, y);
        }
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
#pragma unroll
            for (int h = 0; h < H; ++h) win[k][h] = win[kBatch + k][h];
    }
    // The last W-1 inputs: from x, or from the old state where the sequence is shorter.  Only
    // the first run touches the state, after it has read all of it, so it may be in place.
    if (t0 == 0 && p.state_out) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            const int t = len - (W - 1) + k;
            Raw<IB, V> r;
            r.clear();
            if (t >= 0) {
                r.load(p.x, xb + static_cast<int64_t>(t) * p.st);
            } else {
#pragma unroll
                for (int q = 0; q < W - 1; ++q)
                    if (q == t + W - 1) r = old[q];
            }
            r.store(p.state_out, sbase + static_cast<int64_t>(k) * p.C);
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
    if (!dcheck(b < p.B && c + V <= p.C, p.status)) return;
    const int64_t sbase = b * (W - 1) * p.C + c;
    Raw<IB, V> in[W];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) in[k].load(p.state, sbase + static_cast<int64_t>(k) * p.C);
    in[W - 1].load(p.x, b * p.sb + c);
    constexpr int H = (V + 1) / 2;
    Val<V> win[W][H];
#pragma unroll
    for (int k = 0; k < W; ++k) in[k].widen(win[k]);
    float y[V];
#pragma unroll
    for (int h = 0; h < H; ++h) {
        const int c1 = c + (V > 1 ? 2 * h + 1 : 0);
        Val<V> acc = p.bias ? val<V>(p.bias[c + 2 * h], p.bias[c1]) : val<V>(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < W; ++k)
            acc = fma2(val<V>(p.w[static_cast<int64_t>(c + 2 * h) * W + k], p.w[static_cast<int64_t>(c1) * W + k]), win[k][h], acc);
        if (p.silu) acc = silu2<OB>(acc);
        put<V>(acc, h, y);
    }
    store_vec<OB, V>(p.y, b * p.C + c, y);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) in[k + 1].store(p.state, sbase + static_cast<int64_t>(k) * p.C);
}

template <int W, int V, bool IB, bool OB>
cudaError_t go(const ConvParams& p, cudaStream_t s)
{
    const int ncv = p.C / V;
    // Long runs read fewer rows twice and load their weights less often; short ones where those would leave SMs idle.
    // (B4 T16384 C2304 bf16: 120 us in runs of 64, 155 in runs of 16; B1 T4096: 17 and 15.)
    int run = kRunLong;
    while (run > kRunShort && static_cast<int64_t>(ncv) * p.B * ((p.T + run - 1) / run) < 2ll * 148 * 640) run /= 2;
    const int64_t work = static_cast<int64_t>(ncv) * p.B * ((p.T + run - 1) / run);
    k_conv<W, V, IB, OB><<<static_cast<unsigned>((work + 127) / 128), 128, 0, s>>>(p, ncv, work, run);
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

template <int W, int V, bool IB, class P>
cudaError_t pick_out(const P& p, cudaStream_t s)
{
    return p.out_bf16 ? go<W, V, IB, true>(p, s) : go<W, V, IB, false>(p, s);
}

template <int W, class P>
cudaError_t pick_v(const P& p, int v, cudaStream_t s)
{
    if (p.in_bf16) {
        if (v == 8) return pick_out<W, 8, true>(p, s);
        return v == 2 ? pick_out<W, 2, true>(p, s) : pick_out<W, 1, true>(p, s);
    }
    if (v == 4) return pick_out<W, 4, false>(p, s);
    return v == 2 ? pick_out<W, 2, false>(p, s) : pick_out<W, 1, false>(p, s);
}

template <class P>
cudaError_t pick_w(const P& p, int v, cudaStream_t s)
{
    switch (p.W) {
        case 2: return pick_v<2>(p, v, s);
        case 3: return pick_v<3>(p, v, s);
        case 4: return pick_v<4>(p, v, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

// (y and the states start on 16 bytes, and their rows follow from C)
cudaError_t launch_conv(const ConvParams& p, cudaStream_t s) { return pick_w(p, widest(p.in_bf16, {p.C, p.sb, p.st}, {p.x}), s); }

cudaError_t launch_conv_step(const ConvStepParams& p, cudaStream_t s) { return pick_w(p, widest(p.in_bf16, {p.C, p.sb}, {p.x}), s); }

}  // namespace ramnet
