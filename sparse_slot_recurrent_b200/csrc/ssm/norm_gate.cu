// norm_gate.cu -- RMSNorm of rows in groups of channels, with a SiLU output gate before or
// behind the norm:
//   gate first:  u = x silu(z),  y = u / sqrt(mean_group(u^2) + eps) * w
//   norm first:  y = x / sqrt(mean_group(x^2) + eps) * w * silu(z)
// without z the gate is left out.  Sums in fp32, in a fixed order.
//
// Bound: HBM, x and z read once and y written once.  k_norm_warp: one warp per group of one row,
// with all of the group's loads in flight before the first is used and no barrier (groups up to
// 256 vectors: 2048 bf16 or 1024 fp32 channels at 16 bytes).  k_norm_block: one block per group, for longer groups; what it
// does not keep in registers it reads again, from L2.  Vectors of 16 bytes, or of two values or one where rows and
// addresses allow no more.
// (One block per row for all: 229 us for 65536 x 2048 bf16 rows, the block's barrier and its few
// bytes in flight.)
#include "rows.cuh"

namespace ramnet {
namespace {

// PRE: the gate, if any, comes before the norm (z is then used up before the sum).
template <int V, int NV, bool IB, bool OB, bool PRE>
__global__ void __launch_bounds__(128, 4) k_norm_warp(NormParams p)
{
    const int64_t id = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (id >= p.R * p.groups) return;
    const int lane = threadIdx.x & 31;
    const int64_t row = id / p.groups;
    const int width = p.D / p.groups, first = static_cast<int>(id % p.groups) * width, nv = width / V;
    if (!dcheck(row < p.R && first + width <= p.D && nv * V == width && nv <= 32 * NV, p.status)) return;
    Raw<IB, V> x[NV], z[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        x[k].clear();
        z[k].clear();
        const int i = lane + 32 * k;
        if (i < nv) {
            x[k].load(p.x, row * p.sx + first + static_cast<int64_t>(i) * V);
            if (p.z) z[k].load(p.z, row * p.sz + first + static_cast<int64_t>(i) * V);
        }
    }
    const bool pre = PRE && p.z;
    constexpr int H = (V + 1) / 2;
    Val<V> u[NV][H], sum2 = val<V>(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int h = 0; h < H; ++h) {
            u[k][h] = x[k].pair(h);
            if (pre) u[k][h] = mul2(u[k][h], silu2<OB>(z[k].pair(h)));
            sum2 = fma2(u[k][h], u[k][h], sum2);
        }
    float both[V > 1 ? V : 1] = {};
    put<V>(sum2, 0, both);
    float sum = both[0] + (V > 1 ? both[V > 1 ? 1 : 0] : 0.0f);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float inv = 1.0f / sqrtf(sum / static_cast<float>(width) + p.eps);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int i = lane + 32 * k, d = first + i * V;
        if (i < nv) {
            float y[V];
#pragma unroll
            for (int h = 0; h < H; ++h) {
                Val<V> v = mul2(u[k][h], val<V>(inv, inv));
                if (p.w) {
                    Raw<false, V == 1 ? 1 : 2> w;
                    w.load(p.w, d + 2 * h);
                    v = mul2(v, w.pair(0));
                }
                if (!PRE) v = mul2(v, silu2<OB>(z[k].pair(h)));
                put<V>(v, h, y);
            }
            store_vec<OB, V>(p.y, row * p.D + d, y);
        }
    }
}

constexpr int kThreads = 256;

// One group of one row per block; each thread keeps up to NV vectors of V channels.
template <int V, int NV, bool IB, bool OB>
__global__ void __launch_bounds__(kThreads) k_norm_block(NormParams p)
{
    __shared__ float part[kThreads / 32];
    constexpr int H = (V + 1) / 2;
    const int64_t row = blockIdx.x / p.groups;
    const int width = p.D / p.groups, first = static_cast<int>(blockIdx.x % p.groups) * width, nv = width / V;
    if (!dcheck(row < p.R && first + width <= p.D && nv * V == width, p.status)) return;
    Val<V> u[NV][H], gate[NV][H];

    auto fetch = [&](int i, Val<V> (&uu)[H], Val<V> (&gg)[H]) {
        Raw<IB, V> x, z;
        x.load(p.x, row * p.sx + first + static_cast<int64_t>(i) * V);
        x.widen(uu);
        if (p.z) {
            z.load(p.z, row * p.sz + first + static_cast<int64_t>(i) * V);
#pragma unroll
            for (int h = 0; h < H; ++h) {
                gg[h] = silu2<OB>(z.pair(h));
                if (p.gate_first) uu[h] = mul2(uu[h], gg[h]);
            }
        }
    };
    Val<V> sum2 = val<V>(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int i = threadIdx.x + k * kThreads;
        if (i < nv) {
            fetch(i, u[k], gate[k]);
#pragma unroll
            for (int h = 0; h < H; ++h) sum2 = fma2(u[k][h], u[k][h], sum2);
        }
    }
    for (int i = threadIdx.x + NV * kThreads; i < nv; i += kThreads) {
        Val<V> uu[H], gg[H];
        fetch(i, uu, gg);
#pragma unroll
        for (int h = 0; h < H; ++h) sum2 = fma2(uu[h], uu[h], sum2);
    }
    float both[V > 1 ? V : 1] = {};
    put<V>(sum2, 0, both);
    float sum = both[0] + (V > 1 ? both[V > 1 ? 1 : 0] : 0.0f);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
    __syncthreads();
    sum = part[0];
#pragma unroll
    for (int i = 1; i < kThreads / 32; ++i) sum += part[i];
    const float inv = 1.0f / sqrtf(sum / static_cast<float>(width) + p.eps);

    auto finish = [&](int i, const Val<V> (&uu)[H], const Val<V> (&gg)[H]) {
        const int d = first + i * V;
        float y[V];
#pragma unroll
        for (int h = 0; h < H; ++h) {
            Val<V> v = mul2(uu[h], val<V>(inv, inv));
            if (p.w) v = mul2(v, val<V>(p.w[d + 2 * h], p.w[d + (V > 1 ? 2 * h + 1 : 0)]));
            if (p.z && !p.gate_first) v = mul2(v, gg[h]);
            put<V>(v, h, y);
        }
        store_vec<OB, V>(p.y, row * p.D + d, y);
    };
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int i = threadIdx.x + k * kThreads;
        if (i < nv) finish(i, u[k], gate[k]);
    }
    for (int i = threadIdx.x + NV * kThreads; i < nv; i += kThreads) {
        Val<V> uu[H], gg[H];
        fetch(i, uu, gg);
        finish(i, uu, gg);
    }
}

template <int V, int NV, bool IB>
cudaError_t block(const NormParams& p, cudaStream_t s)
{
    const unsigned grid = static_cast<unsigned>(p.R * p.groups);
    if (p.out_bf16) k_norm_block<V, NV, IB, true><<<grid, kThreads, 0, s>>>(p);
    else k_norm_block<V, NV, IB, false><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <int V, int NV, bool IB>
cudaError_t warp(const NormParams& p, cudaStream_t s)
{
    const unsigned grid = static_cast<unsigned>((p.R * p.groups + 3) / 4);
    const bool pre = p.gate_first || !p.z;
    if (p.out_bf16) pre ? k_norm_warp<V, NV, IB, true, true><<<grid, 128, 0, s>>>(p) : k_norm_warp<V, NV, IB, true, false><<<grid, 128, 0, s>>>(p);
    else pre ? k_norm_warp<V, NV, IB, false, true><<<grid, 128, 0, s>>>(p) : k_norm_warp<V, NV, IB, false, false><<<grid, 128, 0, s>>>(p);
    return cudaGetLastError();
}

template <int V, bool IB>
cudaError_t pick(const NormParams& p, cudaStream_t s)
{
    const int nv = p.D / p.groups / V;
    if constexpr (Raw<IB, V>::kBytes == 16) {
        if (nv <= 32) return warp<V, 1, IB>(p, s);
        if (nv > 64 && nv <= 128) return warp<V, 4, IB>(p, s);
    }
    if (nv <= 64) return warp<V, 2, IB>(p, s);
    if (nv <= 256) return warp<V, 8, IB>(p, s);
    return block<V, V == 8 ? 2 : 4, IB>(p, s);
}

}  // namespace

cudaError_t launch_norm_gate(const NormParams& p, cudaStream_t s)
{
    const int v = widest(p.in_bf16, {p.D / p.groups, p.sx, p.z ? p.sz : 0}, {p.x, p.z});
    if (p.in_bf16) {
        if (v == 8) return pick<8, true>(p, s);
        return v == 2 ? pick<2, true>(p, s) : pick<1, true>(p, s);
    }
    if (v == 4) return pick<4, false>(p, s);
    return v == 2 ? pick<2, false>(p, s) : pick<1, false>(p, s);
}

}  // namespace ramnet
