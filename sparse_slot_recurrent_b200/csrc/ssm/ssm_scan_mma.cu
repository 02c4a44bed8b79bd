// ssm_scan_mma.cu -- selective scan over a prompt on the tensor cores (bf16 in and out):
//   S_t = exp(d_t A) S_{t-1} + d_t B_t (x) x_t,   y_t = C_t . S_t + D x_t.
//
// Mathematics.  Over a chunk of 64 tokens with a_i = sum_{k<=i} d_k A, from the state S before it,
//   y_i  = exp(a_i) C_i . S  +  sum_{j<=i} exp(a_i - a_j) d_j (C_i . B_j) x_j  +  D x_i
//   S'   = exp(a_63) S + sum_j (exp(a_63 - a_j) d_j x_j) (x) B_j
// so a chunk is four products.  All are taken transposed, with 128 channels p of one group's heads
// (128/P heads) down the 128 lanes of tensor memory:
//   G^T [j,i] = B C^T             both from shared memory, M = 64
//   Yb  [p,i] = S^T C^T           S^T in tensor memory as two bf16 pieces
//   Ya  [p,i] = X^T W^T           W[i,j] = exp(a_i - a_j) d_j G[i,j], two bf16 pieces in shared memory,
//                                 one product per head with the other heads' lanes switched off
//   dS  [p,n] = Xw^T B            Xw = exp(a_63 - a_j) d_j x_j in tensor memory, three bf16 pieces
// and y^T = exp(a_i) Yb + Ya + D x^T.  The tiles of x, B and C are used as they arrive by TMA, B and C in
// both roles; x is transposed on the way to registers (ldmatrix.trans) and y on the way back.
//
// Precision.  The state itself stays in fp32 registers and takes dS with one fused multiply-add
// per chunk (the tensor core's accumulation would shave a bit off a long-lived state every
// chunk).  Xw is exact in three pieces of 8 bits; S and W as operands of a bf16 result carry 16
// bits, 2^-16 of each value against the result's 2^-9.  Sums of d A are taken in 64 bits; a_i - a_j is the
// difference of two float pairs, so strong decay early in a chunk costs later tokens nothing.
//
// Work split.  One CTA per (sequence, 128 channels, segment of the sequence), chunks in order; 16
// warps do the elementwise work of a chunk, each on 32 channels x 16 tokens (or N/4 state columns), one
// warp feeds TMA, one issues MMAs, one computes step sizes and decays.  Per chunk the order
//   W -> [MMA Ya] Xw -> [MMA dS] y -> [MMA G of the next chunk] S -> [MMA Yb] ...
// puts elementwise work of the same warps behind every MMA's latency.
// Bound: issue slots of the elementwise work (about 500 instructions per warp and chunk).
#include <mutex>

#include "ssm_mma.cuh"

namespace ramnet {
namespace {

// Registers per thread by role: 20 warps launch with 96 each, and 2 x 80 + 2 x 128 + 64 = 5 x 96.
constexpr int kInRegs = 80, kOutRegs = 128, kMiscRegs = 64;
constexpr int kQ = 64;           // tokens per chunk
constexpr int kInWarps = 8;      // warps that prepare operands (W, Xw)
constexpr int kOutWarps = 8;     // warps that hold the state and write y
constexpr int kWarps = kInWarps + kOutWarps;
constexpr int kDtWarps = 2;      // warps that compute step sizes and decays, in alternate chunks
constexpr int kThreads = (kWarps + 2 + kDtWarps) * 32;
constexpr uint32_t kPatch = 2048;  // a warp's patch of y: 32 tokens x 32 channels, rows of 64 bytes in the 64-byte swizzle
constexpr size_t kSmemMax = 232448 - 1024;  // the rest: barriers

// per (stage, head) step sizes and decays of a chunk
struct Tok {
    float4 t[kQ];    // a_j log2(e) as a float pair, d_j, exp(a_63 - a_j) d_j
    float hi[kQ], lo[kQ];  // the same pair, by token
    float ein[kQ];   // exp(a_i)
    float w[kQ];     // exp(a_63 - a_j) d_j
    float dec, pad[3];     // exp(a_63)
};

enum Bar { kLanded = 0, kToks = 4, kEmpty = 8, kFixed = 12, kG, kW, kY, kYfree, kS, kXw, kDs = kXw + 2, kDsFree = kDs + 2, kDrain = kDsFree + 2, kBars };

struct Layout {
    int stages;
    uint32_t b_off, c_off, stage_bytes, w_off, stg_off, tok_off, total;
};

__host__ __device__ constexpr Layout layout_of(int N, int HP, bool out)
{
    const uint32_t nt = (N + 63) / 64 * 8192u;
    Layout l{};
    l.b_off = 16384;
    l.c_off = l.b_off + nt;
    l.stage_bytes = l.c_off + (out ? nt : 0);
    const uint32_t fixed = (out ? HP * 16384u + kOutWarps * kPatch : 0);
    l.stages = 4;
    while (l.stages > 2 && l.stages * (l.stage_bytes + HP * sizeof(Tok)) + fixed + 1024 > kSmemMax) --l.stages;
    l.w_off = l.stages * l.stage_bytes;
    l.stg_off = l.w_off + (out ? HP * 16384u : 0);
    l.tok_off = l.stg_off + (out ? kOutWarps * kPatch : 0);
    l.total = l.tok_off + l.stages * HP * static_cast<uint32_t>(sizeof(Tok)) + 1024;  // 1024: base alignment
    return l;
}

__device__ __forceinline__ float ex2(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

struct MmaMaps {
    CUtensorMap x, b, c, y;
};

// N state values, HP heads per 128 channels; OUT: outputs and final state, else what a segment adds to a
// zero state.
template <int N, int HP, bool OUT>
__global__ void __launch_bounds__(kThreads, 1) k_ssm_mma(const __grid_constant__ MmaMaps maps, const SsmParams p, int tiles)
{
    constexpr Layout L = layout_of(N, HP, OUT);
    constexpr int NB = OUT ? 1 : 2;  // buffers of Xw and dS
    // tensor-memory columns (G shares those of Ya; without outputs dS and Xw have two buffers)
    constexpr uint32_t cDs = 0, cShi = 128, cSlo = 192, cXw = 256, cYb = 384, cYa = 448;
    extern __shared__ unsigned char raw[];
    __shared__ __align__(8) uint64_t bar_mem[kBars];
    __shared__ uint32_t tmem_holder;
    __shared__ int abort_mem;
    __shared__ double log_mem[kDtWarps][HP];
    unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t s0 = smem_addr(sm), bars = smem_addr(bar_mem);
    Tok* toks = reinterpret_cast<Tok*>(sm + L.tok_off);
    volatile int* abort_flag = &abort_mem;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // which channels and tokens
    const int tile = static_cast<int>(blockIdx.x % tiles);
    const int bg = static_cast<int>(blockIdx.x / tiles);
    const int g = bg % p.G, b = bg / p.G, seg = blockIdx.y;
    const int hg = p.H / p.G, c0 = tile * 128, cend = hg * p.P;  // channels [c0, min(c0+128, cend)) of the group
    const SegRange r = seg_range(seq_len(p.lengths, b, p.T), seg, OUT ? p.split.seg_len : p.split.piece_len());
    const int nch = (r.last - r.first + kQ - 1) / kQ;
    const int head0 = c0 / p.P;  // first head, within the group

    auto bar = [&](int i) { return bars + 8u * i; };
    auto wait = [&](int i, uint32_t parity) {
        wait_phase(bars + 8u * i, parity, abort_flag, p.wait_ns);
    };

    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(bar_mem + kLanded + i, 1);
            mbar_init(bar_mem + kToks + i, 1);
            mbar_init(bar_mem + kEmpty + i, kOutWarps);
        }
        mbar_init(bar_mem + kFixed, 1);
        mbar_init(bar_mem + kG, 1);
        mbar_init(bar_mem + kDrain, 1);
        mbar_init(bar_mem + kW, kInWarps);
        mbar_init(bar_mem + kY, 1);
        mbar_init(bar_mem + kYfree, kOutWarps);
        mbar_init(bar_mem + kS, kOutWarps);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar_mem + kXw + i, kInWarps);
            mbar_init(bar_mem + kDs + i, 1);
            mbar_init(bar_mem + kDsFree + i, kOutWarps);
        }
        abort_mem = 0;
        fence_mbar_init_cluster();
    }
    if (warp == kWarps) tmem_alloc(&tmem_holder, 512);
    if (OUT) {  // the blocks of W above its diagonal stay zero
        uint4* w = reinterpret_cast<uint4*>(sm + L.w_off);
        for (uint32_t i = threadIdx.x; i < HP * 1024u; i += kThreads) w[i] = make_uint4(0, 0, 0, 0);
        fence_async_smem();
    }
    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
    const uint32_t tm = tmem_holder;

    const int q = warp & 3, part = (warp >> 2) & 1;                  // tensor-memory quadrant; half of the tokens or state columns
    const uint32_t tq = tm + (static_cast<uint32_t>(q) << 21);      // this warp's 32 lanes
    const int hw = HP == 4 ? q : HP == 2 ? q >> 1 : 0;              // head of its channels
    // ldmatrix row of this lane in a block of 16 tokens x 16 channels (and stmatrix row in a patch of y)
    const int row = 8 * (lane >> 4) + (lane & 7), pcol = 8 * ((lane >> 3) & 1);
    uint32_t xaddr[2];  // channels q*32 + half*16.., tokens part*32..
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int pp = q * 32 + half * 16 + pcol;
        xaddr[half] = s0 + (pp >> 6) * 8192 + (part * 32 + row) * 128 + ((((pp & 63) >> 3) ^ (row & 7)) << 4);
    }
    auto done = [&](int i) {  // this warp's part of hand-over i
        tmem_fence_before_sync();
        __syncwarp();
        if (lane == 0) arrive(bar(i));
    };

    if (warp < kInWarps) {
        // ------------------------------------------------------------ operands of the chunk: Xw, X^T and W
        regs_down<kInRegs>();
        int st = 0;
        uint32_t ph = 0;
        for (int c = 0; c < nch; ++c) {
            const Tok* tok = toks + st * HP;
            wait(kToks + st, ph);
            wait(kLanded + st, ph);
            if (r.last - r.first - c * kQ < kQ) wait(kFixed, 0);
            const int i = NB == 2 ? c & 1 : 0;
            // Xw's buffer: the product that read it is done
            if (c >= NB) wait(kDs + i, NB == 2 ? ((c >> 1) - 1) & 1 : (c - 1) & 1);
            tmem_fence_after_sync();
#pragma unroll 1
            for (int tg = 0; tg < 2; ++tg) {
                const uint32_t xw = tq + cXw + i * 96 + part * 16 + tg * 8;
                const float* w = tok[hw].w + part * 32 + tg * 16 + 2 * (lane & 3);
                const float2 w0 = *reinterpret_cast<const float2*>(w), w1 = *reinterpret_cast<const float2*>(w + 8);
                const F2 ww[2] = {f2(w0.x, w0.y), f2(w1.x, w1.y)};
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t xx[4];
                    ldsm_t(xaddr[half] + st * L.stage_bytes + tg * 2048, xx);
                    uint32_t piece[3][4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        F2 v = mul2(bf_pair(xx[k]), ww[k >> 1]);
                        piece[0][k] = peel(v);
                        piece[1][k] = peel(v);
                        piece[2][k] = pack_cut(v);
                    }
#pragma unroll
                    for (int s = 0; s < 3; ++s)
                        tmem_st_16x8(xw + (static_cast<uint32_t>(half) << 20) + s * 32, piece[s][0], piece[s][1], piece[s][2], piece[s][3]);
                }
            }
            tmem_wait_st();
            done(kXw + i);
            if constexpr (OUT) {
                wait(kG, c & 1);
                tmem_fence_after_sync();
                // tokens j of block q reach tokens i of blocks q..3; this warp takes every second of them
#pragma unroll 1
                for (int cb = q + part; cb < 4; cb += 2) {
                    float gv[8];
                    tmem_ld_16x16(tq + cYa + cb * 16, gv);
                    const int j = q * 16 + (lane >> 2), i0 = cb * 16 + 2 * (lane & 3);
                    tmem_wait_ld();
                    settle(gv);
#pragma unroll
                    for (int h = 0; h < HP; ++h) {
                        const Tok& tk = tok[h];
                        const float skip = (p.D && head0 + h < hg) ? p.D[g * hg + head0 + h] : 0.0f;
                        const uint32_t wbase = L.w_off + h * 16384 + j * 128 + (i0 & 7) * 2;
                        F2 hi[2], lo[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float2 a = *reinterpret_cast<const float2*>(tk.hi + i0 + 8 * k);
                            const float2 e = *reinterpret_cast<const float2*>(tk.lo + i0 + 8 * k);
                            hi[k] = f2(a.x, a.y);
                            lo[k] = f2(e.x, e.y);
                        }
#pragma unroll
                        for (int rb = 0; rb < 2; ++rb) {
                            const float4 tj = tk.t[j + 8 * rb];
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                float u, v;
                                un(add2(add2(hi[k], f2(-tj.x, -tj.x)), add2(lo[k], f2(-tj.y, -tj.y))), u, v);
                                const F2 e = mul2(f2(ex2(u), ex2(v)), f2(tj.z, tj.z));
                                F2 w = mul2(e, f2(gv[4 * k + 2 * rb], gv[4 * k + 2 * rb + 1]));
                                if (cb == q) {
                                    const int ii = i0 + 8 * k - (j + 8 * rb);
                                    un(w, u, v);
                                    // D x_i rides on the diagonal
                                    w = f2(ii > 0 ? u : ii == 0 ? u + skip : 0.0f, ii > -1 ? v : ii == -1 ? v + skip : 0.0f);
                                }
                                const uint32_t at = wbase + rb * 1024 + ((((i0 >> 3) + k) ^ (j & 7)) << 4);
                                *reinterpret_cast<uint32_t*>(sm + at) = peel(w);
                                *reinterpret_cast<uint32_t*>(sm + at + 8192) = pack_rn(w);
                            }
                        }
                    }
                }
                fence_async_smem();
                done(kW);
            }
            if (++st == L.stages) st = 0, ph ^= 1;
        }
    } else if (warp < kWarps) {
        // ------------------------------------------------------------ state and outputs
        regs_up<kOutRegs>();
        const int ch = c0 + q * 32 + lane;  // channel of this lane's state columns
        const bool mine = ch < cend;
        const int64_t bh = static_cast<int64_t>(b) * p.H + g * hg + ch / p.P;
        const int64_t np = static_cast<int64_t>(N) * p.P;
        const int pc = ch % p.P;
        constexpr int NC = N / 2;            // state columns per warp
        constexpr int NV = NC < 16 ? NC : 16;  // of them per tensor-memory access
        F2 S[NC / 2];
        {
            const float* from = nullptr;
            if (OUT && mine) {
                if (p.split.nseg > 1) from = p.seg_state + (bh * p.split.slots() + seg * p.split.sub) * np;
                else if (p.S_in) from = p.S_in + bh * np;
            }
            from = from ? from + static_cast<int64_t>(part) * NC * p.P + pc : nullptr;
#pragma unroll
            for (int k = 0; k < NC / 2; ++k) {
                S[k] = from ? f2(from[0], from[p.P]) : f2(0.0f, 0.0f);
                if (from) from += 2 * p.P;
                if (k % 8 == 7) asm volatile("" ::: "memory");  // few loads, and few addresses, at a time
            }
        }
        auto put_state = [&](int k0) {  // state columns k0 .. k0+NV as two pieces
            uint32_t hi[NV / 2], lo[NV / 2];
#pragma unroll
            for (int k = 0; k < NV / 2; ++k) {
                F2 v = S[k0 / 2 + k];
                hi[k] = peel(v);
                lo[k] = pack_rn(v);
            }
            tmem_st_cols<NV / 2>(tq + cShi + (part * NC + k0) / 2, hi);
            tmem_st_cols<NV / 2>(tq + cSlo + (part * NC + k0) / 2, lo);
        };
        if (OUT && nch > 0) {
#pragma unroll
            for (int k0 = 0; k0 < NC; k0 += NV) put_state(k0);
            tmem_wait_st();
            done(kS);
        }
        // this warp's patch of y: 32 tokens x 32 channels
        const uint32_t patch = L.stg_off + (warp - kInWarps) * kPatch;
        uint32_t paddr[2];  // stmatrix row of this lane, channels half*16..
#pragma unroll
        for (int half = 0; half < 2; ++half) paddr[half] = s0 + patch + row * 64 + (((half * 2 + (pcol >> 3)) ^ ((row >> 1) & 3)) << 4);
        const bool ych = c0 + q * 32 < cend;
        int st = 0;
        uint32_t ph = 0;
        for (int c = 0; c < nch; ++c) {
            const Tok& tok = toks[st * HP + hw];
            wait(kToks + st, ph);
            if constexpr (OUT) {
                if (lane == 0) store_read_done();  // the patch is free
                __syncwarp();
                wait(kY, c & 1);
                tmem_fence_after_sync();
                const uint32_t ty = tq + part * 32;
                float yb[2][8], ya[2][8];
                tmem_ld_16x16(ty + cYb, yb[0]);
                tmem_ld_16x16(ty + cYa, ya[0]);
#pragma unroll
                for (int k4 = 0; k4 < 4; ++k4) {  // 16 tokens k4/2, 16 channels k4%2; the next loads run meanwhile
                    const int now = k4 & 1, tg = k4 >> 1;
                    const float* e = tok.ein + part * 32 + tg * 16 + 2 * (lane & 3);
                    const float2 e0 = *reinterpret_cast<const float2*>(e), e1 = *reinterpret_cast<const float2*>(e + 8);
                    tmem_wait_ld();
                    settle(yb[now]);
                    settle(ya[now]);
                    if (k4 < 3) {
                        const uint32_t at = ty + (static_cast<uint32_t>((k4 + 1) & 1) << 20) + ((k4 + 1) >> 1) * 16;
                        tmem_ld_16x16(at + cYb, yb[now ^ 1]);
                        tmem_ld_16x16(at + cYa, ya[now ^ 1]);
                    } else {
                        done(kYfree);
                    }
                    uint32_t o[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {  // 8 tokens k/2, 8 channels k%2
                        const int at = 4 * (k >> 1) + 2 * (k & 1);
                        const float2 ee = k < 2 ? e0 : e1;
                        o[k] = pack_rn(fma2(f2(ee.x, ee.y), f2(yb[now][at], yb[now][at + 1]), f2(ya[now][at], ya[now][at + 1])));
                    }
                    stsm_t(paddr[k4 & 1] + tg * 1024, o[0], o[1], o[2], o[3]);
                }
                const int tok0 = r.first + c * kQ + part * 32, left = r.last - tok0;
                if (left >= 32) {
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0 && ych) tma_store_3d(&maps.y, g * cend + c0 + q * 32, tok0, b, s0 + patch);
                } else {  // rows behind the sequence are not this call's to write
                    __syncwarp();
                    const int64_t yrow = static_cast<int64_t>(p.H) * p.P;
                    __nv_bfloat16* yp = reinterpret_cast<__nv_bfloat16*>(p.y) + (static_cast<int64_t>(b) * p.T + tok0) * yrow + g * cend + c0 +
                                        q * 32 + (lane & 3) * 8;
#pragma unroll 1
                    for (int t = lane >> 2; t < left && ych; t += 8)
                        *reinterpret_cast<uint4*>(yp + t * yrow) =
                            *reinterpret_cast<const uint4*>(sm + patch + t * 64 + (((lane & 3) ^ ((t >> 1) & 3)) << 4));
                    __syncwarp();
                }
            }
            // S' = dec S + dS
            const int i = NB == 2 ? c & 1 : 0;
            wait(kDs + i, NB == 2 ? (c >> 1) & 1 : c & 1);
            tmem_fence_after_sync();
            const F2 dec = f2(tok.dec, tok.dec);
            const uint32_t td = tq + cDs + i * 128 + part * NC;
            float d[2][NV];
            tmem_ld_cols<NV>(td, d[0]);
#pragma unroll
            for (int k0 = 0; k0 < NC; k0 += NV) {
                const int now = (k0 / NV) & 1;
                tmem_wait_ld();
                settle(d[now]);
                if (k0 + NV < NC) tmem_ld_cols<NV>(td + k0 + NV, d[now ^ 1]);
                else done(kDsFree + i);  // the next chunk's dS may come while the state is split below
#pragma unroll
                for (int k = 0; k < NV / 2; ++k) S[k0 / 2 + k] = fma2(S[k0 / 2 + k], dec, f2(d[now][2 * k], d[now][2 * k + 1]));
            }
            if (OUT && c + 1 < nch) {
#pragma unroll
                for (int k0 = 0; k0 < NC; k0 += NV) put_state(k0);
            }
            if (OUT && c + 1 < nch) {
                tmem_wait_st();
                done(kS);
            }
            __syncwarp();
            if (lane == 0) arrive(bar(kEmpty + st));
            if (++st == L.stages) st = 0, ph ^= 1;
        }
        if (OUT && lane == 0) store_done();
        float* to = nullptr;
        if (mine) {
            if (!OUT) to = p.seg_state + (bh * p.split.slots() + seg) * np;
            else if (seg == p.split.nseg - 1) to = p.S_out + bh * np;
        }
        if (to) {
            to += static_cast<int64_t>(part) * NC * p.P + pc;
#pragma unroll
            for (int k = 0; k < NC / 2; ++k) {
                un(S[k], to[0], to[p.P]);
                to += 2 * p.P;
            }
        }
    } else if (warp == kWarps) {
        // ------------------------------------------------------------ TMA
        regs_down<kMiscRegs>();
        int issued = 0;
        for (int c = 0; c < nch; ++c) {
            const int st = c % L.stages;
            if (c >= L.stages) wait(kEmpty + st, ((c / L.stages) - 1) & 1);
            if (*abort_flag) break;
            const int t0 = r.first + c * kQ, nv = min(kQ, r.last - t0);
            const uint32_t base = s0 + st * L.stage_bytes;
            if (lane == 0) {
                arrive_tx(bar(kLanded + st), L.stage_bytes);
                tma_load_3d(base, &maps.x, g * cend + c0, t0, b, bar(kLanded + st));
                tma_load_3d(base + 8192, &maps.x, g * cend + c0 + 64, t0, b, bar(kLanded + st));
#pragma unroll
                for (int k = 0; k < (N + 63) / 64; ++k) {
                    tma_load_4d(base + L.b_off + k * 8192, &maps.b, k * 64, g, t0, b, bar(kLanded + st));
                    if (OUT) tma_load_4d(base + L.c_off + k * 8192, &maps.c, k * 64, g, t0, b, bar(kLanded + st));
                }
            }
            issued = c + 1;
            if (nv < kQ) {
                // rows behind the sequence may hold anything: zeros in their place
                wait(kLanded + st, (c / L.stages) & 1);
                for (uint32_t i = lane; i < L.stage_bytes / 16; i += 32)
                    if (static_cast<int>((i >> 3) & 63) >= nv) *reinterpret_cast<uint4*>(sm + st * L.stage_bytes + i * 16) = make_uint4(0, 0, 0, 0);
                fence_async_smem();
                __syncwarp();
                if (lane == 0) arrive(bar(kFixed));
            }
        }
        // no copy may land in this block's memory after it has gone (bounded, also after an abort)
        if (*abort_flag && lane == 0) {
            const uint64_t t_end = now_ns() + 2000000000ull;
            for (int c = issued > L.stages ? issued - L.stages : 0; c < issued; ++c)
                for (uint32_t it = 0; it < kSpinLimit; ++it)
                    if (try_wait(bar(kLanded + c % L.stages), (c / L.stages) & 1) || now_ns() > t_end) break;
        }
    } else if (warp == kWarps + 1) {
        // ------------------------------------------------------------ MMA issue (whole warp, one lane issues)
        regs_down<kMiscRegs>();
        constexpr uint32_t wG = mma_word(64, 64, false, false), wYb = mma_word(128, 64, false, false);
        constexpr uint32_t wYa = mma_word(128, 64, true, true), wDs = mma_word(128, N, false, true);
        const Desc wdesc = desc_of(s0 + L.w_off, 8192);
        auto add_chunk = [&](int c, int st) {  // dS of chunk c
            const Desc down = desc_of(s0 + st * L.stage_bytes + L.b_off, 8192);  // B as [j, n]: contraction down the rows
            const int i = NB == 2 ? c & 1 : 0;
            wait(kXw + i, NB == 2 ? (c >> 1) & 1 : c & 1);
            if (c >= NB) wait(kDsFree + i, NB == 2 ? ((c >> 1) - 1) & 1 : (c - 1) & 1);
            tmem_fence_after_sync();
            if (elect_one()) {
#pragma unroll
                for (int s = 2; s >= 0; --s)  // the small pieces first
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_ts(tm + cDs + i * 128, tm + cXw + i * 96 + s * 32 + k * 8, down + k * 2048, wDs, s < 2 || k > 0);
                mma_commit(bar(kDs + i));
            }
            __syncwarp();
        };
        int st = 0;
        uint32_t ph = 0;
        for (int c = 0; c < nch; ++c) {
            const Desc down = desc_of(s0 + st * L.stage_bytes, 8192);  // x as [j, p]: contraction down the rows
            const Desc along = desc_of(s0 + st * L.stage_bytes, 16);   // contraction along the rows: B and C as [., n]
            wait(kLanded + st, ph);
            if (r.last - r.first - c * kQ < kQ) wait(kFixed, 0);
            if (*abort_flag) break;
            if constexpr (OUT) {
                if (c > 0) wait(kYfree, (c - 1) & 1);
                tmem_fence_after_sync();
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < N / 16; ++k)
                        mma_ss(tm + cYa, along + (L.b_off + (k >> 2) * 8192 + (k & 3) * 32), along + (L.c_off + (k >> 2) * 8192 + (k & 3) * 32),
                               wG, k > 0);
                    mma_commit(bar(kG));
                }
                __syncwarp();
            }
            if constexpr (OUT) {
                add_chunk(c, st);
                wait(kS, c & 1);
                tmem_fence_after_sync();
                if (elect_one()) {
#pragma unroll
                    for (int s = 0; s < 2; ++s)
#pragma unroll
                        for (int k = 0; k < N / 16; ++k)
                            mma_ts(tm + cYb, tm + (s ? cShi : cSlo) + k * 8, along + (L.c_off + (k >> 2) * 8192 + (k & 3) * 32), wYb, s + k > 0);
                }
                __syncwarp();
                wait(kW, c & 1);
                tmem_fence_after_sync();
                if (elect_one()) {
#pragma unroll
                    for (int h = 0; h < HP; ++h)
#pragma unroll
                        for (int s = 0; s < 2; ++s)
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const Desc da = down + k * 2048, db = wdesc + (h * 16384 + (s ? 0 : 8192) + k * 2048);
                                if constexpr (HP == 1) {
                                    mma_ss(tm + cYa, da, db, wYa, s + k > 0);
                                } else {
                                    auto off = [&](int qq) { return (HP == 4 ? qq : qq >> 1) == h ? 0u : 0xffffffffu; };
                                    mma_ss_masked(tm + cYa, da, db, wYa, off(0), off(1), off(2), off(3), s + k > 0);
                                }
                            }
                    mma_commit(bar(kY));
                }
                __syncwarp();
            }
            if constexpr (!OUT) add_chunk(c, st);
            if (++st == L.stages) st = 0, ph ^= 1;
        }
        if (*abort_flag && lane == 0) {  // tensor memory is given back only when nothing writes to it
            const uint64_t t_end = now_ns() + 2000000000ull;
            mma_commit(bar(kDrain));
            for (uint32_t it = 0; it < kSpinLimit; ++it)
                if (try_wait(bar(kDrain), 0) || now_ns() > t_end) break;
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ step sizes and decays
        regs_down<kMiscRegs>();
        const int first = warp - (kWarps + 2);
        const __nv_bfloat16* dt = reinterpret_cast<const __nv_bfloat16*>(p.dt) + b * p.dts.b + (g * hg + head0) * p.dts.h;
        if (!OUT && lane < HP) log_mem[first][lane] = 0.0;
        __syncwarp();
        uint32_t raw_dt[2];  // the step inputs of the next (chunk, head), loaded one ahead
        auto fetch = [&](int c, int h) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int t = r.first + c * kQ + 2 * lane + k;
                raw_dt[k] = (c < nch && head0 + h < hg && t < r.last) ? __bfloat16_as_ushort(dt[t * p.dts.t + h * p.dts.h]) : 0u;
            }
        };
        fetch(first, 0);
#pragma unroll 1
        for (int c = first; c < nch; c += kDtWarps) {
            const int st = c % L.stages;
            if (c >= L.stages) wait(kEmpty + st, ((c / L.stages) - 1) & 1);
            if (*abort_flag) break;
#pragma unroll 1
            for (int h = 0; h < HP; ++h) {
                const bool real = head0 + h < hg;
                const double A = real ? static_cast<double>(p.A[g * hg + head0 + h]) : 0.0;
                const float bias = (real && p.dt_bias) ? p.dt_bias[g * hg + head0 + h] : 0.0f;
                float d[2];
#pragma unroll
                for (int k = 0; k < 2; ++k)  // a token that is not there neither decays nor writes
                    d[k] = (real && r.first + c * kQ + 2 * lane + k < r.last)
                               ? step_size(__uint_as_float(raw_dt[k] << 16), bias, p.softplus, p.dt_min, p.dt_max)
                               : 0.0f;
                if (h + 1 < HP) fetch(c, h + 1);
                else fetch(c + kDtWarps, 0);
                const double a0 = d[0] * A, a1 = d[1] * A;
                double sum = a0 + a1;
#pragma unroll 1
                for (int o = 1; o < 32; o <<= 1) {
                    const double up = __shfl_up_sync(0xffffffffu, sum, o);
                    if (lane >= o) sum += up;
                }
                const double total = __shfl_sync(0xffffffffu, sum, 31);
                Tok& tk = toks[st * HP + h];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const double cum = k ? sum : sum - a1;
                    const double l2 = cum * 1.4426950408889634074;
                    const float hi = static_cast<float>(l2), lo = static_cast<float>(l2 - static_cast<double>(hi));
                    const float w = d[k] * expf(static_cast<float>(total - cum));
                    const int j = 2 * lane + k;
                    tk.t[j] = make_float4(hi, lo, d[k], w);
                    tk.hi[j] = hi;
                    tk.lo[j] = lo;
                    tk.ein[j] = expf(static_cast<float>(cum));
                    tk.w[j] = w;
                }
                const float dec = static_cast<float>(exp(total));
                if (lane == 0) {
                    tk.dec = dec;
                    if (!OUT) log_mem[first][h] += total;
                }
            }
            __syncwarp();
            if (lane == 0) arrive(bar(kToks + st));
        }
    }
    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
    if (warp == kWarps) tmem_dealloc(tm, 512);
    if (threadIdx.x == 0 && *abort_flag) set_status(p.status, kDevTimeout);
    if (!OUT && threadIdx.x < HP && head0 + static_cast<int>(threadIdx.x) < hg && c0 % p.P == 0) {
        double sum = 0.0;
        for (int k = 0; k < kDtWarps; ++k) sum += log_mem[k][threadIdx.x];
        p.seg_decay[(static_cast<int64_t>(b) * p.H + g * hg + head0 + threadIdx.x) * p.split.pieces() + seg] = static_cast<float>(exp(sum));
    }
}

// ------------------------------------------------------------------ host side

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder()
{
    static EncodeFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

// Boxes of `rows` tokens x `inner` elements (64 with the 128-byte swizzle, 32 with the 64-byte one) of a bf16 operand: dims inner (contiguous), then (size, stride in elements).
bool encode(CUtensorMap* map, const void* base, int rank, const int64_t* size, const int64_t* stride, int inner = 64, int rows = 64)
{
    cuuint64_t dims[4], bytes[3];
    cuuint32_t box[4], one[4] = {1, 1, 1, 1};
    for (int i = 0; i < rank; ++i) {
        dims[i] = static_cast<cuuint64_t>(size[i]);
        box[i] = i == 0 ? inner : i == rank - 2 ? rows : 1;
        // the stride of a single element is never used
        if (i > 0) bytes[i - 1] = size[i] == 1 ? 16 : static_cast<cuuint64_t>(stride[i]) * 2;
    }
    return encoder()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<cuuint32_t>(rank), const_cast<void*>(base), dims, bytes, box, one,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, inner == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool map_operands(const SsmParams& p, MmaMaps* m)
{
    const int64_t xsize[3] = {static_cast<int64_t>(p.H) * p.P, p.T, p.B}, xstr[3] = {1, p.xs.t, p.xs.b};
    const int64_t bsize[4] = {p.N, p.G, p.T, p.B}, bstr[4] = {1, p.bs.h, p.bs.t, p.bs.b}, cstr[4] = {1, p.cs.h, p.cs.t, p.cs.b};
    const int64_t ystr[3] = {1, xsize[0], xsize[0] * p.T};
    return encode(&m->y, p.y, 3, xsize, ystr, 32, 32) && encode(&m->x, p.x, 3, xsize, xstr) && encode(&m->b, p.Bm, 4, bsize, bstr) && encode(&m->c, p.Cm, 4, bsize, cstr);
}

template <int N, int HP, bool OUT>
cudaError_t go(const SsmParams& p, const MmaMaps& m, int tiles, int segs, cudaStream_t s)
{
    constexpr Layout L = layout_of(N, HP, OUT);
    static_assert(kThreads == 640, "register split");
    static_assert(L.total <= kSmemMax, "shared memory");
    auto kern = k_ssm_mma<N, HP, OUT>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(L.total));
    if (e != cudaSuccess) return e;
    kern<<<dim3(static_cast<unsigned>(p.B) * p.G * tiles, segs), kThreads, L.total, s>>>(m, p, tiles);
    return cudaGetLastError();
}

template <int N, int HP>
cudaError_t all(const SsmParams& p, const MmaMaps& m, cudaStream_t s)
{
    const int tiles = (p.H / p.G * p.P + 127) / 128;
    if (p.split.nseg > 1) {
        cudaError_t e = go<N, HP, false>(p, m, tiles, p.split.pieces(), s);
        if (e == cudaSuccess) e = launch_ssm_chain(p, s);
        if (e != cudaSuccess) return e;
    }
    return go<N, HP, true>(p, m, tiles, p.split.nseg, s);
}

template <int N>
cudaError_t pick(const SsmParams& p, const MmaMaps& m, cudaStream_t s)
{
    if (p.P == 32) return all<N, 4>(p, m, s);
    if (p.P == 64) return all<N, 2>(p, m, s);
    return all<N, 1>(p, m, s);
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
// TMA wants strides of whole 16 bytes below 2^40; a stride of nothing (an expanded view) is left out
bool ok_stride(int64_t n, int64_t size) { return size == 1 || (n > 0 && n % 8 == 0 && n < (1ll << 39)); }

}  // namespace

bool ssm_mma_takes(const SsmParams& p)
{
    if (!p.in_bf16 || !p.out_bf16 || p.P < 32 || p.N > 128) return false;
    if (!al16(p.x) || !al16(p.Bm) || !al16(p.Cm)) return false;
    if (p.H > 1 && p.xs.h != p.P) return false;  // heads side by side: one row of channels per token
    if (!ok_stride(p.xs.t, p.T) || !ok_stride(p.xs.b, p.B)) return false;
    if (!ok_stride(p.bs.h, p.G) || !ok_stride(p.bs.t, p.T) || !ok_stride(p.bs.b, p.B)) return false;
    if (!ok_stride(p.cs.h, p.G) || !ok_stride(p.cs.t, p.T) || !ok_stride(p.cs.b, p.B)) return false;
    return encoder() != nullptr;
}

cudaError_t launch_ssm_mma(const SsmParams& p, cudaStream_t s)
{
    MmaMaps m;
    if (!map_operands(p, &m)) return cudaErrorInvalidValue;
    switch (p.N) {
        case 16: return pick<16>(p, m, s);
        case 32: return pick<32>(p, m, s);
        case 64: return pick<64>(p, m, s);
        case 128: return pick<128>(p, m, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace ramnet
