// ssm_scan_mma.cu -- selective scan over a prompt on the tensor cores (bf16 in and out):
//   S_t = exp(d_t A) S_{t-1} + d_t B_t (x) x_t,   y_t = C_t . S_t + D x_t.
//
// Mathematics.  Over a chunk of 64 tokens with a_i = sum_{k<=i} d_k A, from the state S before it,
//   y_i  = exp(a_i) C_i . S  +  sum_{j<=i} exp(a_i - a_j) d_j (C_i . B_j) x_j  +  D x_i
//   S'   = exp(a_63) S + sum_j (exp(a_63 - a_j) d_j x_j) (x) B_j
// so a chunk is four products.  All are taken transposed, with 128 channels p of one group's heads
// (128/P heads) down the 128 lanes of tensor memory:
//   G^T [j,i] = B C^T      bf16, both from shared memory, M = 64
//   Ya  [p,i] = X^T W^T    W[i,j] = exp(a_i - a_j) d_j G[i,j] (+ D on the diagonal) as two bf16 pieces in shared
//                          memory, one product per head with the other heads' lanes switched off
//   Yb  [p,i] = S^T C^T    S^T in tensor memory as two bf16 pieces
//   dS  [p,n] = Xw^T B     Xw = exp(a_63 - a_j) d_j x_j in tensor memory as three bf16 pieces
// and y^T = exp(a_i) Yb + Ya.  The tiles of x, B and C are used as they arrive by TMA, B and C in both
// roles; x is transposed on the way to registers (ldmatrix.trans) and y on the way back.
//
// Precision.  The state itself stays in fp32 registers and takes dS with one fused multiply-add
// per chunk (the tensor core's accumulation would shave a bit off a long-lived state every
// chunk).  Xw is exact in three pieces of 8 bits.  As operands of a bf16 result W and S carry two pieces: 2^-16 of each
// value, against the result's own 2^-9 (0.3% of the results become the neighbouring bf16 value; the error against 64 bits is
// 1.658e-3 either way, the rounding of the result).  Sums of d A are taken in 64 bits; a_i - a_j is the
// difference of two float pairs within a block of 16 tokens, and between blocks a product of factors that meet at
// block ends, so strong decay early in a chunk costs later tokens nothing.
//
// Work split.  A first small launch turns dt into step sizes and decays by chunk (k_ssm_decay).  Then one CTA per
// (sequence, 128 channels, segment of the sequence), chunks in order, warps by role:
//   0-7   operands: W, X^T, Xw, then half of the outputs;   8-15  state (32 channels x N/2 values each), half of the outputs;
//   16    TMA loads and stores;  18 issues G and dS, 19 Ya and Yb.
// The loops over chunks chain W -> Ya, Yb -> outputs and state -> Yb; the rest overlaps.  Launches follow one another as
// programmatic dependents.
//
// What is no number spreads forward in time only.  B, C and step sizes meet other tokens through W alone, whose upper triangle
// is selected, not multiplied; but x_j meets every W[i,j] of its chunk in Ya, and 0 NaN is NaN.  So x that is no number is
// taken as 0, and its channel's outputs and final state from that token on are set to NaN.  (Looking for it costs 2% of a
// prompt's time; 20% where a warp of its own reads every chunk of x for it before the others may.)
//
// The code of all roles has to stay within the instruction cache: with the loops fully unrolled (72 KB) every role
// waited for instructions and a prompt took a third longer; unrolling W alone costs 3%.
// Measured, B4 T16384 H16 P128 N128: 318 us over one set of inputs, 360 to 373 over sets in turn (574 MB: 87 us at the copy
// bandwidth; token by token in registers 14 ms).
// About 3700 cycles per chunk, of which the tensor pipe works 1900, shared memory 2100, HBM 1400.  Bound: the
// operand warps of the first quadrant, whose diagonal and off-diagonal blocks of W take 1300 cycles of issue and latency
// between a chunk's G and its Ya.
// B8 T4096 H8 P128 N128: 94 to 105 us with 2 segments per sequence; B6 T1021 H24 P64 N64 in 2 groups: 39 to 42 us.
#include <climits>

#include "ssm_mma.cuh"

namespace ramnet {
namespace {

// Registers per thread by role: 20 warps launch with 96 each, and 2 x 88 + 2 x 128 + 48 = 5 x 96.
constexpr int kInRegs = 88, kOutRegs = 128, kMiscRegs = 48;
constexpr int kQ = kChunk;       // tokens per chunk
constexpr int kInWarps = 8, kOutWarps = 8, kWarps = kInWarps + kOutWarps;
constexpr int kLoadWarp = 16, kMmaWarp = 18;
constexpr int kThreads = 20 * 32;
constexpr uint32_t kPatch = 4096;  // y of 64 tokens x 32 channels, rows of 64 bytes in the 64-byte swizzle
constexpr size_t kSmemMax = 232448 - 1024;  // the rest: barriers

// Hand-overs.  Where a side may run two chunks ahead of the other, chunks alternate between two barriers of a kind;
// elsewhere each side waits for the other before its next, so no waiting warp is ever more than a phase behind.
enum Bar { kLanded = 0, kEmpty = 4, kFixed = 8, kG, kW, kY, kYfree, kS, kOut, kPatchFree = kOut + 2, kXw = kPatchFree + 2, kDs = kXw + 2, kDsFree = kDs + 2,
           kDrain = kDsFree + 2, kBars = kDrain + 2 };

// Buffers of W and of the patch of y: two for one head per 128 channels; with more, the memory goes to W itself.
__host__ __device__ constexpr int buffers(int HP) { return HP == 1 ? 2 : 1; }

struct Layout {
    int stages;
    uint32_t b_off, c_off, stage_bytes, w_off, patch_off, tok_off, total;
};

__host__ __device__ constexpr Layout layout_of(int N, int HP, bool out)
{
    const uint32_t nt = (N + 63) / 64 * 8192u;
    Layout l{};
    l.b_off = 16384;
    l.c_off = l.b_off + nt;
    l.stage_bytes = l.c_off + (out ? nt : 0);
    const uint32_t w = out ? buffers(HP) * HP * 16384u : 0, patch = out ? buffers(HP) * 4 * kPatch : 0;
    const uint32_t tok = HP * static_cast<uint32_t>(sizeof(ChunkTok));
    l.stages = 4;
    while (l.stages > 2 && l.stages * (l.stage_bytes + tok) + w + patch + 1024 > kSmemMax) --l.stages;
    l.w_off = l.stages * l.stage_bytes;
    l.patch_off = l.w_off + w;
    l.tok_off = l.patch_off + patch;
    l.total = l.tok_off + l.stages * tok + 1024;  // 1024: base alignment
    return l;
}

__device__ __forceinline__ float ex2(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// Step sizes and decays of every chunk: one warp per (sequence, head, chunk), two tokens per lane, sums in 64 bits.
__global__ void __launch_bounds__(256) k_ssm_decay(const SsmParams p, int chunks, int64_t work)
{
    let_next();
    const int64_t id = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (id >= work) return;
    const int lane = threadIdx.x & 31;
    // neighbouring warps take neighbouring heads, whose dt share sectors
    const int h = static_cast<int>(id % p.H);
    const int64_t bc = id / p.H;
    const int c = static_cast<int>(bc % chunks), b = static_cast<int>(bc / chunks);
    const int len = seq_len(p.lengths, b, p.T), t0 = c * kQ;
    if (t0 >= len) return;
    if (!dcheck(b < p.B && len <= p.T, p.status)) return;
    const float bias = p.dt_bias ? p.dt_bias[h] : 0.0f;
    const double A = static_cast<double>(p.A[h]) * 1.4426950408889634074;
    float d[2];
    double l[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int t = t0 + 2 * lane + k;
        d[k] = 0.0f, l[k] = 0.0;  // a token that is not there neither decays nor writes
        if (t < len) {
            d[k] = step_size(load_in(p.dt, static_cast<size_t>(b * p.dts.b + t * p.dts.t + h * p.dts.h), 1), bias, p.softplus, p.dt_min, p.dt_max);
            // 2^-1024 leaves nothing of any fp32 state: what decays further is taken as that much, so that sums of 64 tokens
            // stay well within what `hi` and `lo` hold (past 3.4e38 their sum is no number; at 1e12 it is off by 4e-3).
            // What is no number stays none.
            l[k] = d[k] * A;
            if (l[k] == l[k]) l[k] = fmin(fmax(l[k], -1024.0), 1024.0);
        }
    }
    double sum = l[0] + l[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double up = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += up;
    }
    double before = __shfl_up_sync(0xffffffffu, sum, 1);  // up to this lane's tokens, without them: its second may be no number
    if (lane == 0) before = 0.0;
    const double total = __shfl_sync(0xffffffffu, sum, 31);
    const double blk_end = __shfl_sync(0xffffffffu, sum, lane | 7);
    double blk_start = __shfl_sync(0xffffffffu, sum, ((lane & 24) - 1) & 31);
    if (lane < 8) blk_start = 0.0;
    const double end1 = __shfl_sync(0xffffffffu, sum, 23), end0 = __shfl_sync(0xffffffffu, sum, 7);
    ChunkTok& tk = p.toks[(static_cast<int64_t>(b) * p.H + h) * chunks + c];
    float hi[2], lo[2], e[2], w[2], u[2], v[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const double cum = k ? sum : before + l[0];
        hi[k] = static_cast<float>(cum);
        lo[k] = static_cast<float>(cum - static_cast<double>(hi[k]));
        e[k] = exp2f(hi[k]);
        w[k] = d[k] * exp2f(static_cast<float>(total - cum));
        u[k] = exp2f(static_cast<float>(cum - blk_start));
        v[k] = d[k] * exp2f(static_cast<float>(blk_end - cum));
    }
    auto put = [&](float* at, const float (&x)[2]) { reinterpret_cast<float2*>(at)[lane] = make_float2(x[0], x[1]); };
    put(tk.hi, hi);
    put(tk.lo, lo);
    put(tk.d, d);
    put(tk.ein, e);
    put(tk.w, w);
    put(tk.u, u);
    put(tk.v, v);
    if (lane == 0) {
        tk.dec = exp2_of(total);
        tk.blk[2] = exp2f(static_cast<float>(end1 - end0));
        tk.total = total;
    }
    if (lane == 8 || lane == 16) tk.blk[(lane >> 3) - 1] = exp2f(static_cast<float>(blk_end - blk_start));
}

struct MmaMaps {
    CUtensorMap x, b, c, y;
};

// N state values, heads of P channels, HP of them per 128 channels; OUT: outputs and final state, else what a piece
// of the sequence adds to a zero state.
template <int N, int P, bool OUT>
__global__ void __launch_bounds__(kThreads, 1) k_ssm_mma(const __grid_constant__ MmaMaps maps, const SsmParams p, int tiles)
{
    constexpr int HP = P >= 128 ? 1 : 128 / P;
    constexpr Layout L = layout_of(N, HP, OUT);
    constexpr int NBUF = buffers(HP);
    constexpr int HALVES = OUT && N == 128 ? 2 : 1;  // dS comes in halves of 64 columns where tensor memory is short
    // tensor-memory columns
    constexpr uint32_t cDs = 0, cShi = 64, cSlo = 128, cXw = OUT ? 192 : 256, cX = 288, cYb = 320, cYa = 384, cG = 448;
    extern __shared__ unsigned char raw[];
    __shared__ __align__(8) uint64_t bar_mem[kBars];
    __shared__ uint32_t tmem_holder;
    __shared__ __align__(8) int limit_mem[2];
    __shared__ int first_bad[128], any_bad_mem;  // per channel, its first token whose x is no number; whether there is one
    unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t s0 = smem_addr(sm), bars = smem_addr(bar_mem);
    ChunkTok* toks = reinterpret_cast<ChunkTok*>(sm + L.tok_off);
    volatile int* abort_flag = limit_mem;
    const uint32_t limit_addr = smem_addr(limit_mem);
    volatile int* any_bad = &any_bad_mem;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // which channels and tokens
    const int tile = static_cast<int>(blockIdx.x % tiles);
    const int bg = static_cast<int>(blockIdx.x / tiles);
    const int g = bg % p.G, b = bg / p.G, seg = blockIdx.y;
    const int hg = p.H / p.G, c0 = tile * 128, cend = hg * P;  // channels [c0, min(c0+128, cend)) of the group
    const SegRange r = seg_range(seq_len(p.lengths, b, p.T), seg, OUT ? p.split.seg_len : p.split.piece_len());
    const int nch = (r.last - r.first + kQ - 1) / kQ;
    const bool ragged = (r.last - r.first) % kQ != 0;  // the last chunk is not full
    const int head0 = c0 / P;                          // first head, within the group
    // (segments start with a chunk; the workspace holds (T + 63) / 64 of them per head)
    if (!dcheck(b < p.B && c0 < cend && head0 < hg && segment_fits(p, r, seg, OUT) && (nch == 0 || r.first % kQ == 0) &&
                    r.first / kQ + nch <= (p.T + kQ - 1) / kQ, p.status))
        return;

    auto bar = [&](int i) { return bars + 8u * i; };
    auto wait = [&](int i, uint32_t parity) { wait_phase(bars + 8u * i, parity, limit_addr); };

    if (threadIdx.x == 0) {
        for (int i = 0; i < kBars; ++i) {
            int count = 1;  // a commit, a copy or one warp
            if (i == kS) count = kOutWarps;
            if ((i >= kEmpty && i < kEmpty + 4) || i == kYfree || i == kOut || i == kOut + 1) count = OUT ? kWarps : kOutWarps;
            if (i == kW || i == kXw || i == kXw + 1) count = kInWarps;
            if (i == kDsFree || i == kDsFree + 1) count = kOutWarps / HALVES;
            mbar_init(bar_mem + i, count);
        }
        limit_mem[0] = p.poll_cost > kWaitNs;  // not even one: no wait waits, and the kernel gives up
        limit_mem[1] = p.poll_cost;
        any_bad_mem = 0;
        fence_mbar_init_cluster();
    }
    if (OUT && threadIdx.x < 128) first_bad[threadIdx.x] = INT_MAX;
    if (warp == kMmaWarp) tmem_alloc(&tmem_holder, 512);
    if (OUT) {  // the blocks of W above its diagonal stay zero
        uint4* w = reinterpret_cast<uint4*>(sm + L.w_off);
        for (uint32_t i = threadIdx.x; i < NBUF * HP * 1024u; i += kThreads) w[i] = make_uint4(0, 0, 0, 0);
        fence_async_smem();
    }
    if (!OUT) let_next();
    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
    after_before();
    constexpr uint32_t tm = 0;  // where an allocation of all 512 columns starts

    const int q = warp & 3, part = (warp >> 2) & 1;             // tensor-memory quadrant; half of the tokens or state columns
    const uint32_t tq = tm + (static_cast<uint32_t>(q) << 21);  // this warp's 32 lanes
    const int hw = HP == 4 ? q : HP == 2 ? q >> 1 : 0;          // head of its channels
    // ldmatrix row of this lane in a block of 16 tokens x 16 channels (and stmatrix row of a patch of y)
    const int row = 8 * (lane >> 4) + (lane & 7), pcol = 8 * ((lane >> 3) & 1);
    auto done = [&](int i) {  // this warp's part of hand-over i
        tmem_fence_before_sync();
        __syncwarp();
        if (lane == 0) arrive(bar(i));
    };
    auto loaded = [&](int c, int st, uint32_t ph) {  // chunk c is in its stage
        wait(kLanded + st, ph);
        if (ragged && c == nch - 1) wait(kFixed, 0);
    };
    // x of 16 tokens (block `tb` of the chunk) and this warp's 32 channels, transposed
    auto fetch = [&](int st, int tb, uint32_t (&x)[2][4]) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int pp = q * 32 + half * 16 + pcol;
            ldsm_t(s0 + st * L.stage_bytes + (pp >> 6) * 8192 + (tb * 16 + row) * 128 + ((((pp & 63) >> 3) ^ (row & 7)) << 4), x[half]);
        }
    };
    // Xw of them, three exact pieces (the second negated)
    auto weigh = [&](int i, int st, int tb, const uint32_t (&x)[2][4]) {
        const uint32_t xw = tq + cXw + i * 96 + tb * 8;
        const float* w = toks[st * HP + hw].w + tb * 16 + 2 * (lane & 3);
        const float2 w0 = *reinterpret_cast<const float2*>(w), w1 = *reinterpret_cast<const float2*>(w + 8);
        const F2 ww[2] = {f2(w0.x, w0.y), f2(w1.x, w1.y)};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t piece[3][4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                F2 v = mul2(bf_pair(x[half][k]), ww[k >> 1]);
                piece[0][k] = peel(v);
                piece[1][k] = peel(v);
                piece[2][k] = pack_cut(v);
            }
#pragma unroll
            for (int s = 0; s < 3; ++s)
                tmem_st_16x8(xw + (static_cast<uint32_t>(half) << 20) + s * 32, piece[s][0], piece[s][1], piece[s][2], piece[s][3]);
        }
    };
    // y of chunk c, 16 tokens (block tb) x this warp's 32 channels, through registers into the patch that the load warp
    // stores.  Chunk c is known to be in its stage: its products waited for that.
    auto outputs = [&](int c, int st, int tb) {
        const uint32_t patch = L.patch_off + (NBUF == 2 ? (c & 1) * 4 * kPatch : 0) + q * kPatch + tb * 1024;
        const uint32_t ty = tq + tb * 16;
        float yb[2][8], ya[2][8];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            tmem_ld_16x16(ty + (static_cast<uint32_t>(half) << 20) + cYb, yb[half]);
            tmem_ld_16x16(ty + (static_cast<uint32_t>(half) << 20) + cYa, ya[half]);
        }
        const float* e = toks[st * HP + hw].ein + tb * 16 + 2 * (lane & 3);
        const float2 e0 = *reinterpret_cast<const float2*>(e), e1 = *reinterpret_cast<const float2*>(e + 8);
        tmem_wait_ld();
        done(kYfree);
        if (c >= NBUF) wait(kPatchFree + (NBUF == 2 ? c & 1 : 0), NBUF == 2 ? ((c >> 1) - 1) & 1 : (c - 1) & 1);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            settle(yb[half]);
            settle(ya[half]);
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {  // 8 tokens k/2, 8 channels k%2
                const int at = 4 * (k >> 1) + 2 * (k & 1);
                const float2 ee = k < 2 ? e0 : e1;
                o[k] = pack_rn(fma2(f2(ee.x, ee.y), f2(yb[half][at], yb[half][at + 1]), f2(ya[half][at], ya[half][at + 1])));
            }
            stsm_t(s0 + patch + row * 64 + (((half * 2 + (pcol >> 3)) ^ ((row >> 1) & 3)) << 4), o[0], o[1], o[2], o[3]);
        }
        if (ragged && c == nch - 1) {  // rows behind the sequence are not this call's to write
            __syncwarp();
            const int tok0 = r.first + c * kQ + tb * 16, left = r.last - tok0;
            const int64_t yrow = static_cast<int64_t>(p.H) * P;
            __nv_bfloat16* yp = reinterpret_cast<__nv_bfloat16*>(p.y) + (static_cast<int64_t>(b) * p.T + tok0) * yrow + g * cend + c0 + q * 32 + (lane & 3) * 8;
#pragma unroll 1
            for (int t = lane >> 2; t < min(left, 16) && c0 + q * 32 < cend; t += 8)
                *reinterpret_cast<uint4*>(yp + t * yrow) = *reinterpret_cast<const uint4*>(sm + patch + t * 64 + (((lane & 3) ^ ((t >> 1) & 3)) << 4));
        }
        fence_async_smem();
        done(kOut + (c & 1));
    };
    // Before a block ends, whichever of its waits ran out and in whichever role: what was started has come to its end (bounded,
    // and whatever the abort flag says).  No copy may land in its memory, and no product write to its tensor memory, after that.
    auto over = [&](int i, uint32_t parity) {
        const uint64_t t_end = now_ns() + 2000000000ull;
        for (uint32_t it = 0; it < kSpinLimit; ++it)
            if (try_wait(bar(i), parity) || now_ns() > t_end) break;
    };
    auto drain = [&](int i) {  // (a commit covers the products of the thread that makes it, the elected one that issued them)
        if (elect_one()) {
            mma_commit(bar(i));
            over(i, 0);
        }
        __syncwarp();
    };

    if (warp < kInWarps) {
        // ------------------------------------------------------------ operands of the chunk: Xw, W, X^T
        regs_down<kInRegs>();
        int st = 0;
        uint32_t ph = 0;
        const int j = q * 16 + (lane >> 2);  // this lane's rows of W: tokens j and j + 8
        for (int c = 0; c < nch; ++c) {
            const ChunkTok* tok = toks + st * HP;
            loaded(c, st, ph);
            uint32_t x[2][2][4];
#pragma unroll
            for (int tg = 0; tg < 2; ++tg) fetch(st, part * 2 + tg, x[tg]);
            if constexpr (OUT) {
                auto read = [&]() {  // the chunk before is through with X^T, and with its buffer of W; its outputs are there
                    if (c > 0) wait(kY, (c - 1) & 1);
                };
                if (NBUF == 1) read();
                wait(kG, c & 1);
                tmem_fence_after_sync();
                // Tokens j of block q reach tokens i of blocks cb = q..3; the quadrant's two warps take every second cb.
#pragma unroll 1
                for (int cb = q + part; cb < 4; cb += 2) {
                    float gv[8];
                    tmem_ld_16x16(tq + cG + cb * 16, gv);
                    const int i0 = cb * 16 + 2 * (lane & 3);
                    const uint32_t wbuf = L.w_off + (NBUF == 2 ? (c & 1) * HP * 16384 : 0) + j * 128 + 4 * (lane & 3);
                    const uint32_t at0 = wbuf + (((2 * cb) ^ (j & 7)) << 4), at1 = wbuf + (((2 * cb + 1) ^ (j & 7)) << 4);
                    auto put = [&](int h, int rb, int k, F2 w) {
                        const uint32_t at = (k ? at1 : at0) + h * 16384 + rb * 1024;
                        *reinterpret_cast<uint32_t*>(sm + at) = peel(w);
                        *reinterpret_cast<uint32_t*>(sm + at + 8192) = pack_rn(w);
                    };
                    tmem_wait_ld();
                    settle(gv);
                    if (cb != q) {
                        // exp(a_i - a_j) d_j in three factors that meet at block ends, none above 1 in a decaying state
#pragma unroll
                        for (int h = 0; h < HP; ++h) {
                            const ChunkTok& tk = tok[h];
                            const float f = cb == q + 1 ? 1.0f : tk.blk[cb == q + 3 ? 2 : q];
                            const float2 u0 = *reinterpret_cast<const float2*>(tk.u + i0), u1 = *reinterpret_cast<const float2*>(tk.u + i0 + 8);
#pragma unroll
                            for (int rb = 0; rb < 2; ++rb) {
                                const float v = tk.v[j + 8 * rb] * f;
#pragma unroll
                                for (int k = 0; k < 2; ++k)
                                    put(h, rb, k, mul2(mul2(k ? f2(u1.x, u1.y) : f2(u0.x, u0.y), f2(v, v)),
                                                       f2(gv[4 * k + 2 * rb], gv[4 * k + 2 * rb + 1])));
                            }
                        }
                    } else {
#pragma unroll
                        for (int h = 0; h < HP; ++h) {
                            const ChunkTok& tk = tok[h];
                            const float skip = (p.D && head0 + h < hg) ? p.D[g * hg + head0 + h] : 0.0f;
#pragma unroll
                            for (int rb = 0; rb < 2; ++rb) {
                                const float jh = tk.hi[j + 8 * rb], jl = tk.lo[j + 8 * rb], dj = tk.d[j + 8 * rb];
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    const float2 hi = *reinterpret_cast<const float2*>(tk.hi + i0 + 8 * k);
                                    const float2 lo = *reinterpret_cast<const float2*>(tk.lo + i0 + 8 * k);
                                    float u, v;
                                    un(add2(add2(f2(hi.x, hi.y), f2(-jh, -jh)), add2(f2(lo.x, lo.y), f2(-jl, -jl))), u, v);
                                    un(mul2(mul2(f2(ex2(u), ex2(v)), f2(dj, dj)), f2(gv[4 * k + 2 * rb], gv[4 * k + 2 * rb + 1])), u, v);
                                    // nothing from later tokens; D x_i rides on the diagonal
                                    const int ii = i0 + 8 * k - (j + 8 * rb);
                                    put(h, rb, k, f2(ii > 0 ? u : ii == 0 ? u + skip : 0.0f, ii > -1 ? v : ii == -1 ? v + skip : 0.0f));
                                }
                            }
                        }
                    }
                }
                fence_async_smem();
                uint32_t sum[2] = {0, 0};  // (here, since the loads of x have long ended: 2% less than in front of W)
#pragma unroll
                for (int k = 0; k < 16; ++k) add_zeros(sum[k & 1], x[k >> 3][(k >> 2) & 1][k & 3]);
                if (__any_sync(0xffffffffu, ((sum[0] | sum[1]) & 0x7fff7fffu) != 0)) {
                    // In this warp's 32 channels and 32 tokens, which no other reads: zeros in place of what is no number.
                    const int ch = q * 32 + lane, t0 = part * 32;
                    int first = INT_MAX;
#pragma unroll 1
                    for (int t = t0 + 31; t >= t0; --t) {
                        uint16_t* at = reinterpret_cast<uint16_t*>(sm + st * L.stage_bytes + (ch >> 6) * 8192 + t * 128 + ((((ch & 63) >> 3) ^ (t & 7)) << 4) + (ch & 7) * 2);
                        if ((*at & 0x7f80) == 0x7f80) *at = 0, first = r.first + c * kQ + t;
                    }
                    if (first != INT_MAX) atomicMin(first_bad + ch, first);
                    *any_bad = 1;
                    __syncwarp();
#pragma unroll
                    for (int tg = 0; tg < 2; ++tg) fetch(st, part * 2 + tg, x[tg]);
                }
                if (NBUF == 2) read();
                tmem_fence_after_sync();
#pragma unroll
                for (int tg = 0; tg < 2; ++tg)
#pragma unroll
                    for (int half = 0; half < 2; ++half)
                        tmem_st_16x8(tq + (static_cast<uint32_t>(half) << 20) + cX + part * 16 + tg * 8, x[tg][half][0], x[tg][half][1],
                                     x[tg][half][2], x[tg][half][3]);
                tmem_wait_st();
                done(kW);
                if (c > 0) {  // every second block of the outputs before
                    const int before = st == 0 ? L.stages - 1 : st - 1;
                    outputs(c - 1, before, part * 2 + 1);
                    if (lane == 0) arrive(bar(kEmpty + before));
                }
            }
            // Xw's buffer: the product that read it is done
            if (OUT && c > 0) wait(kDs + HALVES - 1, (c - 1) & 1);
            if (!OUT && c >= 2) wait(kDs + (c & 1), ((c >> 1) - 1) & 1);
            tmem_fence_after_sync();
            const int xb = OUT ? 0 : c & 1;
#pragma unroll
            for (int tg = 0; tg < 2; ++tg) weigh(xb, st, part * 2 + tg, x[tg]);
            tmem_wait_st();
            done(kXw + xb);
            if (++st == L.stages) st = 0, ph ^= 1;
        }
        if (OUT && nch > 0) {
            wait(kY, (nch - 1) & 1);
            tmem_fence_after_sync();
            outputs(nch - 1, st == 0 ? L.stages - 1 : st - 1, part * 2 + 1);
        }
    } else if (warp < kWarps) {
        // ------------------------------------------------------------ state and outputs
        regs_up<kOutRegs>();
        const int ch = c0 + q * 32 + lane;  // channel of this lane's state columns
        const bool mine = ch < cend;
        const int64_t bh = static_cast<int64_t>(b) * p.H + g * hg + ch / P;
        constexpr int64_t np = static_cast<int64_t>(N) * P;
        constexpr int NC = N / 2;              // state columns per warp
        constexpr int NV = NC < 16 ? NC : 16;  // of them per tensor-memory access
        const int64_t own = static_cast<int64_t>(part) * NC * P + ch % P;
        F2 S[NC / 2];
        {
            const float* from = nullptr;
            if (OUT && mine) {
                if (p.split.nseg > 1) from = p.seg_state + (bh * p.split.slots() + seg * p.split.sub) * np + own;
                else if (p.S_in) from = p.S_in + bh * np + own;
            }
#pragma unroll
            for (int k = 0; k < NC / 2; ++k) S[k] = from ? f2(from[2 * k * P], from[(2 * k + 1) * P]) : f2(0.0f, 0.0f);
        }
        auto put_state = [&]() {  // the state as an operand of Yb, two pieces (the second negated)
#pragma unroll
            for (int k0 = 0; k0 < NC; k0 += NV) {
                uint32_t hi[NV / 2], lo[NV / 2];
#pragma unroll
                for (int k = 0; k < NV / 2; ++k) {
                    F2 v = S[k0 / 2 + k];
                    hi[k] = peel(v);
                    lo[k] = pack_rn(v);
                }
                tmem_st_cols<NV / 2>(tq + cShi + (part * NC + k0) / 2, hi);
                tmem_st_cols<NV / 2>(tq + cSlo + (part * NC + k0) / 2, lo);
            }
            tmem_wait_st();
            done(kS);
        };
        auto add_chunk = [&](int c, int st) {  // S' = dec S + dS
            const int i = OUT ? (HALVES == 2 ? part : 0) : c & 1;
            wait(kDs + i, OUT ? c & 1 : (c >> 1) & 1);
            tmem_fence_after_sync();
            const float decay = toks[st * HP + hw].dec;
            const F2 dec = f2(decay, decay);
            const uint32_t td = tq + cDs + (OUT ? 0 : i * 128) + (HALVES == 2 ? 0 : part * NC);
            float d[2][NV];
            tmem_ld_cols<NV>(td, d[0]);
#pragma unroll
            for (int k0 = 0; k0 < NC; k0 += NV) {
                const int now = (k0 / NV) & 1;
                tmem_wait_ld();
                settle(d[now]);
                if (k0 + NV < NC) tmem_ld_cols<NV>(td + k0 + NV, d[now ^ 1]);
                else done(kDsFree + i);
#pragma unroll
                for (int k = 0; k < NV / 2; ++k) S[k0 / 2 + k] = fma2(S[k0 / 2 + k], dec, f2(d[now][2 * k], d[now][2 * k + 1]));
            }
        };
        if (OUT && nch > 0) put_state();
        int st = 0;
        uint32_t ph = 0;
        for (int c = 0; c < nch; ++c) {
            if constexpr (OUT) {
                // The state takes dS before the outputs are there, but for the second half where dS comes in halves
                // (one copy of both parts, for the instruction cache).
#pragma unroll 1
                for (int step = 0; step < 2; ++step) {
                    if (step == (HALVES == 2 ? part : 0)) {
                        add_chunk(c, st);
                    } else {
                        wait(kY, c & 1);
                        tmem_fence_after_sync();
                        outputs(c, st, part * 2);
                    }
                }
                if (c + 1 < nch) put_state();
            } else {
                loaded(c, st, ph);
                add_chunk(c, st);
            }
            __syncwarp();
            if (lane == 0) arrive(bar(kEmpty + st));
            if (++st == L.stages) st = 0, ph ^= 1;
        }
        float* to = nullptr;
        if (mine) {
            if (!OUT) to = p.seg_state + (bh * p.split.slots() + seg) * np + own;
            else if (seg == p.split.nseg - 1) to = p.S_out + bh * np + own;
        }
        if (OUT && to && first_bad[q * 32 + lane] != INT_MAX) {
            const float none = __int_as_float(0x7fffffff);
#pragma unroll
            for (int k = 0; k < NC / 2; ++k) S[k] = f2(none, none);
        }
        if (to) {
#pragma unroll
            for (int k = 0; k < NC / 2; ++k) un(S[k], to[2 * k * P], to[(2 * k + 1) * P]);
        }
    } else if (warp == kLoadWarp) {
        // ------------------------------------------------------------ TMA
        regs_down<kMiscRegs>();
        const int heads = min(HP, hg - head0);
        const int chunks = (p.T + kQ - 1) / kQ;
        const ChunkTok* src = p.toks + (static_cast<int64_t>(b) * p.H + g * hg + head0) * chunks + r.first / kQ;
        int issued = 0;
        auto load = [&](int c) {
            const int st = c % L.stages, t0 = r.first + c * kQ, nv = min(kQ, r.last - t0);
            const uint32_t base = s0 + st * L.stage_bytes;
            const uint32_t landed = bar(kLanded + st);
            if (lane == 0) arrive_tx(landed, L.stage_bytes + heads * static_cast<uint32_t>(sizeof(ChunkTok)));
            __syncwarp();
            // one copy per lane: x, B and C in boxes of 64 columns, then the heads' decays
            const int col = (lane & 1) * 64;
            if (lane < 2) tma_load_3d(base + lane * 8192, &maps.x, g * cend + c0 + col, t0, b, landed);
            else if (lane < 4 && col < N) tma_load_4d(base + L.b_off + (lane & 1) * 8192, &maps.b, col, g, t0, b, landed);
            else if (OUT && lane >= 4 && lane < 6 && col < N) tma_load_4d(base + L.c_off + (lane & 1) * 8192, &maps.c, col, g, t0, b, landed);
            else if (lane >= 6 && lane < 6 + heads)
                bulk_load(s0 + L.tok_off + (st * HP + lane - 6) * static_cast<uint32_t>(sizeof(ChunkTok)),
                          src + static_cast<int64_t>(lane - 6) * chunks + c, sizeof(ChunkTok), landed);
            __syncwarp();
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
        };
#pragma unroll 1
        for (int c = -L.stages; c < nch && !*abort_flag; ++c) {  // the first rounds only load
            if (OUT && c >= 0) {
                wait(kOut + (c & 1), (c >> 1) & 1);
                if (!(ragged && c == nch - 1)) {
                    if (lane < 4 && c0 + lane * 32 < cend) {
                        tma_store_3d(&maps.y, g * cend + c0 + lane * 32, r.first + c * kQ, b,
                                     s0 + L.patch_off + (NBUF == 2 ? (c & 1) * 4 * kPatch : 0) + lane * kPatch);
                        store_read_done();
                    }
                    __syncwarp();
                    if (lane == 0) arrive(bar(kPatchFree + (NBUF == 2 ? c & 1 : 0)));
                }
            }
            if (c + L.stages < nch) {
                if (c >= 0) wait(kEmpty + c % L.stages, (c / L.stages) & 1);
                if (!*abort_flag) load(c + L.stages);
            }
        }
        if (OUT && lane < 4) store_done();
        if (OUT && *any_bad) {
            __syncwarp();
            // all outputs are there: none of a channel from its first x that is no number on
            for (int k = 0; k < 128; ++k) {
                if (c0 + k >= cend) break;
                for (int64_t t = static_cast<int64_t>(first_bad[k]) + lane; t < r.last; t += 32)
                    reinterpret_cast<uint16_t*>(p.y)[((static_cast<int64_t>(b) * p.T + t) * p.H + g * hg) * P + c0 + k] = 0x7fff;
            }
        }
        if (lane == 0)
            for (int c = issued > L.stages ? issued - L.stages : 0; c < issued; ++c) over(kLanded + c % L.stages, (c / L.stages) & 1);
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ MMA issue: G and dS (whole warp, one lane issues)
        regs_down<kMiscRegs>();
        constexpr int ND = HALVES == 2 ? 64 : N;  // columns of one dS product
        constexpr uint32_t wG = mma_word(64, 64, false, false), wDs = mma_word(128, ND, false, true), wDsNeg = mma_word(128, ND, false, true, true);
        auto issue_g = [&](int st) {
            const Desc along = desc_of(s0 + st * L.stage_bytes, 16);  // B and C as [token, n]: contraction along the rows
            tmem_fence_after_sync();
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < N / 16; ++k)
                    mma_ss(tm + cG, along + (L.b_off + (k >> 2) * 8192 + (k & 3) * 32), along + (L.c_off + (k >> 2) * 8192 + (k & 3) * 32), wG,
                           k > 0);
                mma_commit(bar(kG));
            }
            __syncwarp();
        };
        auto issue_ds = [&](int i, int xb, int half, int st) {  // a part of dS, signalled on kDs + i
            const Desc down = desc_of(s0 + st * L.stage_bytes + L.b_off + half * 8192, 8192);  // B as [j, n]: contraction down the rows
            tmem_fence_after_sync();
            if (elect_one()) {
#pragma unroll
                for (int s = 2; s >= 0; --s)  // the small pieces first
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_ts(tm + cDs + (OUT ? 0 : i * 128), tm + cXw + xb * 96 + s * 32 + k * 8, down + k * 2048, s == 1 ? wDsNeg : wDs,
                               s < 2 || k > 0);
                mma_commit(bar(kDs + i));
            }
            __syncwarp();
        };
        int st = 0;
        uint32_t ph = 0;
        if (OUT && nch > 0) {
            loaded(0, 0, 0);
            issue_g(0);
        }
        for (int c = 0; c < nch && !*abort_flag; ++c) {
            const int st1 = st + 1 == L.stages ? 0 : st + 1;
            const uint32_t ph1 = st1 == 0 ? ph ^ 1 : ph;
            if constexpr (OUT) {
                wait(kW, c & 1);  // G's columns have been read
                if (c + 1 < nch) {
                    loaded(c + 1, st1, ph1);
                    issue_g(st1);
                }
                wait(kXw, c & 1);
                if (c > 0) wait(kDsFree + HALVES - 1, (c - 1) & 1);
#pragma unroll 1
                for (int half = 0; half < HALVES; ++half) {
                    if (half == 1) wait(kDsFree, c & 1);
                    issue_ds(half, 0, half, st);
                }
            } else {
                loaded(c, st, ph);
                wait(kXw + (c & 1), (c >> 1) & 1);
                if (c >= 2) wait(kDsFree + (c & 1), ((c >> 1) - 1) & 1);
                issue_ds(c & 1, c & 1, 0, st);
            }
            st = st1, ph = ph1;
        }
        drain(kDrain);
    } else if (warp == kMmaWarp + 1) {
        // ------------------------------------------------------------ MMA issue: Yb and Ya
        regs_down<kMiscRegs>();
        if constexpr (OUT) {
            int st = 0;
            for (int c = 0; c < nch && !*abort_flag; ++c) {
                const Desc along = desc_of(s0 + st * L.stage_bytes + L.c_off, 16);  // C as [i, n]: contraction along the rows
                const Desc wd = desc_of(s0 + L.w_off + (NBUF == 2 ? (c & 1) * HP * 16384 : 0), 8192);
                wait(kW, c & 1);                       // W and X^T are there
                if (c > 0) wait(kYfree, (c - 1) & 1);  // the columns of Ya and Yb have been read
                tmem_fence_after_sync();
                if (elect_one()) {
#pragma unroll
                    for (int h = 0; h < HP; ++h)
#pragma unroll
                        for (int s = 0; s < 2; ++s)
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const Desc db = wd + (h * 16384 + (s ? 0 : 8192) + k * 2048);
                                constexpr uint32_t w0 = mma_word(128, 64, false, true, false, true), w1 = mma_word(128, 64, false, true);
                                if constexpr (HP == 1) {
                                    mma_ts(tm + cYa, tm + cX + k * 8, db, s ? w1 : w0, s + k > 0);
                                } else {
                                    auto off = [&](int qq) { return (HP == 4 ? qq : qq >> 1) == h ? 0u : 0xffffffffu; };
                                    mma_ts_masked(tm + cYa, tm + cX + k * 8, db, s ? w1 : w0, off(0), off(1), off(2), off(3), s + k > 0);
                                }
                            }
                }
                __syncwarp();
                wait(kS, c & 1);
                tmem_fence_after_sync();
                if (elect_one()) {
#pragma unroll
                    for (int s = 0; s < 2; ++s)
#pragma unroll
                        for (int k = 0; k < N / 16; ++k)
                            mma_ts(tm + cYb, tm + (s ? cShi : cSlo) + k * 8, along + ((k >> 2) * 8192 + (k & 3) * 32),
                                   s ? mma_word(128, 64, false, false) : mma_word(128, 64, false, false, true), s + k > 0);
                    mma_commit(bar(kY));
                }
                __syncwarp();
                if (++st == L.stages) st = 0;
            }
            drain(kDrain + 1);
        }
    } else {
        regs_down<kMiscRegs>();  // the warp that makes up the group
    }
    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
    if (warp == kMmaWarp) tmem_dealloc(tm, 512);
    if (threadIdx.x == 0 && *abort_flag) set_status(p.status, kDevTimeout);
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
    return encode(&m->y, p.y, 3, xsize, ystr, 32, 64) && encode(&m->x, p.x, 3, xsize, xstr) && encode(&m->b, p.Bm, 4, bsize, bstr) && encode(&m->c, p.Cm, 4, bsize, cstr);
}

template <int N, int P, bool OUT>
cudaError_t go(const SsmParams& p, const MmaMaps& m, int tiles, int segs, cudaStream_t s)
{
    constexpr Layout L = layout_of(N, P >= 128 ? 1 : 128 / P, OUT);
    static_assert(kThreads == 640, "register split");
    static_assert(L.total <= kSmemMax, "shared memory");
    auto kern = k_ssm_mma<N, P, OUT>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(L.total));
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, dim3(static_cast<unsigned>(p.B) * p.G * tiles, segs), kThreads, L.total, s, m, p, tiles);
}

template <int N, int P>
cudaError_t all(const SsmParams& p, const MmaMaps& m, cudaStream_t s)
{
    const int tiles = (p.H / p.G * p.P + 127) / 128;
    if (p.split.nseg > 1) {
        cudaError_t e = go<N, P, false>(p, m, tiles, p.split.pieces(), s);
        if (e == cudaSuccess) e = launch_ssm_chain(p, s);
        if (e != cudaSuccess) return e;
    }
    return go<N, P, true>(p, m, tiles, p.split.nseg, s);
}

template <int N>
cudaError_t pick(const SsmParams& p, const MmaMaps& m, cudaStream_t s)
{
    switch (p.P) {
        case 32: return all<N, 32>(p, m, s);
        case 64: return all<N, 64>(p, m, s);
        case 128: return all<N, 128>(p, m, s);
        default: return all<N, 256>(p, m, s);
    }
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
// TMA wants strides of whole 16 bytes below 2^40; a stride of nothing (an expanded view) is left out
bool ok_stride(int64_t n, int64_t size) { return size == 1 || (n > 0 && n % 8 == 0 && n < (1ll << 39)); }

}  // namespace

// (N = 256 would take 512 columns of tensor memory for the state's pieces and dS alone, and P = 16 eight copies of W, 128
// KB: those sizes, like fp32 and layouts that TMA does not read, go token by token.)
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
    const int chunks = (p.T + kQ - 1) / kQ;
    const int64_t work = static_cast<int64_t>(p.B) * p.H * chunks;
    k_ssm_decay<<<static_cast<unsigned>((work + 7) / 8), 256, 0, s>>>(p, chunks, work);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    switch (p.N) {
        case 16: return pick<16>(p, m, s);
        case 32: return pick<32>(p, m, s);
        case 64: return pick<64>(p, m, s);
        case 128: return pick<128>(p, m, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace ramnet
