// ssm_mma.cuh -- device helpers of the tensor-core scan: bounded waits, tensor-map loads, tcgen05
// descriptors and issue, and the tensor-memory and shared-memory fragment moves it uses.
#pragma once

#include <cuda.h>

#include "pairs.cuh"
#include "ssm_common.cuh"

namespace ramnet {
namespace {

// ------------------------------------------------------------------ bounded waits

__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(20000u)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ uint64_t now_ns()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// Bounded wait for phase `parity`.  `limit` is the address of two words of shared memory: the block's abort flag, and what a
// poll costs of a wait's budget of kWaitNs.  The hardware suspends a poll until the phase is there or kPollNs have passed
// (whatever time the instruction is given).  When the budget runs out the flag is raised, after which every wait of the block
// returns at its next poll; the kernel reports the flag in the status word at its end.  Few instructions, because this is
// inlined at every hand-over and the roles of a block share the instruction cache: with a clock in here a prompt takes 10%
// longer, 4% with one in a warp that does nothing else, 2% with the number of polls as a parameter.
__device__ __forceinline__ void wait_phase(uint32_t bar, uint32_t parity, uint32_t limit)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .s32 n, c;\n\t.reg .u32 a;\n\tmov.s32 n, %3;\n"
        "L_poll_%=:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%0], %1;\n\t"
        "@p bra L_done_%=;\n\t"
        "ld.volatile.shared.v2.u32 {a, c}, [%2];\n\t"
        "setp.ne.u32 p, a, 0;\n\t"
        "@p bra L_done_%=;\n\t"
        "sub.s32 n, n, c;\n\t"
        "setp.gt.s32 p, n, 0;\n\t"
        "@p bra L_poll_%=;\n\t"
        "st.volatile.shared.u32 [%2], 1;\n"
        "L_done_%=:\n\t}" ::"r"(bar),
        "r"(parity), "r"(limit), "n"(kWaitNs)
        : "memory");
}

__device__ __forceinline__ void arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void arrive_tx(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ------------------------------------------------------------------ tensor-map loads (no multicast)

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
                 : "memory");
}

// ... and stores: a box of shared memory out, in this thread's bulk group.  The box may be
// written again once store_read_done() has returned in the same thread.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, int c0, int c1, int c2, uint32_t src)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];\n\tcp.async.bulk.commit_group;" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}
__device__ __forceinline__ void store_read_done() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void store_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// ... and plain bytes (both addresses and the size in units of 16)
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// ------------------------------------------------------------------ tcgen05

// Shared-memory operand in 128-byte rows with the 128-byte swizzle.  Rows of one 8-row group
// are 128 bytes apart and groups 1024; `lbo` is the distance between 64-element blocks along
// the row direction (used by operands whose contraction runs down the rows).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo)
{
    return static_cast<uint64_t>((addr & 0x3ffff) >> 4) | (static_cast<uint64_t>(lbo >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// Instruction word: bf16 x bf16 -> fp32, M x N; ta / tb: the operand's contraction runs down the
// rows of shared memory (its other dimension is contiguous); na / nb: the operand is taken negated.
__host__ __device__ constexpr uint32_t mma_word(int M, int N, bool ta, bool tb, bool na = false, bool nb = false)
{
    return (static_cast<uint32_t>(na) << 13) | (static_cast<uint32_t>(nb) << 14) |
           (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(ta) << 15) | (static_cast<uint32_t>(tb) << 16) |
           (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// The two halves of a descriptor: the address moves within the low word, the high word is fixed.
struct Desc {
    uint32_t lo, hi;
    __device__ __forceinline__ Desc operator+(uint32_t bytes) const { return Desc{lo + (bytes >> 4), hi}; }
};
__device__ __forceinline__ Desc desc_of(uint32_t addr, uint32_t lbo)
{
    const uint64_t d = smem_desc(addr, lbo);
    return Desc{static_cast<uint32_t>(d), static_cast<uint32_t>(d >> 32)};
}

__device__ __forceinline__ void mma_ss(uint32_t d, Desc a, Desc b, uint32_t word, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tmov.b64 x, {%1, %2};\n\tmov.b64 y, {%3, %4};\n\tsetp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %5, p;\n\t}" ::"r"(d),
        "r"(a.lo), "r"(a.hi), "r"(b.lo), "r"(b.hi), "r"(word), "r"(static_cast<uint32_t>(add))
        : "memory");
}

// first operand in tensor memory (two bf16 along the contraction per 32-bit column)
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, Desc b, uint32_t word, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tmov.b64 y, {%2, %3};\n\tsetp.ne.u32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b.lo), "r"(b.hi), "r"(word), "r"(static_cast<uint32_t>(add))
        : "memory");
}

// ... leaving alone the tensor-memory lanes whose bit is set in m0 (lanes 0..31) .. m3 (96..127)
__device__ __forceinline__ void mma_ts_masked(uint32_t d, uint32_t a, Desc b, uint32_t word, uint32_t m0, uint32_t m1, uint32_t m2,
                                              uint32_t m3, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tmov.b64 y, {%2, %3};\n\tsetp.ne.u32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, {%6, %7, %8, %9}, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b.lo), "r"(b.hi), "r"(word), "r"(static_cast<uint32_t>(add)), "r"(m0), "r"(m1), "r"(m2), "r"(m3)
        : "memory");
}

// One lane of the (whole) warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}

// Arrives on `bar` once every MMA this thread has issued is complete.
__device__ __forceinline__ void mma_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// 16 lanes x 16 columns: v[4k + r]: lane t/4 (+8 for r >= 2), column 8k + 2 (t%4) + r%2.
__device__ __forceinline__ void tmem_ld_16x16(uint32_t a, float (&v)[8])
{
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(a));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// 16 lanes x 8 columns: v[2k + r]: lane t/4 + 8r, column 4k + t%4.
__device__ __forceinline__ void tmem_st_16x8(uint32_t a, uint32_t v0, uint32_t v1, uint32_t v2, uint32_t v3)
{
    asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v0), "r"(v1), "r"(v2), "r"(v3) : "memory");
}

__device__ __forceinline__ void tmem_ld_x16(uint32_t a, float* v)
{
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(a));
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// Placed behind tmem_wait_ld: ties the loaded registers to that point, so that no arithmetic on
// them is moved in front of the wait.  No instruction.
template <int N>
__device__ __forceinline__ void settle(float (&v)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}

// N consecutive columns of the warp's 32 lanes.
template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t a, float (&v)[N])
{
    if constexpr (N >= 16) {
#pragma unroll
        for (int i = 0; i < N; i += 16) tmem_ld_x16(a + i, v + i);
    } else {
        tmem_ld<N>(a, v);
    }
}

template <int N>
__device__ __forceinline__ void tmem_st_cols(uint32_t a, const uint32_t (&v)[N])
{
    if constexpr (N == 16)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(a),
                     "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
                     "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
                     : "memory");
    else {
        float f[N];
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = __uint_as_float(v[i]);
        tmem_st<N>(a, f);
    }
}

// Registers per thread of the calling warpgroup from here on.
template <int N>
__device__ __forceinline__ void regs_up()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// ------------------------------------------------------------------ shared-memory fragments

// Four 8x8 blocks of 16-bit values, transposed: lane t gets, of block k, rows 2 (t%4) and +1 of
// column t/4; `addr`: lane 8k + r points at row r of block k.
__device__ __forceinline__ void ldsm_t(uint32_t addr, uint32_t (&v)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(addr));
}

__device__ __forceinline__ void stsm_t(uint32_t addr, uint32_t v0, uint32_t v1, uint32_t v2, uint32_t v3)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v0), "r"(v1), "r"(v2), "r"(v3)
                 : "memory");
}

}  // namespace
}  // namespace ramnet
