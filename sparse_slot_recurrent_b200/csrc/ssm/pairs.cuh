// pairs.cuh -- pairs of fp32 values that one instruction works on, and values as bf16 pieces.
#pragma once

#include <cstdint>

namespace ramnet {
namespace {

// ------------------------------------------------------------------ pairs of fp32 in one instruction

struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b)
{
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void un(F2 p, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p.v)); }
__device__ __forceinline__ F2 add2(F2 a, F2 b)
{
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b)
{
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// ------------------------------------------------------------------ values as bf16 pieces

__device__ __forceinline__ float bf_lo(uint32_t pair) { return __uint_as_float(pair << 16); }
__device__ __forceinline__ float bf_hi(uint32_t pair) { return __uint_as_float(pair & 0xffff0000u); }
__device__ __forceinline__ F2 bf_pair(uint32_t pair) { return f2(bf_lo(pair), bf_hi(pair)); }

__device__ __forceinline__ uint32_t pack_rn(F2 p)  // the first value in the low half
{
    float a, b;
    un(p, a, b);
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ uint32_t pack_cut(F2 p)  // the leading 8 bits of both
{
    float a, b;
    un(p, a, b);
    return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
// Adds the products of a pair of bf16 with 0: a sum of these stays +-0 unless one of the values is no number.
__device__ __forceinline__ void add_zeros(uint32_t& sum, uint32_t pair) { asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum) : "r"(pair), "r"(0)); }
// The leading 8 bits of both as one pair of bf16; p keeps what is left, negated (exact).  The differences take the
// bf16 halves as they are, on the multiply-add pipe: the integer pipe has enough to do (a split that masks and
// subtracts in 32 bits measured 7.4 issue cycles per pair, this one 4.8).
__device__ __forceinline__ uint32_t peel(F2& p)
{
    float a, b;
    un(p, a, b);
    const uint32_t h = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
    asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tsub.rn.f32.bf16 %0, x, %0;\n\tsub.rn.f32.bf16 %1, y, %1;\n\t}" : "+f"(a), "+f"(b) : "r"(h));
    p = f2(a, b);
    return h;
}

}  // namespace
}  // namespace ramnet
