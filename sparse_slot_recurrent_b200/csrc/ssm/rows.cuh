// rows.cuh -- device helpers of the kernels that stream rows of channels: pairs of fp32, vectors of V
// neighbouring values (16 bytes, or one value where addresses do not allow that), SiLU.
#pragma once

#include <initializer_list>
#include <type_traits>

#include "../common.cuh"
#include "pairs.cuh"
#include "ssm.h"

namespace ramnet {
namespace {

// What one step of arithmetic works on: a pair of values, or a lone one.
template <int V>
using Val = typename std::conditional<V == 1, float, F2>::type;
__device__ __forceinline__ float fma2(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float mul2(float a, float b) { return a * b; }
template <int V>
__device__ __forceinline__ Val<V> val(float a, float b)
{
    if constexpr (V == 1) return a;
    else return f2(a, b);
}
template <int V>
__device__ __forceinline__ void put(Val<V> p, int h, float (&y)[V])
{
    if constexpr (V == 1) y[0] = p;
    else un(p, y[2 * h], y[2 * h + 1]);
}

// V values as they lie in memory, bf16 (BF) or fp32: one value, or 4, 8 or 16 bytes.
template <bool BF, int V>
struct Raw {
    static constexpr int kBytes = V * (BF ? 2 : 4);
    static constexpr int kWords = kBytes >= 4 ? kBytes / 4 : 1;
    static_assert(kBytes <= 16 && (V & (V - 1)) == 0, "one access");
    uint32_t r[kWords];

    __device__ __forceinline__ void take(const void* at)
    {
        if constexpr (kBytes == 2) r[0] = *reinterpret_cast<const uint16_t*>(at);
        if constexpr (kBytes == 4) r[0] = *reinterpret_cast<const uint32_t*>(at);
        if constexpr (kBytes == 8) {
            const uint2 v = *reinterpret_cast<const uint2*>(at);
            r[0] = v.x, r[1] = v.y;
        }
        if constexpr (kBytes == 16) {
            const uint4 v = *reinterpret_cast<const uint4*>(at);
            r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
        }
    }
    __device__ __forceinline__ void load(const void* base, int64_t i) { take(reinterpret_cast<const unsigned char*>(base) + i * (BF ? 2 : 4)); }
    __device__ __forceinline__ void store(void* base, int64_t i) const
    {
        unsigned char* at = reinterpret_cast<unsigned char*>(base) + i * (BF ? 2 : 4);
        if constexpr (kBytes == 2) *reinterpret_cast<uint16_t*>(at) = static_cast<uint16_t>(r[0]);
        if constexpr (kBytes == 4) *reinterpret_cast<uint32_t*>(at) = r[0];
        if constexpr (kBytes == 8) *reinterpret_cast<uint2*>(at) = make_uint2(r[0], r[1]);
        if constexpr (kBytes == 16) *reinterpret_cast<uint4*>(at) = make_uint4(r[0], r[1], r[2], r[3]);
    }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int k = 0; k < kWords; ++k) r[k] = 0;
    }
    __device__ __forceinline__ Val<V> pair(int h) const  // values 2h and 2h+1
    {
        if constexpr (V == 1) return BF ? bf_lo(r[0]) : __uint_as_float(r[0]);
        else if constexpr (BF) return bf_pair(r[h]);
        else return f2(__uint_as_float(r[2 * h]), __uint_as_float(r[2 * h + 1]));
    }
    __device__ __forceinline__ void widen(Val<V> (&p)[(V + 1) / 2]) const
    {
#pragma unroll
        for (int h = 0; h < (V + 1) / 2; ++h) p[h] = pair(h);
    }
};

// The widest vector that divides every number in `at` (element strides, lengths) and the addresses, of those that kernels are
// built for: 16 bytes, two values, one.
inline int widest(bool bf16, std::initializer_list<int64_t> at, std::initializer_list<const void*> addresses)
{
    const int es = bf16 ? 2 : 4;
    int v = 16 / es;
    for (const int64_t n : at)
        while (n % v != 0) v /= 2;
    for (const void* p : addresses)
        while (reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(v * es) != 0) v /= 2;
    return bf16 && v == 4 ? 2 : v;
}

template <bool BF, int V>
__device__ __forceinline__ void store_vec(void* base, int64_t i, const float (&v)[V])
{
    if constexpr (V == 1) {
        store_out(base, static_cast<size_t>(i), v[0], BF);
    } else if constexpr (BF) {
        Raw<true, V> u;
#pragma unroll
        for (int j = 0; j < V / 2; ++j) u.r[j] = pack_rn(f2(v[2 * j], v[2 * j + 1]));
        u.store(base, i);
    } else {
        store_row_g<V>(reinterpret_cast<float*>(base) + i, v);
    }
}

// SiLU.  For a bf16 result the hardware's exp2 and reciprocal are enough: they are off by about 2^-21 of the value, and for
// negative p the rounding of the exponent by |p| 2^-24 more (2^-17.7 at p = -80), against bf16's 2^-9; below p = -87,
// where the value is under 1e-36, they give 0.  An fp32 result takes the accurate forms.
template <bool FAST>
__device__ __forceinline__ F2 silu2(F2 p)
{
    float a, b;
    if constexpr (FAST) {
        un(mul2(p, f2(-1.44269504f, -1.44269504f)), a, b);
        asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(a));
        asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(b));
        un(add2(f2(a, b), f2(1.0f, 1.0f)), a, b);
        asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a));
        asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(b));
        return mul2(p, f2(a, b));
    } else {
        un(p, a, b);
        return f2(a / (1.0f + expf(-a)), b / (1.0f + expf(-b)));
    }
}

template <bool FAST>
__device__ __forceinline__ float silu2(float a)
{
    if constexpr (FAST) return __fdividef(a, 1.0f + __expf(-a));
    else return a / (1.0f + expf(-a));
}

}  // namespace
}  // namespace ramnet
