// Elements of the operators' rows: eight at a time between memory and fp32, and as e4m3 codes.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

namespace idx {

template <typename T>
struct Elt;
template <>
struct Elt<__nv_bfloat16> {
    static __device__ __forceinline__ float load(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __forceinline__ __nv_bfloat16 store(float v) { return __float2bfloat16(v); }
};
template <>
struct Elt<__half> {
    static __device__ __forceinline__ float load(__half v) { return __half2float(v); }
    static __device__ __forceinline__ __half store(float v) { return __float2half(v); }
};
template <>
struct Elt<float> {
    static __device__ __forceinline__ float load(float v) { return v; }
    static __device__ __forceinline__ float store(float v) { return v; }
};

// Eight elements at p (16-byte aligned), to fp32, and back with one rounding.
template <typename T>
struct Eight {
    uint4 w[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* p)
    {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
            w[i] = reinterpret_cast<const uint4*>(p)[i];
    }
    __device__ __forceinline__ void values(float (&v)[8]) const
    {
        const T* e = reinterpret_cast<const T*>(w);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = Elt<T>::load(e[i]);
    }
};

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8])
{
    constexpr int n = sizeof(T) / 2;
    uint4 w[n];
    T* e = reinterpret_cast<T*>(w);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        e[i] = Elt<T>::store(v[i]);
#pragma unroll
    for (int i = 0; i < n; ++i)
        reinterpret_cast<uint4*>(p)[i] = w[i];
}

// Two fp32 values in a 64-bit register: one instruction for both.
__device__ __forceinline__ uint64_t pack(float x, float y)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void unpack(uint64_t v, float& x, float& y)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// The largest magnitude of eight values.  NaN becomes 0, since the indexer takes no NaN codes:
// the maximum that passes a NaN on shows whether there is one, so values without any pay one
// compare instead of sixteen instructions.
__device__ __forceinline__ float largest(float (&v)[8])
{
    float m = fabsf(v[0]);
#pragma unroll
    for (int i = 1; i < 7; i += 2)
        asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(fabsf(v[i])), "f"(fabsf(v[i + 1])));
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(v[7])));
    if (m == m)
        return m;
    m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = v[i] == v[i] ? v[i] : 0.0f;
        m = fmaxf(m, fabsf(v[i]));
    }
    return m;
}

// e4m3 codes of eight values over `scale` (saturating, ties to even).  The quotient is the fp32 one:
// x inv, inv the rounded reciprocal, less what that is too much (Markstein's theorem: a faithful
// quotient and a correctly rounded reciprocal give the correctly rounded quotient; the signs keep
// that of a zero).  x inv alone took 42 us instead of 45 for 16,384 rows, but values half way between
// two codes, such as three quarters of their vector's largest, went to either.
__device__ __forceinline__ uint2 e4m3x8(const float (&v)[8], float scale, float inv)
{
    uint32_t two[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t q = mul2(pack(v[2 * i], v[2 * i + 1]), pack(inv, inv));
        const uint64_t over = fma2(q, pack(scale, scale), pack(-v[2 * i], -v[2 * i + 1]));
        float2 f;
        unpack(fma2(over, pack(-inv, -inv), q), f.x, f.y);
        two[i] = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
    }
    return make_uint2(two[0] | two[1] << 16, two[2] | two[3] << 16);
}

// Infinite values as the largest finite one (they would leave a NaN of a quotient).
__device__ __forceinline__ void finite8(float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = fminf(fmaxf(v[i], -3.402823466e38f), 3.402823466e38f);
}

// Scale of an e4m3 row from its largest magnitude (an infinite one as the largest finite
// value): amax / 448, never below the smallest normal number (so its reciprocal is finite), 1
// for a zero row.  The division as above: 1 / 448 is a constant.
__device__ __forceinline__ float e4m3_scale(float amax)
{
    amax = fminf(amax, 3.402823466e38f);
    constexpr float kInv = 1.0f / 448.0f;
    const float q = amax * kInv;
    return amax > 0.0f ? fmaxf(fmaf(fmaf(q, -448.0f, amax), kInv, q), 1.17549435e-38f) : 1.0f;
}

}  // namespace idx
