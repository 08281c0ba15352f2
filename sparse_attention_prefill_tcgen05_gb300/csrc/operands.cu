// Rotary positions and the quantised operands and caches the indexer and the sparse
// attention read: rotation, quantising rows into cache slots, reading them back.
//
// Every kernel here reads its input once and writes its output once; what bounds them is
// HBM traffic (large calls) or launch latency (small ones).
#include <algorithm>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "indexer.h"
#include "internal.h"
#include "ptx.cuh"

namespace idx {
namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------ element types

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

// Eight elements at p (16-byte aligned) as fp32, and back with one rounding.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8])
{
    constexpr int n = sizeof(T) / 2;   // 16-byte words
    uint4 w[n];
#pragma unroll
    for (int i = 0; i < n; ++i)
        w[i] = reinterpret_cast<const uint4*>(p)[i];
    const T* e = reinterpret_cast<const T*>(w);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = Elt<T>::load(e[i]);
}

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

// Cosine and sine (times the amplitude) of pair i's turn at a position.  position * inc
// modulo 2^64 is the angle in 2^-64 turns, exactly; its top 32 bits as a signed number
// are half turns in [-1, 1), rounded once to fp32 (an error below 2e-7 rad at every
// position, where a 32-bit product of position and frequency would be off by 0.03 rad at
// position 487,935).
__device__ __forceinline__ float2 turn(const RopeParams& rp, int32_t pos, int i)
{
    const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(pos)) * rp.inc[i];
    const float half_turns =
        static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f;   // 2^-31
    float s, c;
    sincospif(half_turns, &s, &c);
    return make_float2(c * rp.amplitude, (rp.inverse ? -s : s) * rp.amplitude);
}

// A vector's 16 elements of one thread: unit u of the rotated part holds eight pairs, as
// eight elements at `a` and their partners at `b` (half layout) or as sixteen neighbours
// (interleaved; b = a + 8); units past the rotated part hold sixteen (or the last eight)
// other elements.
struct Unit {
    int a, b;       // element offsets of the two groups of eight; b < 0: only one
    bool rotated;
    int pair;       // first pair of a rotated unit
};

__device__ __forceinline__ Unit unit_of(const RopeParams& rp, int u, int D)
{
    Unit r;
    const int nrot = rp.rot / 16;
    r.rotated = u < nrot;
    r.pair = 8 * u;
    if (r.rotated) {
        r.a = rp.offset + (rp.interleaved ? 16 * u : 8 * u);
        r.b = rp.interleaved ? r.a + 8 : r.a + rp.rot / 2;
    } else {
        const int e = 16 * (u - nrot);          // among the elements left alone
        r.a = e < rp.offset ? e : e + rp.rot;
        const int f = e + 8;
        r.b = f >= D - rp.rot ? -1 : f < rp.offset ? f : f + rp.rot;
    }
    return r;
}

__device__ __forceinline__ void rotate16(bool interleaved, const float2 (&cs)[8], float (&a)[8],
                                         float (&b)[8])
{
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float(&v)[8] = i < 4 ? a : b;
            const int e = 2 * (i & 3);
            const float x = v[e], y = v[e + 1];
            v[e] = fmaf(x, cs[i].x, -y * cs[i].y);
            v[e + 1] = fmaf(x, cs[i].y, y * cs[i].x);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = a[i], y = b[i];
            a[i] = fmaf(x, cs[i].x, -y * cs[i].y);
            b[i] = fmaf(x, cs[i].y, y * cs[i].x);
        }
    }
}

// ------------------------------------------------------------------------- rotation

// One thread per (row, unit of 16 elements), for `hp` heads: the eight angles are computed
// once and turn that unit of every head.  Units that are left alone are copied (skipped
// when the output is the input itself).
template <typename T>
__global__ void __launch_bounds__(kThreads)
rope_kernel(const __grid_constant__ RopeParams rp, const __grid_constant__ RopeCall c, int units,
            int hp)
{
    pdl_wait_then_release();
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int t = static_cast<int>(i / units);
    if (t >= c.rows)
        return;
    const Unit u = unit_of(rp, static_cast<int>(i % units), c.D);
    const int h0 = blockIdx.y * hp, h1 = min(c.heads, h0 + hp);
    const T* x = static_cast<const T*>(c.x) + t * c.x_row;
    T* out = static_cast<T*>(c.out) + t * c.out_row;
    float2 cs[8];
    if (u.rotated) {
        const int32_t pos = c.positions[t];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            cs[k] = turn(rp, pos, u.pair + k);
    } else if (c.x == c.out) {
        return;
    }
#pragma unroll 4
    for (int h = h0; h < h1; ++h) {
        float a[8], b[8];
        load8(x + h * c.x_head + u.a, a);
        if (u.b >= 0)
            load8(x + h * c.x_head + u.b, b);
        if (u.rotated)
            rotate16(rp.interleaved, cs, a, b);
        store8(out + h * c.out_head + u.a, a);
        if (u.b >= 0)
            store8(out + h * c.out_head + u.b, b);
    }
}

// Any sizes, strides and alignment: one thread per (row, head, pair or other element).
template <typename T>
__global__ void __launch_bounds__(kThreads)
rope_any_kernel(const __grid_constant__ RopeParams rp, const __grid_constant__ RopeCall c)
{
    pdl_wait_then_release();
    const int pairs = rp.rot / 2, per = c.D - pairs;
    const int64_t n = (int64_t)c.rows * c.heads * per;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n;
         i += (int64_t)gridDim.x * kThreads) {
        const int e = static_cast<int>(i % per);
        const int64_t rh = i / per;
        const int h = static_cast<int>(rh % c.heads);
        const int64_t t = rh / c.heads;
        const T* x = static_cast<const T*>(c.x) + t * c.x_row + h * c.x_head;
        T* out = static_cast<T*>(c.out) + t * c.out_row + h * c.out_head;
        if (e < pairs) {
            const int a = rp.offset + (rp.interleaved ? 2 * e : e);
            const int b = rp.interleaved ? a + 1 : a + pairs;
            const float2 cs = turn(rp, c.positions[t], e);
            const float xa = Elt<T>::load(x[a]), xb = Elt<T>::load(x[b]);
            out[a] = Elt<T>::store(fmaf(xa, cs.x, -xb * cs.y));
            out[b] = Elt<T>::store(fmaf(xa, cs.y, xb * cs.x));
        } else if (c.x != c.out) {
            const int k = e - pairs;
            const int a = k < rp.offset ? k : k + rp.rot;
            out[a] = x[a];
        }
    }
}

// --------------------------------------------------------------------- quantisation

// |x| for the scale: NaN counts as 0 and infinities as the largest finite value, so a
// scale is always positive and finite.
__device__ __forceinline__ float magnitude(float x)
{
    return x == x ? fminf(fabsf(x), 3.402823466e38f) : 0.0f;
}

// e4m3 codes of eight values times `inv` (saturating, ties to even; NaN as 0, since the
// indexer takes no NaN codes).
__device__ __forceinline__ uint2 e4m3x8(const float (&v)[8], float inv)
{
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t r = 0;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float x = v[4 * i + 2 * j], y = v[4 * i + 2 * j + 1];
            x = x == x ? x * inv : 0.0f;
            y = y == y ? y * inv : 0.0f;
            r |= static_cast<uint32_t>(
                     __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3))
                 << (16 * j);
        }
        w[i] = r;
    }
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8], float inv)
{
    uint32_t r = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float x = v[2 * j], y = v[2 * j + 1];
        x = x == x ? x * inv : 0.0f;
        y = y == y ? y * inv : 0.0f;
        r |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(make_float2(x, y), __NV_E2M1,
                                                            cudaRoundNearest) &
                                   0xFFu)
             << (8 * j);
    }
    return r;
}

// Scale of an e4m3 row from its largest magnitude: amax / 448, never below the smallest
// normal number (so its reciprocal is finite), 1 for a zero row.
__device__ __forceinline__ float e4m3_scale(float amax)
{
    return amax > 0.0f ? fmaxf(amax / 448.0f, 1.17549435e-38f) : 1.0f;
}

// Biased exponent floor(log2(amax)) - 2 of an e2m1 block, clamped to ue8m0's 0..254; 127
// for a zero block.  A subnormal amax has an exponent below the clamp anyway.
__device__ __forceinline__ uint32_t e2m1_exponent(float amax)
{
    if (!(amax > 0.0f))
        return 127u;
    const int e = static_cast<int>(__float_as_uint(amax) >> 23) - 2;
    return static_cast<uint32_t>(max(e, 0));
}

// 2^(127 - e) for a biased exponent e in 0..252 (the exponents e2m1_exponent returns).
__device__ __forceinline__ float exp2_neg(uint32_t e) { return __uint_as_float((254u - e) << 23); }

// A group of `lanes` (a power of two, D / 16 rounded up) threads per (row, `hp` heads),
// one unit of 16 elements each, as in rope_kernel; the largest magnitude of the vector
// (e4m3) by a shuffle reduction over the group.  For e2m1 the scale covers 32 neighbours:
// the rotated vector is exchanged through shared memory so that a lane holds 16
// neighbouring elements and shares its scale with lane ^ 1.
template <typename T, bool kFp4>
__global__ void __launch_bounds__(kThreads)
cache_write_kernel(const __grid_constant__ RopeParams rp,
                   const __grid_constant__ CacheWriteCall c, int lanes, int hp)
{
    extern __shared__ float sm_rows[];   // kFp4: [threads][16] values
    pdl_wait_then_release();
    const int units = c.D / 16;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t t = i / lanes;
    const int l = static_cast<int>(i % lanes);
    const bool row_ok = t < c.rows;
    const int32_t slot = !row_ok ? -1 : c.slots ? c.slots[t] : static_cast<int32_t>(t);
    // a skipped row's lanes stay in the shuffles of the warp's other rows
    const bool keep = slot >= 0 && slot < c.num_slots;
    const bool on = keep && l < units;
    Unit u = unit_of(rp, l, c.D);
    float2 cs[8];
    if (on && u.rotated) {
        const int32_t pos = c.positions[t];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            cs[k] = turn(rp, pos, u.pair + k);
    }
    const int h0 = blockIdx.y * hp, h1 = min(c.heads, h0 + hp);
    const T* x = static_cast<const T*>(c.x) + (on ? t * c.x_row : 0);
    float* mine = kFp4 ? sm_rows + (threadIdx.x - l) * 16 : nullptr;   // the group's vector
#pragma unroll 2
    for (int h = h0; h < h1; ++h) {
        float a[8] = {}, b[8] = {};
        if (on) {
            load8(x + h * c.x_head + u.a, a);
            load8(x + h * c.x_head + u.b, b);
            if (u.rotated)
                rotate16(rp.interleaved, cs, a, b);
        }
        const int64_t vec = (int64_t)slot * c.heads + h;
        if (kFp4) {
            if (on) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    mine[u.a + k] = a[k];
                    mine[u.b + k] = b[k];
                }
            }
            __syncwarp();
            float m = 0.0f;
            if (on) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    a[k] = mine[16 * l + k];
                    b[k] = mine[16 * l + 8 + k];
                    m = fmaxf(m, fmaxf(magnitude(a[k]), magnitude(b[k])));
                }
            }
            __syncwarp();
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
            if (on) {
                const uint32_t e = e2m1_exponent(m);
                const float inv = exp2_neg(e);
                *reinterpret_cast<uint2*>(c.codes + vec * (c.D / 2) + 8 * l) =
                    make_uint2(e2m1x8(a, inv), e2m1x8(b, inv));
                if ((l & 1) == 0)
                    static_cast<uint8_t*>(c.scales)[vec * (c.D / 32) + l / 2] =
                        static_cast<uint8_t>(e);
            }
        } else {
            float m = 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                m = fmaxf(m, fmaxf(magnitude(a[k]), magnitude(b[k])));
            for (int d = lanes / 2; d > 0; d >>= 1)
                m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
            if (on) {
                const float s = e4m3_scale(m);
                const float inv = 1.0f / s;
                uint8_t* o = c.codes + vec * c.D;
                *reinterpret_cast<uint2*>(o + u.a) = e4m3x8(a, inv);
                *reinterpret_cast<uint2*>(o + u.b) = e4m3x8(b, inv);
                if (l == 0)
                    static_cast<float*>(c.scales)[vec] = s;
            }
        }
    }
}

// Any rotation (parts that are no multiple of eight elements) and any input alignment:
// one warp per (row, head), the vector in shared memory.
template <typename T, bool kFp4>
__global__ void __launch_bounds__(kThreads)
cache_write_any_kernel(const __grid_constant__ RopeParams rp,
                       const __grid_constant__ CacheWriteCall c)
{
    __shared__ float sm[kThreads / 32][kMaxHeadDim];
    pdl_wait_then_release();
    float* v = sm[threadIdx.x / 32];
    const int l = threadIdx.x & 31;
    const int64_t n = (int64_t)c.rows * c.heads;
    for (int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; i < n;
         i += (int64_t)gridDim.x * (kThreads / 32)) {
        const int64_t t = i / c.heads;
        const int h = static_cast<int>(i % c.heads);
        const int32_t slot = c.slots ? c.slots[t] : static_cast<int32_t>(t);
        if (slot < 0 || slot >= c.num_slots)
            continue;
        const T* x = static_cast<const T*>(c.x) + t * c.x_row + h * c.x_head;
        for (int e = l; e < c.D; e += 32)
            v[e] = Elt<T>::load(x[e]);
        __syncwarp();
        for (int p = l; p < rp.rot / 2; p += 32) {
            const int a = rp.offset + (rp.interleaved ? 2 * p : p);
            const int b = rp.interleaved ? a + 1 : a + rp.rot / 2;
            const float2 cs = turn(rp, c.positions[t], p);
            const float xa = v[a], xb = v[b];
            v[a] = fmaf(xa, cs.x, -xb * cs.y);
            v[b] = fmaf(xa, cs.y, xb * cs.x);
        }
        __syncwarp();
        const int64_t vec = (int64_t)slot * c.heads + h;
        float m = 0.0f;
        if (kFp4) {
            // lane l: the 32 elements of block l
            const int b = l < c.D / 32 ? l : 0;
            for (int e = 0; e < 32; ++e)
                m = fmaxf(m, magnitude(v[32 * b + e]));
            const uint32_t ex = e2m1_exponent(m);
            if (l < c.D / 32) {
                static_cast<uint8_t*>(c.scales)[vec * (c.D / 32) + l] = static_cast<uint8_t>(ex);
                for (int g = 0; g < 4; ++g) {
                    float w[8];
                    for (int k = 0; k < 8; ++k)
                        w[k] = v[32 * l + 8 * g + k];
                    *reinterpret_cast<uint32_t*>(c.codes + vec * (c.D / 2) + 16 * l + 4 * g) =
                        e2m1x8(w, exp2_neg(ex));
                }
            }
        } else {
            for (int e = l; e < c.D; e += 32)
                m = fmaxf(m, magnitude(v[e]));
            for (int d = 16; d > 0; d >>= 1)
                m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
            const float s = e4m3_scale(m);
            const float inv = 1.0f / s;
            if (l == 0)
                static_cast<float*>(c.scales)[vec] = s;
            if (l < c.D / 8) {
                float w[8];
                for (int k = 0; k < 8; ++k)
                    w[k] = v[8 * l + k];
                *reinterpret_cast<uint2*>(c.codes + vec * c.D + 8 * l) = e4m3x8(w, inv);
            }
        }
        __syncwarp();
    }
}

// ------------------------------------------------------------------------ read back

// Sixteen values of 16 e4m3 codes, or of one 8-byte half of a 32-code e2m1 block.
__device__ __forceinline__ void e4m3_values(uint2 w, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t two = ((i < 2 ? w.x : w.y) >> (16 * (i & 1))) & 0xFFFFu;
        const __half2_raw h =
            __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ void e2m1_values(uint32_t w, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(
            static_cast<__nv_fp4x2_storage_t>((w >> (8 * i)) & 0xFFu), __NV_E2M1);
        const float2 f = __half22float2(__half2(h));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

// One thread per 16 bytes of codes (16 e4m3 or 32 e2m1 codes, one scale) of a row.
template <typename T, bool kFp4>
__global__ void __launch_bounds__(kThreads)
cache_read_kernel(const __grid_constant__ CacheReadCall c, int chunks)
{
    pdl_wait_then_release();
    const int64_t n = (int64_t)c.rows * chunks;
    constexpr int kVals = kFp4 ? 32 : 16;
    const int per_vec = c.D / kVals;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n;
         i += (int64_t)gridDim.x * kThreads) {
        const int64_t t = i / chunks;
        const int k = static_cast<int>(i % chunks);
        const int32_t slot = c.slots ? c.slots[t] : static_cast<int32_t>(t);
        const bool ok = slot >= 0 && slot < c.num_slots;
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        float s = 1.0f;
        if (ok) {
            const int64_t at = (int64_t)slot * chunks + k;
            w = __ldg(reinterpret_cast<const uint4*>(c.codes) + at);
            if (kFp4)
                s = ldexpf(1.0f, static_cast<int>(__ldg(static_cast<const uint8_t*>(c.scales) + at)) -
                                     127);
            else
                s = __ldg(static_cast<const float*>(c.scales) + (int64_t)slot * c.heads +
                          k / per_vec);
        }
        T* o = static_cast<T*>(c.out) + i * kVals;
        float v[8];
        if (kFp4) {
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                e2m1_values(ws[g], v);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] *= s;
                store8(o + 8 * g, v);
            }
        } else {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                e4m3_values(g == 0 ? make_uint2(w.x, w.y) : make_uint2(w.z, w.w), v);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] *= s;
                store8(o + 8 * g, v);
            }
        }
    }
}

// Codes and scales as they are.  A row outside the cache reads as zero codes of scale 1.
__global__ void __launch_bounds__(kThreads)
cache_copy_kernel(const __grid_constant__ CacheReadCall c, int chunks)
{
    pdl_wait_then_release();
    const int64_t n = (int64_t)c.rows * chunks;
    const int per_vec = chunks / c.heads;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n;
         i += (int64_t)gridDim.x * kThreads) {
        const int64_t t = i / chunks;
        const int k = static_cast<int>(i % chunks);
        const int32_t slot = c.slots ? c.slots[t] : static_cast<int32_t>(t);
        const bool ok = slot >= 0 && slot < c.num_slots;
        const int64_t at = (int64_t)slot * chunks + k;
        reinterpret_cast<uint4*>(c.out)[i] =
            ok ? __ldg(reinterpret_cast<const uint4*>(c.codes) + at) : make_uint4(0u, 0u, 0u, 0u);
        if (c.fp4)
            static_cast<uint8_t*>(c.out_scales)[i] =
                ok ? static_cast<const uint8_t*>(c.scales)[at] : 127;
        else if (k % per_vec == 0)
            static_cast<float*>(c.out_scales)[i / per_vec] =
                ok ? static_cast<const float*>(c.scales)[at / per_vec] : 1.0f;
    }
}

__global__ void __launch_bounds__(kThreads)
page_slots_kernel(const __grid_constant__ PageSlotParams p)
{
    pdl_wait_then_release();
    const int total = p.key_begin[p.num_requests];
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * kThreads) {
        int lo = 0, hi = p.num_requests - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (p.key_begin[mid] <= i)
                lo = mid;
            else
                hi = mid - 1;
        }
        const int32_t j = static_cast<int32_t>(i) - p.key_begin[lo];
        const int64_t pg = p.table[(int64_t)lo * p.ld_table + j / p.page];
        const int64_t slot = pg * p.page + j % p.page;
        p.slots[i] = pg >= 0 && slot <= 0x7FFFFFFF ? static_cast<int32_t>(slot) : -1;
    }
}

// ------------------------------------------------------------------------- launches

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int elt_bytes(int dtype) { return dtype == IDX_FP32 ? 4 : 2; }

// Rows of 16-byte vectors: base and strides.
bool vector_rows(const void* p, int64_t row, int64_t head, int dtype)
{
    const int64_t v = 16 / elt_bytes(dtype);
    return aligned16(p) && row % v == 0 && head % v == 0;
}

// The rotated part divides into whole units of eight pairs on 8-element boundaries.
bool whole_units(const RopeParams& rp)
{
    return rp.rot % 16 == 0 && rp.offset % 8 == 0;
}

// Heads per thread: as many as leave two blocks per SM and more (angles shared by more
// heads), one where there are fewer rows than that.
int heads_per_thread(int64_t threads_per_head, int heads, int sms)
{
    int hp = 1;
    while (hp < 8 && hp * 2 <= heads && threads_per_head * (heads / (2 * hp)) >= (int64_t)sms * 2048)
        hp *= 2;
    return hp;
}

template <typename T>
cudaError_t rope_of(const RopeParams& rp, const RopeCall& c, cudaStream_t st)
{
    if (whole_units(rp) && c.D % 8 == 0 && vector_rows(c.x, c.x_row, c.x_head, c.dtype) &&
        vector_rows(c.out, c.out_row, c.out_head, c.dtype)) {
        const int units = rp.rot / 16 + (c.D - rp.rot + 15) / 16;
        const int64_t n = (int64_t)c.rows * units;
        const int hp = heads_per_thread(n, c.heads, device_sms());
        const dim3 grid(static_cast<unsigned>((n + kThreads - 1) / kThreads),
                        static_cast<unsigned>((c.heads + hp - 1) / hp));
        return launch_pdl(rope_kernel<T>, grid, dim3(kThreads), 0, st, rp, c, units, hp);
    }
    const int64_t n = (int64_t)c.rows * c.heads * (c.D - rp.rot / 2);
    const unsigned blocks =
        static_cast<unsigned>(std::min<int64_t>((n + kThreads - 1) / kThreads, 152 * 32));
    return launch_pdl(rope_any_kernel<T>, dim3(blocks), dim3(kThreads), 0, st, rp, c);
}

template <typename T, bool kFp4>
cudaError_t cache_write_of(const RopeParams& rp, const CacheWriteCall& c, cudaStream_t st)
{
    if (whole_units(rp) && vector_rows(c.x, c.x_row, c.x_head, c.dtype)) {
        int lanes = 2;
        while (lanes * 16 < c.D)
            lanes *= 2;
        const int64_t n = (int64_t)c.rows * lanes;
        const int hp = heads_per_thread(n, c.heads, device_sms());
        const dim3 grid(static_cast<unsigned>((n + kThreads - 1) / kThreads),
                        static_cast<unsigned>((c.heads + hp - 1) / hp));
        return launch_pdl(cache_write_kernel<T, kFp4>, grid, dim3(kThreads),
                          kFp4 ? kThreads * 16 * sizeof(float) : 0, st, rp, c, lanes, hp);
    }
    const int64_t n = (int64_t)c.rows * c.heads;
    const unsigned blocks = static_cast<unsigned>(
        std::min<int64_t>((n + kThreads / 32 - 1) / (kThreads / 32), 152 * 16));
    return launch_pdl(cache_write_any_kernel<T, kFp4>, dim3(blocks), dim3(kThreads), 0, st, rp, c);
}

unsigned stride_blocks(int64_t items)
{
    return static_cast<unsigned>(std::min<int64_t>((items + kThreads - 1) / kThreads, 152 * 64));
}

}  // namespace

cudaError_t launch_rope(const RopeParams& rp, const RopeCall& c, cudaStream_t st)
{
    if (c.rows <= 0)
        return cudaSuccess;
    return c.dtype == IDX_BF16   ? rope_of<__nv_bfloat16>(rp, c, st)
           : c.dtype == IDX_FP16 ? rope_of<__half>(rp, c, st)
                                 : rope_of<float>(rp, c, st);
}

cudaError_t launch_cache_write(const RopeParams& rp, const CacheWriteCall& c, cudaStream_t st)
{
    if (c.rows <= 0)
        return cudaSuccess;
    if (c.fp4)
        return c.dtype == IDX_BF16   ? cache_write_of<__nv_bfloat16, true>(rp, c, st)
               : c.dtype == IDX_FP16 ? cache_write_of<__half, true>(rp, c, st)
                                     : cache_write_of<float, true>(rp, c, st);
    return c.dtype == IDX_BF16   ? cache_write_of<__nv_bfloat16, false>(rp, c, st)
           : c.dtype == IDX_FP16 ? cache_write_of<__half, false>(rp, c, st)
                                 : cache_write_of<float, false>(rp, c, st);
}

cudaError_t launch_cache_read(const CacheReadCall& c, cudaStream_t st)
{
    if (c.rows <= 0)
        return cudaSuccess;
    const int chunks = c.heads * (c.fp4 ? c.D / 32 : c.D / 16);
    const dim3 grid(stride_blocks((int64_t)c.rows * chunks)), block(kThreads);
    if (c.out_dtype == IDX_CODES)
        return launch_pdl(cache_copy_kernel, grid, block, 0, st, c, chunks);
    if (c.fp4)
        return c.out_dtype == IDX_BF16
                   ? launch_pdl(cache_read_kernel<__nv_bfloat16, true>, grid, block, 0, st, c, chunks)
               : c.out_dtype == IDX_FP16
                   ? launch_pdl(cache_read_kernel<__half, true>, grid, block, 0, st, c, chunks)
                   : launch_pdl(cache_read_kernel<float, true>, grid, block, 0, st, c, chunks);
    return c.out_dtype == IDX_BF16
               ? launch_pdl(cache_read_kernel<__nv_bfloat16, false>, grid, block, 0, st, c, chunks)
           : c.out_dtype == IDX_FP16
               ? launch_pdl(cache_read_kernel<__half, false>, grid, block, 0, st, c, chunks)
               : launch_pdl(cache_read_kernel<float, false>, grid, block, 0, st, c, chunks);
}

cudaError_t launch_page_slots(const PageSlotParams& p, cudaStream_t st)
{
    const int total = p.key_begin[p.num_requests];
    if (total <= 0)
        return cudaSuccess;
    return launch_pdl(page_slots_kernel, dim3(stride_blocks(total)), dim3(kThreads), 0, st, p);
}

}  // namespace idx
