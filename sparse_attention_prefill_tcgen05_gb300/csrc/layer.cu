// What stands in front of and behind a layer's attention: the norm whose output its projections
// read, and the join of attentions over disjoint keys.
//
// Both read their inputs once and write their outputs once; HBM bounds them (large calls) or the
// launch (small ones).
#include <algorithm>

#include "indexer.h"
#include "elements.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace idx {
namespace {

// ------------------------------------------------------------------------------- norm
//
//     h = x + residual,   y = h / sqrt(mean h^2 + eps) * weight
//
// in fp32, h and y rounded once where they are stored; codes are e4m3(y / s) of the unrounded y, s
// the largest |y| of its group over 448.

// Sum or maximum over a block, in every thread.  `part`: 32 floats of shared memory of its own.
template <bool kMax>
__device__ __forceinline__ float block_reduce(float v, float* part)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const float o = __shfl_xor_sync(0xFFFFFFFFu, v, d);
        v = kMax ? fmaxf(v, o) : v + o;
    }
    const int warps = blockDim.x / 32;
    if (warps == 1)
        return v;
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x / 32] = v;
    __syncthreads();
    v = (threadIdx.x & 31) < warps ? part[threadIdx.x & 31] : 0.0f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const float o = __shfl_xor_sync(0xFFFFFFFFu, v, d);
        v = kMax ? fmaxf(v, o) : v + o;
    }
    return v;
}

// A block per row, which stays in registers (one read of it, one write of each output): eights of
// neighbours, V a thread, a warp's side by side, so that a group's eights are neighbouring lanes.  16,384
// rows of 7,168 bf16 with residual and e4m3 codes: 170 us (6.2 TB/s of the 6.8 a copy reaches), HBM
// bounds it; 64 rows 12 us, the call on the host.  Rows above 32,768 elements (V = 8) do not fit: some 5 KB
// a thread go through local memory, and 256 rows of 65,536 take 176 us, of 32,768 16.
template <typename T, typename W, int V>
__global__ void __launch_bounds__(1024)
norm_kernel(const __grid_constant__ NormCall c)
{
    __shared__ float part[2][32];
    pdl_wait_then_release();
    const int64_t t = blockIdx.x;
    const int eights = c.n / 8;
    const T* x = static_cast<const T*>(c.x) + t * c.x_row;
    Eight<T> wx[V], wr[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int i = k * blockDim.x + threadIdx.x;
        if (i < eights)
            wx[k].load(x + 8 * i);
    }
    if (c.residual) {
        const T* r = static_cast<const T*>(c.residual) + t * c.residual_row;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int i = k * blockDim.x + threadIdx.x;
            if (i < eights)
                wr[k].load(r + 8 * i);
        }
    }
    float h[V][8], sum = 0.0f;
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int i = k * blockDim.x + threadIdx.x;
        if (i >= eights) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                h[k][e] = 0.0f;
            continue;
        }
        wx[k].values(h[k]);
        if (c.residual) {
            float r[8];
            wr[k].values(r);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                h[k][e] += r[e];
            if (c.total)
                store8(static_cast<T*>(c.total) + t * c.total_row + 8 * i, h[k]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            sum = fmaf(h[k][e], h[k][e], sum);
    }
    sum = block_reduce<false>(sum, part[0]);
    const float f = 1.0f / sqrtf(sum / static_cast<float>(c.n) + c.eps);
    float all = 0.0f;
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int i = k * blockDim.x + threadIdx.x;
        if (i < eights) {
            float w[8];
            if (c.weight) {
                Eight<W> ww;
                ww.load(static_cast<const W*>(c.weight) + 8 * i);
                ww.values(w);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[k][e] *= f;
                if (c.weight)
                    h[k][e] *= w[e];
            }
            if (c.out)
                store8(static_cast<T*>(c.out) + t * c.out_row + 8 * i, h[k]);
        }
        if (c.codes && c.group != c.n) {
            // (the lanes of a group have a place in the row together, or none)
            float m = largest(h[k]);
            for (int d = c.group / 16; d > 0; d >>= 1)
                m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
            if (i < eights) {
                const float s = e4m3_scale(m);
                if (m == INFINITY)
                    finite8(h[k]);
                *reinterpret_cast<uint2*>(c.codes + t * c.n + 8 * i) = e4m3x8(h[k], s, 1.0f / s);
                if (8 * i % c.group == 0)
                    c.scales[t * (c.n / c.group) + 8 * i / c.group] = s;
            }
        } else if (c.codes) {
            all = fmaxf(all, largest(h[k]));
        }
    }
    if (c.codes && c.group == c.n) {
        all = block_reduce<true>(all, part[1]);
        const float s = e4m3_scale(all), inv = 1.0f / s;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int i = k * blockDim.x + threadIdx.x;
            if (i >= eights)
                continue;
            if (all == INFINITY)
                finite8(h[k]);
            *reinterpret_cast<uint2*>(c.codes + t * c.n + 8 * i) = e4m3x8(h[k], s, inv);
        }
        if (threadIdx.x == 0)
            c.scales[t] = s;
    }
}

// Any size and alignment: a thread takes every blockDim-th element.  Codes need their group's
// largest magnitude from other threads: maxima of non-negative floats as integers in shared
// memory, whose order does not matter.
template <typename T, typename W, int V>
__global__ void __launch_bounds__(1024)
norm_any_kernel(const __grid_constant__ NormCall c)
{
    __shared__ float part[32];
    __shared__ int maxima[kMaxNorm / 32];
    pdl_wait_then_release();
    const int64_t t = blockIdx.x;
    const T* x = static_cast<const T*>(c.x) + t * c.x_row;
    const T* r = static_cast<const T*>(c.residual) + t * c.residual_row;
    const int groups = c.codes ? c.n / c.group : 0;
    for (int i = threadIdx.x; i < groups; i += blockDim.x)
        maxima[i] = 0;
    float h[V], sum = 0.0f;
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int i = k * blockDim.x + threadIdx.x;
        h[k] = 0.0f;
        if (i < c.n) {
            h[k] = Elt<T>::load(x[i]);
            if (c.residual)
                h[k] += Elt<T>::load(r[i]);
        }
        sum = fmaf(h[k], h[k], sum);
    }
    sum = block_reduce<false>(sum, part);
    const float f = 1.0f / sqrtf(sum / static_cast<float>(c.n) + c.eps);
    if (groups)
        __syncthreads();
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int i = k * blockDim.x + threadIdx.x;
        if (i >= c.n)
            continue;
        if (c.residual && c.total)
            static_cast<T*>(c.total)[t * c.total_row + i] = Elt<T>::store(h[k]);
        h[k] *= f;
        if (c.weight)
            h[k] *= Elt<W>::load(static_cast<const W*>(c.weight)[i]);
        if (c.out)
            static_cast<T*>(c.out)[t * c.out_row + i] = Elt<T>::store(h[k]);
        if (groups) {
            h[k] = h[k] == h[k] ? h[k] : 0.0f;
            atomicMax(maxima + i / c.group, __float_as_int(fabsf(h[k])));
        }
    }
    if (!groups)
        return;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int i = k * blockDim.x + threadIdx.x;
        if (i >= c.n)
            continue;
        const float s = e4m3_scale(__int_as_float(maxima[i / c.group]));
        float v[8] = {h[k]};
        finite8(v);
        c.codes[t * c.n + i] = static_cast<uint8_t>(e4m3x8(v, s, 1.0f / s).x & 0xFFu);
        if (i % c.group == 0)
            c.scales[t * groups + i / c.group] = s;
    }
}

bool vectors(const void* p, int64_t row, int bytes)
{
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && row * bytes % 16 == 0;
}

template <typename T, typename W>
cudaError_t norm_of(const NormCall& c, cudaStream_t st)
{
    constexpr int eb = sizeof(T);
    const dim3 grid(static_cast<unsigned>(c.rows));
    const auto block = [](int threads) { return dim3(static_cast<unsigned>((threads + 31) / 32 * 32)); };
    if (c.n % 8 == 0 && vectors(c.x, c.x_row, eb) && vectors(c.residual, c.residual_row, eb) &&
        vectors(c.total, c.total_row, eb) && vectors(c.out, c.out_row, eb) &&
        vectors(c.weight, 0, eb) && reinterpret_cast<uintptr_t>(c.codes) % 8 == 0) {
        const int eights = c.n / 8;
        if (eights <= 128)
            return launch_pdl(norm_kernel<T, W, 1>, grid, block(eights), 0, st, c);
        if (eights <= 512)
            return launch_pdl(norm_kernel<T, W, 2>, grid, block((eights + 1) / 2), 0, st, c);
        if (eights <= 4096)
            return launch_pdl(norm_kernel<T, W, 4>, grid, block((eights + 3) / 4), 0, st, c);
        return launch_pdl(norm_kernel<T, W, 8>, grid, block((eights + 7) / 8), 0, st, c);
    }
    if (c.n <= 8192)
        return launch_pdl(norm_any_kernel<T, W, 8>, grid, block((c.n + 7) / 8), 0, st, c);
    return launch_pdl(norm_any_kernel<T, W, 64>, grid, dim3(1024), 0, st, c);
}

// ------------------------------------------------------------------------------- join
//
//     lse = log(sum_p exp(lse_p) + exp(sink)),   out = sum_p exp(lse_p - lse) out_p
//
// A part whose lse is -inf has no key and is not read.

// 16,384 x 64 vectors of 128, three parts: 170 us (6.4 TB/s); 256 threads 175, 64 263; 64 rows 7.4 us, the
// call on the host.
constexpr int kJoinThreads = 128;

__device__ __forceinline__ int quotient(int n, const Divisor& d)
{
    return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * d.mul) >> d.shift);
}

// The weights of a vector's parts, relative to their sum (and the sink's part of it); its lse is
// ref + log2(sum) ln 2.  A vector's threads each compute them: instructions bound the kernel next to HBM,
// so exponentials and the quotient are the approximate ones (2^-22 of a weight).
template <int P>
__device__ __forceinline__ void join_weights(const JoinCall& c, int vec, int head, float (&w)[P],
                                             float& ref, float& sum)
{
    constexpr float kLog2e = 1.4426950408889634f;
    const float none = c.sink ? c.sink[head] : -INFINITY;
    float m = none;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        w[p] = p < c.parts ? c.part_lse[p][vec] : -INFINITY;
        m = fmaxf(m, w[p]);
    }
    ref = m == -INFINITY ? 0.0f : m;
    sum = c.sink ? ex2((none - ref) * kLog2e) : 0.0f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        w[p] = ex2((w[p] - ref) * kLog2e);
        sum += w[p];
    }
    const float inv = sum == 0.0f ? 0.0f : __fdividef(1.0f, sum);
#pragma unroll
    for (int p = 0; p < P; ++p)
        w[p] *= inv;
}

__device__ __forceinline__ float join_lse(float ref, float sum)
{
    return sum == 0.0f ? -INFINITY : fmaf(log2f(sum), 0.693147180559945309f, ref);
}

// D / 8 threads a vector (row, head), eight elements each; the parts' loads are under way together.
// (With 64-bit divisions, IEEE quotients and a logarithm in every thread 204 us, 84 % of the issue slots.)
template <typename T, typename O, int P>
__global__ void __launch_bounds__(kJoinThreads)
join_kernel(const __grid_constant__ JoinCall c)
{
    pdl_wait_then_release();
    const int lanes = c.D / 8, groups = kJoinThreads / lanes;
    const int g = threadIdx.x / lanes, l = threadIdx.x - g * lanes;
    const int n = c.rows * c.heads, vec = blockIdx.x * groups + g;
    const bool on = g < groups && vec < n && vec >= 0;
    float ref = 0.0f, sum = 0.0f;
    if (on) {
        const int t = quotient(vec, c.by_heads);
        const int h = vec - t * c.heads;
        Eight<T> v[P];
#pragma unroll
        for (int p = 0; p < P; ++p)
            if (p < c.parts)
                v[p].load(static_cast<const T*>(c.part[p]) + t * c.part_row[p] + h * c.part_head[p] +
                          8 * l);
        float w[P];
        join_weights<P>(c, vec, h, w, ref, sum);
        float o[8] = {};
#pragma unroll
        for (int p = 0; p < P; ++p) {
            if (p >= c.parts || w[p] == 0.0f)
                continue;
            float x[8];
            v[p].values(x);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                o[e] = fmaf(w[p], x[e], o[e]);
        }
        store8(static_cast<O*>(c.out) + t * c.out_row + h * c.out_head + 8 * l, o);
    }
    if (!c.lse)
        return;
    // (lse may be one of the parts': every thread of the vector has read it)
    __syncthreads();
    if (on && l == 0)
        c.lse[vec] = join_lse(ref, sum);
}

// Any size and alignment: a warp a vector.
template <typename T, typename O>
__global__ void __launch_bounds__(kJoinThreads)
join_any_kernel(const __grid_constant__ JoinCall c)
{
    pdl_wait_then_release();
    const int64_t vec = (int64_t)blockIdx.x * (kJoinThreads / 32) + threadIdx.x / 32;
    if (vec >= (int64_t)c.rows * c.heads)
        return;
    const int lane = threadIdx.x & 31;
    const int t = quotient(static_cast<int>(vec), c.by_heads);
    const int h = static_cast<int>(vec) - t * c.heads;
    float w[kMaxParts], ref, sum;
    join_weights<kMaxParts>(c, static_cast<int>(vec), h, w, ref, sum);
    for (int e = lane; e < c.D; e += 32) {
        float o = 0.0f;
#pragma unroll
        for (int p = 0; p < kMaxParts; ++p)
            if (p < c.parts && w[p] != 0.0f)
                o = fmaf(w[p],
                         Elt<T>::load(static_cast<const T*>(c.part[p])[t * c.part_row[p] +
                                                                       h * c.part_head[p] + e]),
                         o);
        static_cast<O*>(c.out)[t * c.out_row + h * c.out_head + e] = Elt<O>::store(o);
    }
    __syncwarp();
    if (lane == 0 && c.lse)
        c.lse[vec] = join_lse(ref, sum);
}

template <typename T, typename O>
cudaError_t join_of(const JoinCall& c, cudaStream_t st)
{
    const int64_t n = (int64_t)c.rows * c.heads;
    bool whole = c.D % 8 == 0 && vectors(c.out, c.out_row, sizeof(O)) &&
                 vectors(c.out, c.out_head, sizeof(O));
    for (int p = 0; p < c.parts; ++p)
        whole = whole && vectors(c.part[p], c.part_row[p], sizeof(T)) &&
                vectors(c.part[p], c.part_head[p], sizeof(T));
    if (!whole)
        return launch_pdl(join_any_kernel<T, O>,
                          dim3(static_cast<unsigned>((n + kJoinThreads / 32 - 1) / (kJoinThreads / 32))),
                          dim3(kJoinThreads), 0, st, c);
    const int groups = kJoinThreads / (c.D / 8);
    const dim3 grid(static_cast<unsigned>((n + groups - 1) / groups));
    if (c.parts <= 2)
        return launch_pdl(join_kernel<T, O, 2>, grid, dim3(kJoinThreads), 0, st, c);
    if (c.parts == 3)
        return launch_pdl(join_kernel<T, O, 3>, grid, dim3(kJoinThreads), 0, st, c);
    if (c.parts == 4)
        return launch_pdl(join_kernel<T, O, 4>, grid, dim3(kJoinThreads), 0, st, c);
    return launch_pdl(join_kernel<T, O, kMaxParts>, grid, dim3(kJoinThreads), 0, st, c);
}

}  // namespace

cudaError_t launch_norm(const NormCall& c, cudaStream_t st)
{
    if (c.dtype == IDX_FP32)
        return norm_of<float, float>(c, st);
    if (c.dtype == IDX_BF16)
        return c.weight_fp32 ? norm_of<__nv_bfloat16, float>(c, st)
                             : norm_of<__nv_bfloat16, __nv_bfloat16>(c, st);
    return c.weight_fp32 ? norm_of<__half, float>(c, st) : norm_of<__half, __half>(c, st);
}

cudaError_t launch_join(const JoinCall& c, cudaStream_t st)
{
    if (c.part_dtype == IDX_FP32)
        return c.out_dtype == IDX_BF16   ? join_of<float, __nv_bfloat16>(c, st)
               : c.out_dtype == IDX_FP16 ? join_of<float, __half>(c, st)
                                         : join_of<float, float>(c, st);
    return c.part_dtype == IDX_BF16 ? join_of<__nv_bfloat16, __nv_bfloat16>(c, st)
                                    : join_of<__half, __half>(c, st);
}

}  // namespace idx
