// Attention over the selected keys, and the block lists of candidate masks.
#include <algorithm>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "indexer.h"
#include "internal.h"
#include "ptx.cuh"

namespace idx {
namespace {

__device__ __forceinline__ int request_of(const int32_t* begin, int n, int64_t t)
{
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (begin[mid] <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// Cache slot of key position `c` of row t's list (entry c / block), or -1.
__device__ __forceinline__ int32_t selected_slot(const AttnParams& p, int64_t t, int r, int n_sel,
                                                 int len, int64_t c)
{
    const int64_t e = c >> p.block_shift;
    if (e >= n_sel)
        return -1;
    const int32_t s = p.sel[t * p.ld_sel + e];
    if (s < 0)
        return -1;
    const int64_t j = ((int64_t)s << p.block_shift) + (c & ((1 << p.block_shift) - 1));
    if (j >= len)
        return -1;
    if (p.page == 0) {
        const int64_t slot = p.key_begin[r] + j;
        return slot < p.num_slots ? static_cast<int32_t>(slot) : -1;
    }
    const int32_t page = static_cast<int32_t>(j) / p.page;
    const int64_t pg = p.table[r * p.ld_table + page];
    const int64_t slot = pg * p.page + (j - (int64_t)page * p.page);
    return pg >= 0 && slot < p.num_slots ? static_cast<int32_t>(slot) : -1;
}

template <typename T>
__device__ __forceinline__ float value(T v);
template <>
__device__ __forceinline__ float value(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float value(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float value(__nv_fp8_e4m3 v) { return static_cast<float>(v); }

// One warp per (row, query head): the keys one after another, the running maximum and sum
// of the softmax, D / 32 elements of the output per lane.
template <typename T, typename KV, int D>
__global__ void __launch_bounds__(128)
attention_kernel(const __grid_constant__ AttnParams p)
{
    pdl_wait_then_release();
    const int64_t item = (int64_t)blockIdx.x * 4 + threadIdx.x / 32;
    if (item >= (int64_t)p.rows * p.Hq)
        return;
    const int lane = threadIdx.x & 31;
    const int64_t t = item / p.Hq;
    const int h = static_cast<int>(item % p.Hq), g = h / p.group;
    const int r = request_of(p.row_begin, p.num_requests, t);
    const int len = min(p.clen[t], p.key_begin[r + 1] - p.key_begin[r]);
    const int n_sel = p.sel_count ? min(p.num_sel, p.sel_count[t]) : p.num_sel;
    constexpr int N = D / 32;
    float q[N], o[N] = {};
    for (int i = 0; i < N; ++i)
        q[i] = value(reinterpret_cast<const T*>(p.q + t * p.q_row + h * p.q_head)[lane + 32 * i]);
    float m = -INFINITY, l = 0.0f;
    bool any = false;
    const int64_t total = (int64_t)max(n_sel, 0) << p.block_shift;
    for (int64_t c0 = 0; c0 < total; c0 += 32) {
        const int32_t mine = selected_slot(p, t, r, n_sel, len, c0 + lane);
        for (int i = 0; i < 32; ++i) {
            const int64_t slot = __shfl_sync(0xFFFFFFFFu, mine, i);
            if (slot < 0)
                continue;
            any = true;
            const KV* kr = reinterpret_cast<const KV*>(p.k + slot * p.k_slot + g * p.k_head);
            const KV* vr = reinterpret_cast<const KV*>(p.v + slot * p.v_slot + g * p.v_head);
            float a = 0.0f;
            for (int x = 0; x < N; ++x)
                a = fmaf(q[x], value(kr[lane + 32 * x]), a);
            for (int d = 16; d > 0; d >>= 1)
                a += __shfl_xor_sync(0xFFFFFFFFu, a, d);
            a *= p.scale_log2 * (p.k_scale ? p.k_scale[slot * p.Hkv + g] : 1.0f);
            const float mn = fmaxf(m, a);
            const float f = m == mn ? 1.0f : exp2f(m - mn), w = exp2f(a - mn);
            const float sv = p.v_scale ? p.v_scale[slot * p.Hkv + g] : 1.0f;
            l = l * f + w;
            for (int x = 0; x < N; ++x)
                o[x] = o[x] * f + w * sv * value(vr[lane + 32 * x]);
            m = mn;
        }
    }
    T* out = reinterpret_cast<T*>(p.out + t * p.out_row + h * p.out_head);
    for (int x = 0; x < N; ++x)
        out[lane + 32 * x] = static_cast<T>(any ? o[x] / l : 0.0f);
    if (p.lse && lane == 0)
        p.lse[item] = any ? (m + log2f(l)) * 0.693147180559945309f : -INFINITY;
}

// One warp per row: 32 mask bytes at a time, each set byte's place by a ballot.
__global__ void __launch_bounds__(128)
mask_blocks_kernel(const __grid_constant__ MaskBlocksParams p)
{
    pdl_wait_then_release();
    const int64_t t = (int64_t)blockIdx.x * 4 + threadIdx.x / 32;
    if (t >= p.rows)
        return;
    const int lane = threadIdx.x & 31;
    const int r = request_of(p.row_begin, p.num_requests, t);
    const int len = max(0, min(p.clen[t], p.key_count[r]));
    const int nb = (len + p.block - 1) / p.block;
    const uint8_t* m = p.mask + t * p.ld_mask;
    int32_t* out = p.blocks + t * p.num_sel;
    int n = 0;
    for (int b0 = 0; b0 < nb && n < p.num_sel; b0 += 32) {
        const bool set = b0 + lane < nb && m[b0 + lane] != 0;
        const uint32_t bits = __ballot_sync(0xFFFFFFFFu, set);
        const int at = n + __popc(bits & ((1u << lane) - 1u));
        if (set && at < p.num_sel)
            out[at] = b0 + lane;
        n += __popc(bits);
    }
    n = min(n, p.num_sel);
    for (int i = n + lane; i < p.num_sel; i += 32)
        out[i] = -1;
    if (p.count && lane == 0)
        p.count[t] = n;
}

template <typename T, typename KV>
cudaError_t attention_of(const AttnParams& p, int D, cudaStream_t st)
{
    const unsigned blocks = static_cast<unsigned>(((int64_t)p.rows * p.Hq + 3) / 4);
    return D == 64 ? launch_pdl(attention_kernel<T, KV, 64>, dim3(blocks), dim3(128), 0, st, p)
                   : launch_pdl(attention_kernel<T, KV, 128>, dim3(blocks), dim3(128), 0, st, p);
}

}  // namespace

cudaError_t launch_attention(const AttnParams& p, int D, int dtype, bool fp8, cudaStream_t st)
{
    if (dtype == IDX_BF16)
        return fp8 ? attention_of<__nv_bfloat16, __nv_fp8_e4m3>(p, D, st)
                   : attention_of<__nv_bfloat16, __nv_bfloat16>(p, D, st);
    return fp8 ? attention_of<__half, __nv_fp8_e4m3>(p, D, st)
               : attention_of<__half, __half>(p, D, st);
}

cudaError_t launch_mask_blocks(const MaskBlocksParams& p, cudaStream_t st)
{
    return launch_pdl(mask_blocks_kernel, dim3(static_cast<unsigned>((p.rows + 3) / 4)), dim3(128),
                      0, st, p);
}

}  // namespace idx
