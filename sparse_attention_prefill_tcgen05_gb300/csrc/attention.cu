// Attention over the selected keys, and the block lists of candidate masks.
#include <algorithm>
#include <type_traits>
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

// ---------------------------------------------------------------- tensor-core kernel

// Modes: k and v of q's type (bf16 or fp16), or e4m3 caches under bf16 or fp16 queries.
constexpr int kModeBf16 = 0, kModeFp16 = 1, kModeFp8Bf16 = 2, kModeFp8Fp16 = 3;

// Tiles whose validity bits (and scales) are held for the softmax.  No barrier guards them:
// with d tiles in the ring of stages (d <= 4) the bits of tile n + 8 are written after the slots
// of tile n + 8 - d were read, thus after a v stage came free of tile n + 8 - 2 d >= n, whose
// weights were complete.
constexpr int kMaskDepth = 8;
constexpr long long kWaitCycles = 4000000000LL;   // about two seconds
constexpr int kSmemLimit = 232448;

template <int D, int NH, int MODE>
struct AttnCfg {
    static constexpr bool kFp8 = MODE >= kModeFp8Bf16;
    static constexpr int kQTerms = MODE == kModeFp8Bf16 ? 2 : MODE == kModeFp8Fp16 ? 3 : 1;
    static constexpr int kPTerms = kFp8 ? 2 : 1;
    static constexpr int kEb = kFp8 ? 1 : 2;            // bytes of an operand element
    static constexpr int kRow = D * kEb;                // bytes of a cached vector
    static constexpr int kAtom = kRow < 128 ? kRow : 128;
    static constexpr int kAtoms = kRow / kAtom;
    static constexpr int kStage = kAttnTile * kRow;
    static constexpr int kQRows = NH * kQTerms;
    static constexpr int kQBytes = kQRows * kRow;
    static constexpr int kPRow = NH * kPTerms * kEb;    // 2 NH
    static constexpr int kPBytes = kAttnTile * kPRow;
    static constexpr int kGroups = NH / 16;             // softmax warpgroups, 16 heads each
    static constexpr int kSoftmaxWarps = 4 * kGroups;
    
    // at most four tiles of stages, and the slots of as many tiles
    static constexpr int kSlotTile = kAttnTile * 4;
    static constexpr int kMaskBytes = kMaskDepth * (16 + (kFp8 ? kAttnTile * 8 : 0));
    static constexpr int kMisc =
        kMaskBytes + NH * 4 * 4 + 2 * NH * 4 + (kFp8 ? 2 * NH * 4 : 0) + 8 * (3 * 8 + 2 * 10 + 2);
    static constexpr int kFit = (kSmemLimit - kMisc - 2 * kPBytes - 2 * kQBytes) /
                                (2 * kStage + kSlotTile);
    // Tiles held.  A warp fills the same stage of the ring every time and reads the same
    // slot buffer, so it sees every phase of the barriers it waits on (a parity wait two
    // phases early would pass at once).
    static constexpr int kTiles = kFit < 4 ? kFit : 4;
    static constexpr int kStages = 2 * kTiles;
    static constexpr int kThreads = 32 * (kSoftmaxWarps + 4 + kStages + 2);
    static constexpr int kSmem =
        kStages * kStage + 2 * kPBytes + 2 * kQBytes + kTiles * kSlotTile + kMisc;
    static constexpr int kSCols = kQRows;               // TMEM columns of a score tile
    static constexpr int kOCols = NH * kPTerms;
    static constexpr int kCols = 2 * (kSCols + kOCols);
    static constexpr int kTmem = kCols <= 64 ? 64 : kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
    static_assert(kCols <= 512 && kTiles >= 2 && kSmem <= kSmemLimit, "tile does not fit");
};

// Byte offset in a tile of `W`-byte rows as the W-byte swizzle places it.
template <int W>
__device__ __forceinline__ uint32_t swizzled(uint32_t off)
{
    return off ^ (((off >> 7) & (W / 16 - 1)) << 4);
}

// Row `off` / W of such a tile (W-byte rows, off below 8 W) as what its chunks' addresses
// are combined with: for an address a whose bits from 16 up to the row are a chunk of row 0
// of an aligned group of 8 rows, a ^ swizzle_of(off) is that chunk of the row.
template <int W>
__device__ __forceinline__ constexpr uint32_t swizzle_of(uint32_t off)
{
    return off | (((off >> 7) & (W / 16 - 1)) << 4);
}

struct AttnItem {
    int t, g, ht, split;
    int n_sel;          // entries of the row
    int tile, tiles;    // key tiles [tile, tiles) of this item
};

__device__ __forceinline__ int quotient(int n, const Divisor& d)
{
    return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * d.mul) >> d.shift);
}

template <bool kOneLane = false>
__device__ __forceinline__ AttnItem attn_item(const AttnParams& p, int item)
{
    AttnItem w;
    int q = quotient(item, p.by_splits);
    w.split = item - q * p.splits;
    item = q;
    q = quotient(item, p.by_head_tiles);
    w.ht = item - q * p.head_tiles;
    item = q;
    q = quotient(item, p.by_hkv);
    w.g = item - q * p.Hkv;
    item = q;
    w.t = item;
    w.n_sel = p.num_sel;
    if (p.sel_count) {
        w.n_sel = max(0, min(p.num_sel, p.sel_count[w.t]));
        // (the shuffle tells the compiler that the count, and the loops over it, are uniform)
        if (!kOneLane)
            w.n_sel = __shfl_sync(0xFFFFFFFFu, w.n_sel, 0);
    }
    const int all = ((w.n_sel << p.block_shift) + kAttnTile - 1) / kAttnTile;
    w.tile = w.split * p.split_tiles;
    w.tiles = min(all, w.tile + p.split_tiles);
    return w;
}

// 16 values of every lane, combined over the warp: lane i ends with value i / 2.
template <bool kMax>
__device__ __forceinline__ float reduce16(const float (&v)[16])
{
    const int lane = threadIdx.x & 31;
    float a[8], b[4], c[2];
    auto op = [](float x, float y) { return kMax ? fmaxf(x, y) : x + y; };
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const bool up = lane & 16;
        const float r = __shfl_xor_sync(0xFFFFFFFFu, up ? v[i] : v[i + 8], 16);
        a[i] = op(up ? v[i + 8] : v[i], r);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool up = lane & 8;
        const float r = __shfl_xor_sync(0xFFFFFFFFu, up ? a[i] : a[i + 4], 8);
        b[i] = op(up ? a[i + 4] : a[i], r);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const bool up = lane & 4;
        const float r = __shfl_xor_sync(0xFFFFFFFFu, up ? b[i] : b[i + 2], 4);
        c[i] = op(up ? b[i + 2] : b[i], r);
    }
    const bool up = lane & 2;
    const float r = __shfl_xor_sync(0xFFFFFFFFu, up ? c[0] : c[1], 2);
    const float d = op(up ? c[1] : c[0], r);
    return op(d, __shfl_xor_sync(0xFFFFFFFFu, d, 1));
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// The rest of a wait that is not over at once.  Out of line: the roles' loops together have to
// stay in the instruction cache (with every wait inlined a third of the fetches missed it).
__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, volatile int* ab,
                                     uint32_t* status)
{
    if (mbar_wait(bar, parity, kWaitCycles, ab))
        return true;
    if (!*ab) {
        *ab = 1;
        atomicOr(status, kStatusTimeout);
    }
    return false;
}

template <int D, int NH, int MODE>
__global__ void __launch_bounds__(AttnCfg<D, NH, MODE>::kThreads, 1)
attention_tc_kernel(const __grid_constant__ AttnParams p)
{
    using C = AttnCfg<D, NH, MODE>;
    using T = typename std::conditional<MODE == kModeBf16 || MODE == kModeFp8Bf16, __nv_bfloat16,
                                        __half>::type;
    extern __shared__ __align__(1024) uint8_t sm[];
    uint8_t* stages = sm;
    uint8_t* pbuf = stages + C::kStages * C::kStage;
    uint8_t* qbuf = pbuf + 2 * C::kPBytes;
    int32_t* slots = reinterpret_cast<int32_t*>(qbuf + 2 * C::kQBytes);   // [kTiles][128]
    uint32_t* mask = reinterpret_cast<uint32_t*>(slots + C::kTiles * kAttnTile);   // [kMaskDepth][4]
    float* exch = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(mask) + C::kMaskBytes);
    float* factor = exch + C::kGroups * 64;                    // [2][NH]: of an item's output
    float* qscale = factor + 2 * NH;                           // [2][NH]
    uint64_t* bars = reinterpret_cast<uint64_t*>(qscale + (C::kFp8 ? 2 * NH : 0));
    uint64_t* kv_full = bars;
    uint64_t* kv_empty = kv_full + C::kStages;
    uint64_t* slot_full = kv_empty + C::kStages;
    uint64_t* slot_empty = slot_full + C::kTiles;
    uint64_t* q_full = slot_empty + C::kTiles;
    uint64_t* q_empty = q_full + 2;
    uint64_t* s_full = q_empty + 2;
    uint64_t* s_empty = s_full + 2;
    uint64_t* p_full = s_empty + 2;
    uint64_t* p_empty = p_full + 2;
    uint64_t* o_full = p_empty + 2;
    uint64_t* o_empty = o_full + 2;
    uint64_t* f_full = o_empty + 2;
    uint64_t* f_empty = f_full + 2;
    uint64_t* drained = f_empty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x / 32), 0);
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(kv_full + i, 1);
            mbar_init(kv_empty + i, 1);
        }
        for (int i = 0; i < C::kTiles; ++i) {
            mbar_init(slot_full + i, 1);
            mbar_init(slot_empty + i, 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full + i, 1);
            mbar_init(q_empty + i, 1);
            mbar_init(s_full + i, 1);
            mbar_init(s_empty + i, C::kSoftmaxWarps);
            mbar_init(p_full + i, C::kSoftmaxWarps);
            mbar_init(p_empty + i, 1);
            mbar_init(o_full + i, 1);
            mbar_init(o_empty + i, 4);
            mbar_init(f_full + i, C::kSoftmaxWarps);
            mbar_init(f_empty + i, 4);
        }
        mbar_init(drained, 1);
        // the swizzled tiles need their 1024-byte boundaries
        *abort_flag = (smem_u32(sm) & 1023u) != 0;
        fence_mbar_init();
    }
    constexpr int kGatherWarp = C::kSoftmaxWarps + 4;
    constexpr int kSlotWarp = kGatherWarp + C::kStages, kMmaWarp = kSlotWarp + 1;
    if (warp == kMmaWarp) {
        tmem_alloc(tmem_slot, C::kTmem);
        tmem_relinquish();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tmem_s = tmem, tmem_o = tmem + 2 * C::kSCols;
    pdl_wait_then_release();
    // The status word is cleared by the call itself; a wait that gives up sets it a whole
    // wait budget later.
    if (blockIdx.x == 0 && threadIdx.x == 0)
        *p.status = *abort_flag ? kStatusBadArg : 0u;

    const int total = p.rows * p.Hkv * p.head_tiles * p.splits;
    volatile int* ab = abort_flag;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        return mbar_try_wait(bar, parity) || wait_on(bar, parity, ab, p.status);
    };

    if (warp < C::kSoftmaxWarps) {
        // ---------------------------------------------------------------- softmax
        // Thread = one key of the tile (a TMEM lane) x 16 heads.
        const int wg = warp / 4, quad = warp & 3, key = 32 * quad + lane;
        const uint32_t lanes = static_cast<uint32_t>(32 * quad) << 16;
        const int bar_id = 1 + wg;
        float* x4 = exch + wg * 64;                  // [4 quadrants][16 heads]
        bool bad = false, out_of_here = false;
        int n = 0, iq = 0;
        for (int item = blockIdx.x; item < total && !out_of_here; item += gridDim.x) {
            const AttnItem w = attn_item(p, item);
            float m[16], l[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                m[i] = -3.0e38f;
                l[i] = 0.0f;
            }
            for (int j = w.tile; j < w.tiles; ++j, ++n) {
                const int b = n & 1;
                bad |= !wait(s_full + b, (n >> 1) & 1);
                tc_fence_after();
                float x[16];
                tmem_ld_32x32b_x16(tmem_s + lanes + b * C::kSCols + 16 * wg, x);
                tmem_wait_ld();
                tc_fence_before();
                // (the scores' arrival implies the mask's)
                const uint32_t ok = mask[(n % kMaskDepth) * 4 + quad];
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(s_empty + b);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    x[i] *= p.scale_log2;
                if (ok != 0xFFFFFFFFu) {
                    const bool mine = (ok >> lane) & 1u;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        x[i] = mine ? x[i] : -INFINITY;
                }
                float over = x[0] - m[0];
#pragma unroll
                for (int i = 1; i < 16; ++i)
                    over = fmaxf(over, x[i] - m[i]);
                // The running maximum is replaced only where a score passes it by more than
                // 2^8: weights then stay below 2^8, and most tiles need no rescaling of the
                // accumulated output (and no exchange over the keys).
                const bool first = j == w.tile;
                if (first || bar_any(over > 8.0f || bad, bar_id, 128)) {
                    float v[16];
                    const float mine = reduce16<true>(x);
                    if (first)
                        bar_all(true, bar_id, 128);  // the last item's sums have been read
                    if ((lane & 1) == 0)
                        x4[quad * 16 + lane / 2] = mine;
                    if (!bar_all(!bad, bar_id, 128)) {
                        out_of_here = true;
                        break;
                    }
                    float f[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float mn =
                            fmaxf(fmaxf(fmaxf(m[i], x4[i]), fmaxf(x4[16 + i], x4[32 + i])),
                                  x4[48 + i]);
                        f[i] = ex2(m[i] - mn);
                        m[i] = mn;
                        l[i] *= f[i];
                    }
                    if (!first) {
                        // the products of the tiles before are complete
                        bad |= !wait(p_empty + ((n - 1) & 1), ((n - 1) >> 1) & 1);
                        tc_fence_after();
                        const uint32_t at = tmem_o + lanes + (iq & 1) * C::kOCols + 16 * wg;
                        tmem_ld_32x32b_x16(at, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            v[i] *= f[i];
                        tmem_st_32x32b_x16(at, v);
                        tmem_wait_st();
                        tc_fence_before();
                    }
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    x[i] = ex2(x[i] - m[i]);   // a key that is none: 0
                    l[i] += x[i];
                }
                bad |= !wait(p_empty + b, ((n >> 1) & 1) ^ 1);
                uint8_t* prow = pbuf + b * C::kPBytes;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const uint4 v4 = make_uint4(
                        pack2<T>(x[8 * c], x[8 * c + 1]), pack2<T>(x[8 * c + 2], x[8 * c + 3]),
                        pack2<T>(x[8 * c + 4], x[8 * c + 5]), pack2<T>(x[8 * c + 6], x[8 * c + 7]));
                    *reinterpret_cast<uint4*>(
                        prow + swizzled<C::kPRow>(key * C::kPRow + 32 * wg + 16 * c)) = v4;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(p_full + b);
            }
            if (out_of_here)
                break;
            if (w.tiles == w.tile)
                continue;
            // The item's sums; the epilogue's warps get 1 / sum (the output waits for the last
            // product, the next item's first scores do not).
            const float mine = reduce16<false>(l);
            if (!bar_all(!bad, bar_id, 128))             // the last maxima have been read
                break;
            if ((lane & 1) == 0)
                x4[quad * 16 + lane / 2] = mine;
            bad |= !wait(f_empty + (iq & 1), ((iq >> 1) & 1) ^ 1);
            if (!bar_all(!bad, bar_id, 128))
                break;
            if (quad == 0) {
                const int i = lane & 15;
                float mi = 0.0f;
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    mi = i == k ? m[k] : mi;
                const float li = (x4[i] + x4[16 + i]) + (x4[32 + i] + x4[48 + i]);
                if (lane < 16) {
                    const int h = w.ht * NH + 16 * wg + i;
                    factor[(iq & 1) * NH + 16 * wg + i] =
                        p.splits > 1 ? 1.0f : li == 0.0f ? 0.0f : 1.0f / li;
                    if (p.splits > 1)
                        reinterpret_cast<float2*>(p.part_ml)[(int64_t)item * NH + 16 * wg + i] =
                            make_float2(mi, li);
                    else if (p.lse && h < p.group)
                        p.lse[(int64_t)w.t * p.Hq + w.g * p.group + h] =
                            (mi + log2f(li)) * 0.693147180559945309f;
                }
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(f_full + (iq & 1));
            ++iq;
        }
    } else if (warp < kGatherWarp) {
        // --------------------------------------------------------------- epilogue
        // Thread = one element (of D) of NH heads.
        const int quad = warp & 3, dim = 32 * quad + lane;
        const uint32_t lanes = static_cast<uint32_t>(32 * quad) << 16;
        int iq = 0;
        bool ok = true;
        for (int item = blockIdx.x; item < total && ok; item += gridDim.x) {
            const AttnItem w = attn_item(p, item);
            const bool some = w.tiles > w.tile;
            uint8_t* out = p.out + w.t * p.out_row + (int64_t)(w.g * p.group + w.ht * NH) * p.out_head;
            const int heads = min(NH, p.group - w.ht * NH);
            if (some) {
                ok = wait(f_full + (iq & 1), (iq >> 1) & 1) && wait(o_full + (iq & 1), (iq >> 1) & 1);
                if (!__all_sync(0xFFFFFFFFu, ok))
                    break;
                tc_fence_after();
            }
            const bool parts = p.splits > 1, write = D == 128 || dim < D;
            const int count = parts ? NH : heads;
            float* part = p.part_o + (int64_t)item * NH * D + dim;
#pragma unroll 1
            for (int h0 = 0; h0 < count; h0 += 16) {
                float o[16] = {};
                if (some) {
                    tmem_ld_32x32b_x16(tmem_o + lanes + (iq & 1) * C::kOCols + h0, o);
                    tmem_wait_ld();
                }
                if (parts) {
                    float* to = part + h0 * D;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (write)
                            to[i * D] = o[i];
                } else {
                    const float* f = factor + (iq & 1) * NH + h0;
                    uint8_t* to = out + h0 * p.out_head + 2 * dim;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float v = f[i] != 0.0f ? o[i] * f[i] : 0.0f;
                        if (write && h0 + i < heads)
                            *reinterpret_cast<T*>(to) = static_cast<T>(some ? v : 0.0f);
                        to += p.out_head;
                    }
                }
            }
            if (!some) {
#pragma unroll 1
                for (int h = dim; h < count; h += kAttnTile) {
                    if (parts)
                        reinterpret_cast<float2*>(p.part_ml)[(int64_t)item * NH + h] =
                            make_float2(-3.0e38f, 0.0f);
                    else if (p.lse)
                        p.lse[(int64_t)w.t * p.Hq + w.g * p.group + w.ht * NH + h] = -INFINITY;
                }
            }
            if (some) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(o_empty + (iq & 1));
                    mbar_arrive(f_empty + (iq & 1));
                }
                ++iq;
            }
        }
    } else if (warp < kSlotWarp) {
        // ---------------------------------------------------------------- gather
        // Warp i fills stage i of the ring: it waits for the stage, copies the 128 vectors
        // (zeros for keys that are none), waits for its own copies and signals.  The other
        // stages' warps keep the memory system busy meanwhile.
        const int pw = warp - kGatherWarp;
        constexpr int kPerRow = C::kRow / 16;            // copies of 16 bytes a vector takes
        constexpr int kSpans = 32 / kPerRow;             // vectors copied at a time,
        constexpr int kSpan = kAttnTile / kSpans;        // kSpan keys apart
        const int chunk = lane % kPerRow, row0 = lane / kPerRow * kSpan;
        const uint32_t stage = smem_u32(stages + pw * C::kStage) + row0 * C::kAtom +
                               (chunk * 16 / C::kAtom) * (kAttnTile * C::kAtom) +
                               (chunk * 16) % C::kAtom;
        const bool is_v = pw & 1;
        const uint8_t* kv = (is_v ? p.v : p.k) + chunk * 16;
        const int64_t kv_head = is_v ? p.v_head : p.k_head;
        const uint32_t kv_slot = static_cast<uint32_t>(is_v ? p.v_slot : p.k_slot);
        const int sl = pw / 2;                   // the pair's place in the ring of tiles
        int n = 0, uses = 0;
        bool ok = true;
        for (int item = blockIdx.x; item < total && ok; item += gridDim.x) {
            const AttnItem w = attn_item(p, item);
            const int end = n + max(0, w.tiles - w.tile);
            const uint8_t* src = kv + w.g * kv_head;
            // the pair's tiles of the item
            for (int m = uses * C::kTiles + sl; m < end; m += C::kTiles) {
                ok = wait(kv_empty + pw, (uses & 1) ^ 1) && wait(slot_full + sl, uses & 1);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok)
                    break;
                const int32_t* rows = slots + sl * kAttnTile + row0;
                const uint4 bits = *reinterpret_cast<const uint4*>(mask + (m % kMaskDepth) * 4);
                if ((bits.x & bits.y & bits.z & bits.w) == 0xFFFFFFFFu) {
#pragma unroll 1
                    for (int i = 0; i < kSpan; i += 8) {
                        const int4 s0 = *reinterpret_cast<const int4*>(rows + i);
                        const int4 s1 = *reinterpret_cast<const int4*>(rows + i + 4);
                        const int32_t s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            cp_async16((stage + i * C::kAtom) ^ swizzle_of<C::kAtom>(k * C::kAtom),
                                       src + (uint64_t)(uint32_t)s[k] * kv_slot);
                    }
                } else {
#pragma unroll 1
                    for (int i = 0; i < kSpan; ++i) {
                        const int32_t s = rows[i];
                        cp_async16((stage + i / 8 * 8 * C::kAtom) ^
                                       swizzle_of<C::kAtom>(i % 8 * C::kAtom),
                                   src + (uint64_t)(uint32_t)max(s, 0) * kv_slot, s >= 0);
                    }
                }
                cp_async_commit();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(slot_empty + sl);
                cp_async_wait<0>();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(kv_full + pw);
                ++uses;
            }
            n = end;
        }
    } else if (warp == kSlotWarp) {
        // ----------------------------------------------------------------- slots
        // Cache slots of the selected keys, four keys of a tile per lane.  The list entries are
        // read two tiles ahead and their pages one tile ahead, over the items' ends.
        struct Tile {
            int item, t, g, ht, base, r, len, tile;      // item < 0: no tile
        };
        Tile d1{-1}, d2{-1};                             // whose pages, whose entries are read
        int32_t entry[4] = {}, key[4] = {}, page[4] = {};
        AttnItem w;
        w.tile = w.tiles = w.n_sel = 0;
        int next_item = blockIdx.x, r = 0, base = 0, len = 0;
        int n = 0, iq = 0, last_item = -1, drain = 0;
        bool ok = true;
        while (ok && drain < 3) {
            // tile n: slots from its pages
            int32_t slot[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t at = (int64_t)page[i] * p.page + key[i];
                slot[i] = page[i] >= 0 && at < p.num_slots ? static_cast<int32_t>(at) : -1;
            }
            const Tile d0 = d1;
            // tile n + 1: keys and pages from its entries
            d1 = d2;
            if (d1.item >= 0) {
                const int32_t* table = p.table + d1.r * p.ld_table;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int pos = d1.tile * kAttnTile + 32 * i + lane;
                    const int64_t k = ((int64_t)entry[i] << p.block_shift) +
                                      (pos & ((1 << p.block_shift) - 1));
                    const bool in = entry[i] >= 0 && k < d1.len;
                    key[i] = static_cast<int32_t>(k);
                    page[i] = in ? 0 : -1;
                    if (p.page == 0) {
                        key[i] += d1.base;
                    } else if (in) {
                        const int pg = quotient(key[i], p.by_page);
                        page[i] = table[pg];
                        key[i] -= pg * p.page;
                    }
                }
            }
            // tile n + 2: entries
            while (w.tile >= w.tiles && next_item < total) {
                w = attn_item(p, next_item);
                r = request_of(p.row_begin, p.num_requests, w.t);
                base = p.key_begin[r];
                len = min(p.clen[w.t], p.key_begin[r + 1] - base);
                next_item += gridDim.x;
            }
            d2 = Tile{-1};
            if (w.tile < w.tiles) {
                d2 = Tile{next_item, w.t, w.g, w.ht, base, r, len, w.tile};
                const int32_t* sel = p.sel + w.t * p.ld_sel;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int at = (w.tile * kAttnTile + 32 * i + lane) >> p.block_shift;
                    entry[i] = at < w.n_sel ? sel[at] : -1;
                }
                ++w.tile;
            }
            drain = d2.item < 0 ? drain + 1 : 0;
            if (d0.item < 0)
                continue;
            const bool new_item = d0.item != last_item;
            if (new_item) {
                // the item's queries, before its first tile
                ok = wait(q_empty + (iq & 1), ((iq >> 1) & 1) ^ 1);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok)
                    break;
                constexpr int kPerRow = C::kRow / 16;
                const uint8_t* q = p.q + d0.t * p.q_row + (int64_t)d0.g * p.group * p.q_head;
                const uint32_t dst = smem_u32(qbuf + (iq & 1) * C::kQBytes);
#pragma unroll 1
                for (int i = lane; i < C::kQBytes / 16; i += 32) {
                    const int h = i / kPerRow, c16 = i % kPerRow;
                    const bool in = d0.ht * NH + h < p.group;
                    const uint32_t off = (c16 / 8) * (NH * 128) + h * 128 + (c16 % 8) * 16;
                    cp_async16(dst + swizzled<128>(off),
                               in ? q + (int64_t)(d0.ht * NH + h) * p.q_head + c16 * 16 : q, in);
                }
                cp_async_commit();
            }
            ok = wait(slot_empty + n % C::kTiles, ((n / C::kTiles) & 1) ^ 1);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok)
                break;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                slots[(n % C::kTiles) * kAttnTile + 32 * i + lane] = slot[i];
                const uint32_t bits = __ballot_sync(0xFFFFFFFFu, slot[i] >= 0);
                if (lane == i)
                    mask[(n % kMaskDepth) * 4 + i] = bits;
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(slot_full + n % C::kTiles);
            if (new_item) {
                cp_async_wait<0>();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(q_full + (iq & 1));
                ++iq;
                last_item = d0.item;
            }
            ++n;
        }
    } else {
        // --------------------------------------------------------------------- MMA
        constexpr int kK = 32 / C::kEb;                 // contraction elements of one MMA
        constexpr uint32_t idesc_s =
            idesc_dense(128, C::kQRows, MODE == kModeBf16 ? 1 : 0, false, false);
        constexpr uint32_t idesc_o =
            idesc_dense(128, C::kOCols, MODE == kModeBf16 ? 1 : 0, true, true);
        // One elected lane waits and issues.
        if (elect_one()) {
            struct Pending {
                bool any, first, last;
                int n, iq;
            } pv{false, false, false, 0, 0};
            const uint64_t k_desc = smem_desc(smem_u32(stages), C::kAtom, 16, 8 * C::kAtom);
            // v rows are keys: both operands of the second product are read along their rows.
            // D = 64 takes the same 64 elements for both halves of the 128 output rows.
            constexpr uint32_t lbo = C::kAtoms > 1 ? kAttnTile * C::kAtom : 0;
            const uint64_t v_desc = smem_desc(smem_u32(stages), C::kAtom, lbo, 8 * C::kAtom);
            const uint64_t q_desc = smem_desc(smem_u32(qbuf), C::kAtom, 16, 8 * C::kAtom);
            const uint64_t p_desc = smem_desc(smem_u32(pbuf), C::kPRow, 0, 8 * C::kPRow);
            int vst = 0;                                // the pending product's stage
            auto product = [&]() {                      // O += P V of a tile
                const int b = pv.n & 1;
                if (!(wait(kv_full + vst, (pv.n / C::kTiles) & 1) &&
                      (!pv.first || wait(o_empty + (pv.iq & 1), ((pv.iq >> 1) & 1) ^ 1)) &&
                      wait(p_full + b, (pv.n >> 1) & 1)))
                    return false;
                tc_fence_after();
                const uint64_t a0 = v_desc + vst * (C::kStage / 16);
                const uint64_t b0 = p_desc + b * (C::kPBytes / 16);
                const uint32_t d = tmem_o + (pv.iq & 1) * C::kOCols;
#pragma unroll
                for (int k = 0; k < kAttnTile / kK; ++k)
                    mma_f16(d, a0 + k * (kK * C::kAtom / 16), b0 + k * (kK * C::kPRow / 16),
                            idesc_o, !pv.first || k > 0);
                mma_commit(kv_empty + vst);
                mma_commit(p_empty + b);
                if (pv.last)
                    mma_commit(o_full + (pv.iq & 1));
                return true;
            };
            int n = 0, iq = 0, st = 0;                  // st: the k stage of tile n
            int item = blockIdx.x, j = 0, first = 0, end = 0;
            if (item < total) {
                const AttnItem w = attn_item<true>(p, item);
                first = j = w.tile;
                end = w.tiles;
            }
            while (true) {
                while (j >= end && (item += gridDim.x) < total) {
                    const AttnItem w = attn_item<true>(p, item);
                    first = j = w.tile;
                    end = w.tiles;
                }
                const bool more = j < end;
                const Pending next{more, j == first, j + 1 == end, n, iq};
                const int next_st = st + 1;
                if (more) {                             // S = Q K of tile n
                    const int b = n & 1;
                    if (!((!next.first || wait(q_full + (iq & 1), (iq >> 1) & 1)) &&
                          wait(kv_full + st, (n / C::kTiles) & 1) &&
                          wait(s_empty + b, ((n >> 1) & 1) ^ 1)))
                        break;
                    tc_fence_after();
                    const uint64_t a0 = k_desc + st * (C::kStage / 16);
                    const uint64_t b0 = q_desc + (iq & 1) * (C::kQBytes / 16);
#pragma unroll
                    for (int k = 0; k < D / kK; ++k) {
                        const int atom = k * 32 / C::kAtom, in = (k * 32) % C::kAtom;
                        mma_f16(tmem_s + b * C::kSCols,
                                a0 + (atom * (kAttnTile * C::kAtom) + in) / 16,
                                b0 + (atom * (C::kQRows * C::kAtom) + in) / 16, idesc_s, k > 0);
                    }
                    mma_commit(s_full + b);
                    mma_commit(kv_empty + st);
                    if (next.last)
                        mma_commit(q_empty + (iq & 1));
                    iq += next.last;
                    ++j;
                    ++n;
                    st = st + 2 == C::kStages ? 0 : st + 2;
                }
                if (pv.any && !product())
                    break;
                if (!more)
                    break;
                pv = next;
                vst = next_st;
            }
            // what was issued, and its arrivals, end before the memory goes
            mma_commit(drained);
            volatile int never = 0;
            mbar_wait(drained, 0, kWaitCycles, &never);
        }
        __syncwarp();
    }
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmem);
    }
}

// Split rows: the partial outputs of a row and head, weighted by their running maxima.  One
// warp per (row, query head).
template <typename T, int D>
__global__ void __launch_bounds__(128)
attention_join_kernel(const __grid_constant__ AttnParams p, int nh)
{
    pdl_wait_then_release();
    const int64_t i = (int64_t)blockIdx.x * 4 + threadIdx.x / 32;
    if (i >= (int64_t)p.rows * p.Hq)
        return;
    const int lane = threadIdx.x & 31;
    const int64_t t = i / p.Hq;
    const int h = static_cast<int>(i % p.Hq), g = h / p.group, hg = h % p.group;
    const int64_t item0 = ((t * p.Hkv + g) * p.head_tiles + hg / nh) * p.splits;
    const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
    float m = -3.0e38f;
    for (int s = 0; s < p.splits; ++s)
        m = fmaxf(m, ml[(item0 + s) * nh + hg % nh].x);
    constexpr int N = D / 32;
    float o[N] = {}, l = 0.0f;
    for (int s = 0; s < p.splits; ++s) {
        const int64_t at = (item0 + s) * nh + hg % nh;
        const float2 v = ml[at];
        const float f = ex2(v.x - m);
        l = fmaf(v.y, f, l);
#pragma unroll
        for (int k = 0; k < N; ++k)
            o[k] = fmaf(p.part_o[at * D + lane + 32 * k], f, o[k]);
    }
    T* out = reinterpret_cast<T*>(p.out + t * p.out_row + h * p.out_head);
#pragma unroll
    for (int k = 0; k < N; ++k)
        out[lane + 32 * k] = static_cast<T>(l == 0.0f ? 0.0f : o[k] / l);
    if (p.lse && lane == 0)
        p.lse[i] = (m + log2f(l)) * 0.693147180559945309f;
}

template <int D, int NH, int MODE>
cudaError_t attention_tc(const AttnParams& p, cudaStream_t st)
{
    using C = AttnCfg<D, NH, MODE>;
    static const cudaError_t attr =
        cudaFuncSetAttribute(attention_tc_kernel<D, NH, MODE>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (attr != cudaSuccess)
        return attr;
    const int items = p.rows * p.Hkv * p.head_tiles * p.splits;
    return launch_pdl(attention_tc_kernel<D, NH, MODE>, dim3(std::min(items, device_sms())),
                      dim3(C::kThreads), C::kSmem, st, p);
}

template <int D, int MODE>
cudaError_t attention_heads(const AttnParams& p, int nh, cudaStream_t st)
{
    cudaError_t e = nh == 16   ? attention_tc<D, 16, MODE>(p, st)
                    : nh == 32 ? attention_tc<D, 32, MODE>(p, st)
                               : attention_tc<D, 64, MODE>(p, st);
    if (e != cudaSuccess || p.splits == 1)
        return e;
    using T = typename std::conditional<MODE == kModeBf16, __nv_bfloat16, __half>::type;
    count_launch();
    const unsigned blocks = static_cast<unsigned>(((int64_t)p.rows * p.Hq + 3) / 4);
    return launch_pdl(attention_join_kernel<T, D>, dim3(blocks), dim3(128), 0, st, p, nh);
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

int attention_heads_per_tile(int group, int dtype, bool fp8)
{
    (void)dtype;
    (void)fp8;
    return group <= 16 ? 16 : group <= 32 ? 32 : 64;
}

cudaError_t launch_attention(const AttnParams& p, int D, int dtype, bool fp8, cudaStream_t st)
{
    if (!fp8) {
        const int nh = attention_heads_per_tile(p.group, dtype, fp8);
        if (dtype == IDX_BF16)
            return D == 64 ? attention_heads<64, kModeBf16>(p, nh, st)
                           : attention_heads<128, kModeBf16>(p, nh, st);
        return D == 64 ? attention_heads<64, kModeFp16>(p, nh, st)
                       : attention_heads<128, kModeFp16>(p, nh, st);
    }
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
