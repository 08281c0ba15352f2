// Attention of single rows over keys of their own on the tensor cores: the keys a row's list names
// (indexer_sparse_attention), or those of a range (indexer_causal_attention's single tokens).
#pragma once
#include <algorithm>
#include <atomic>
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

template <typename T>
__device__ __forceinline__ float value(T v);
template <>
__device__ __forceinline__ float value(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float value(__half v) { return __half2float(v); }

// ---------------------------------------------------------------- tensor-core kernel
//
// A work item is a row, a key/value head, a tile of NH query heads and a part of the row's key
// tiles; a persistent block per SM takes items in turn.  Per tile of 128 selected keys:
//     S^T [keys x heads] = K Q^T,   P = exp2(S scale log2(e) - reference),   O^T += V^T P
// in one pass: the reference per head is replaced (and O and the sums rescaled) only when a score
// leaves its range, the sums are kept per key lane and added up once per item.  Keys are the MMA's
// 128 rows, so a group of 16 heads fills the tensor cores' rows as well as one of 64, softmax
// needs no exchange between threads for a key, and V is read transposed where it lies.
//
// What it has to do is gather: a row's keys are its own, so T x S x Hkv x 2 x D elements come
// through L2 whatever the tiling (2,048 rows x 2,048 keys of 128 bf16: 2.1 GB; only the 64 MB
// behind them come from HBM once).  cp.async of 16 bytes by a warp per stage moved 21 TB/s alone,
// gathering TMA 9, plain loads 14.  Around it the roles overlap, each a warp or more of its own:
// gather (two warps per tile of the ring, which also look up its slots and convert e4m3 values),
// scores, products, two softmax warpgroups, four warps for queries and outputs, one of each ahead
// of or behind the others by a tile or an item.  All waits are bounded.  Rows that do not fill the
// SMs are split over blocks, two or four of them a cluster that joins its parts in shared memory (64
// rows over 2,048 e4m3 keys, 32 heads: 14.0 us, 8 of them the latency of a single tile).
//
// Roundings: scores, maxima, sums and outputs are fp32; weights are rounded to bf16 (fp16 under fp16
// keys, two bf16 terms under fp16 queries over e4m3 caches) because the tensor cores take 16-bit
// operands at twice tf32's rate and half its bytes in shared memory, which bounds the kernel, and
// roundings of 2^-8 of a weight at most, of either sign, add up to less than the output's own: over
// 2,048 x 2,048 bf16 keys it is off by 0.0024 of its size where fp32 weights leave 0.0017, the
// output's rounding alone.
//
// Measured (GB300; items fill the SMs): 32 heads of 128 over 2,048 bf16 keys, 2,048 rows 176 us
// (12.2 TB/s gathered, 390 TFLOP/s), 64 heads 234 us (587 TFLOP/s), 16 heads 152 us; e4m3 caches 219,
// 302 and 190 us; 512 keys of 16,384 rows, 64 heads, e4m3: 0.76 ms.  What bounds it: shared memory at
// 32 heads (a tile's 64 KB are written once and read by two MMAs: 1,220 of its 1,600 cycles; e4m3
// tiles too, whose values are written twice), the softmax warps' chain of waits, exponentials and
// conversions at 64, the instruction cache throughout (all roles' loops are some 60 KB; at 100 KB
// a third of the fetches missed and everything took a third longer).

// Modes: k and v of q's type (bf16 or fp16), or e4m3 caches under bf16 or fp16 queries.
constexpr int kModeBf16 = 0, kModeFp16 = 1, kModeFp8Bf16 = 2, kModeFp8Fp16 = 3;

// Polls of a wait, each suspended for up to about a microsecond: a tenth of a second at least,
// several at most.
constexpr int kWaitTries = 1 << 22;
constexpr int kGaveUp = 2;   // in the block's abort flag
constexpr int kSmemLimit = 232448;
// Items whose query scales are held.  No barrier guards them: the scales of item i + 4 are
// written after the scores of item i + 2's last tile were issued, and the scores of a tile are
// issued after those of the tile two before were read.
constexpr int kScaleItems = 4;

template <int D, int NH, int MODE>
struct AttnCfg {
    static constexpr bool kFp8 = MODE >= kModeFp8Bf16;
    static constexpr int kQTerms = MODE == kModeFp8Bf16 ? 2 : MODE == kModeFp8Fp16 ? 3 : 1;
    // Keys meet the queries as they are cached.  Values of e4m3 caches become bf16 in shared memory
    // (exactly), so that a weight, times its value's scale, keeps a bf16 number's range and its 8
    // bits whatever the sizes of the list's other weights and scales.  As e4m3 terms relative to the
    // largest product, which saved the conversion, weights ended at 2^-18 of it: a value of zeros
    // (scale 1) or a long list took the others' place.  fp16 outputs have 11 bits: a second bf16
    // term holds what is left of a weight, into the same accumulator.
    static constexpr int kPTerms = MODE == kModeFp8Fp16 ? 2 : 1;
    static constexpr bool kWide = MODE != kModeFp16;    // weights have an fp32 number's range
    static constexpr int kEb = kFp8 ? 1 : 2;            // bytes of a cached element
    static constexpr int kRow = D * kEb;                // bytes of a cached vector
    static constexpr int kAtom = kRow < 128 ? kRow : 128;
    static constexpr int kKStage = kAttnTile * kRow;
    static constexpr int kVStage = kAttnTile * D * 2;
    static constexpr int kTileBytes = kKStage + kVStage;
    static constexpr int kQRows = NH * kQTerms;
    static constexpr int kQBytes = kQRows * kRow;
    static constexpr int kPRow = NH * 2;
    static constexpr int kPTile = kAttnTile * kPRow;    // of a term
    static constexpr int kPBytes = kPTerms * kPTile;
    // Two softmax warpgroups.  Up to 32 heads they take alternate tiles of an item, each with
    // an output accumulator, running maximum and sum of its own (joined by the epilogue): a
    // tile's chain of waits, exponentials and stores then overlaps the next tile's.  64 heads
    // are shared between them, 32 each.
    static constexpr bool kAlternate = NH <= 32;
    static constexpr int kHeads = NH < 32 ? NH : 32;    // heads of a softmax thread
    static constexpr int kTileWarps = kAlternate ? 4 : 8;   // softmax warps that take a tile
    static constexpr int kAccs = kAlternate ? 2 : 1;    // accumulators of an item
    static constexpr int kSCols = kQRows;               // TMEM columns of a score tile
    static constexpr int kOCols = NH;                   // of an accumulator
    static constexpr int kCols = 2 * kSCols + 2 * kAccs * kOCols;
    static constexpr int kTmem = kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
    // Shared memory after the stages, the weights and the queries.
    static constexpr int kStats = 2 * 4 * kHeads * 4;   // sums by warpgroup and quadrant
    static constexpr int kMax = 2 * kHeads * 4;         // maxima by warpgroup
    static constexpr int kQScale = kFp8 ? (kScaleItems + 1) * NH * 4 : 0;
    static constexpr int kKeyInfo = kAttnTile * (kFp8 ? 9 : 1);   // of a tile, 2 kTiles of them
    static constexpr int kFixed = kStats + kMax + kQScale + 2 * kPBytes + 2 * kQBytes + 8 * 21;
    static constexpr int kFit =
        (kSmemLimit - kFixed) / (kTileBytes + 2 * kKeyInfo + 8 * 4);
    // Tiles in the ring: three; four where the stages are small and so few heads leave the
    // softmax's registers free (16 heads of 128, e4m3 190 us against 193 with three; 8 heads of 64
    // 103 against 109, e4m3 143 against 155; but 32 heads of 64 143 against 134, e4m3 250 against 187:
    // two more warps, fewer registers each).
    static constexpr int kMostTiles = NH == 16 && kTileBytes <= 49152 ? 4 : 3;
    static constexpr int kTiles = kFit < kMostTiles ? kFit : kMostTiles;   // tiles in the ring
    static constexpr int kStages = 2 * kTiles;          // and as many warps that fill them
    static constexpr int kSmem = kFixed + kTiles * (kTileBytes + 2 * kKeyInfo + 8 * 4);
    static constexpr int kGatherWarp = 8 + 4, kMmaWarp = kGatherWarp + kStages;
    static constexpr int kThreads = 32 * (kMmaWarp + 2);
    // Registers: the softmax warpgroups hold a thread's heads twice over (scores and sums), what
    // feeds them (gather and MMA warps) needs few, so where the block is whole warpgroups they
    // trade: at 96 each the 32-head loops spill (e4m3, 32 heads 219 -> 272 us, 64 heads 302 -> 339).
    // What is traded was launched with: 640 threads of 96.  32 heads take 136 against 56 (176 us; 128
    // against 64: 180), 16 heads 128 against 64 (152 us; 136 against 56 the same, without 157).
    static constexpr bool kTrade = kThreads == 640;
    static constexpr int kSoftmaxRegs = kHeads == 32 ? 136 : 128;
    static constexpr int kFeedRegs = kHeads == 32 ? 56 : 64;
    static constexpr int kLaunchRegs = 96;
    static_assert(256 * kSoftmaxRegs + 128 * kLaunchRegs + 256 * kFeedRegs <= 640 * kLaunchRegs,
                  "registers");
    static_assert(NH * D * 4 <= kTiles * kTileBytes && NH * 8 <= kStages * kAttnTile,
                  "a split's part in shared memory");
    static_assert(kCols <= 512 && kTiles >= 2 && kSmem <= kSmemLimit, "tile does not fit");
};

// Byte offset in a tile of `W`-byte rows as the W-byte swizzle places it.
template <int W>
__device__ __forceinline__ constexpr uint32_t swizzled(uint32_t off)
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
    int len;            // kRange: its length
    int tile, tiles;    // key tiles [tile, tiles) of this item
};

__device__ __forceinline__ int quotient(int n, const Divisor& d)
{
    return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * d.mul) >> d.shift);
}

// The entries of an item's row (kRange: the row's length), read an item ahead of its use: every role
// walks the items.
template <bool kRange>
__device__ __forceinline__ int item_entries(const AttnParams& p, int item, int total)
{
    if constexpr (kRange) {
        if (item >= total)
            return 0;
        const int t = quotient(quotient(quotient(item, p.by_splits), p.by_head_tiles), p.by_hkv);
        const int r = request_of(p.row_begin, p.num_requests, t);
        return max(0, min(p.clen[t], p.key_begin[r + 1] - p.key_begin[r]));
    }
    if (!p.sel_count || item >= total)
        return p.num_sel;
    return p.sel_count[quotient(quotient(quotient(item, p.by_splits), p.by_head_tiles), p.by_hkv)];
}

template <bool kRange, bool kOneLane = false>
__device__ __forceinline__ AttnItem attn_item(const AttnParams& p, int item, int entries)
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
    w.t = q;
    if constexpr (kRange) {
        // a list without a list: the first keys under a window, then those up to the row's length
        w.len = kOneLane ? entries : __shfl_sync(0xFFFFFFFFu, entries, 0);
        w.n_sel = p.window > 0 && w.len > p.window ? p.window + min(p.sinks, w.len - p.window) : w.len;
        const int all = (w.n_sel + kAttnTile - 1) / kAttnTile;
        const int per = quotient(all + p.splits - 1, p.by_splits);
        w.tile = min(all, w.split * per);
        w.tiles = min(all, w.tile + per);
        return w;
    }
    w.n_sel = max(0, min(p.num_sel, entries));
    // (the shuffle tells the compiler that the count, and the loops over it, are uniform)
    if (!kOneLane)
        w.n_sel = __shfl_sync(0xFFFFFFFFu, w.n_sel, 0);
    const int all = ((w.n_sel << p.block_shift) + kAttnTile - 1) / kAttnTile;
    w.tile = w.split * p.split_tiles;
    w.tiles = max(w.tile, min(all, w.tile + p.split_tiles));
    return w;
}

// 16 values of every lane, combined over the warp: lane i ends with value i / 2.
template <bool kMax>
__device__ __forceinline__ float reduce16_of(float v0, float v1, float v2, float v3, float v4,
                                          float v5, float v6, float v7, float v8, float v9,
                                          float v10, float v11, float v12, float v13, float v14,
                                          float v15)
{
    const float v[16] = {v0, v1, v2, v3, v4, v5, v6, v7, v8, v9, v10, v11, v12, v13, v14, v15};
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

template <bool kMax>
__device__ __forceinline__ float reduce16(const float* v)
{
    return reduce16_of<kMax>(v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7], v[8], v[9], v[10],
                             v[11], v[12], v[13], v[14], v[15]);
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

// Pairs of fp32 values on the packed FMA pipe: a = a * s + c, a = a * s, a += b, a += b * s.
__device__ __forceinline__ uint64_t pair(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t r, float& a, float& b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ void fma2(float& a0, float& a1, float s0, float s1, float c0, float c1)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(r)
        : "l"(pair(a0, a1)), "l"(pair(s0, s1)), "l"(pair(c0, c1)));
    unpair(r, a0, a1);
}
__device__ __forceinline__ void mul2(float& a0, float& a1, float s0, float s1)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair(a0, a1)), "l"(pair(s0, s1)));
    unpair(r, a0, a1);
}
__device__ __forceinline__ void add2(float& a0, float& a1, float b0, float b1)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair(a0, a1)), "l"(pair(b0, b1)));
    unpair(r, a0, a1);
}
__device__ __forceinline__ void add2_scaled(float& a0, float& a1, float b0, float b1, float s)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(r)
        : "l"(pair(b0, b1)), "l"(pair(s, s)), "l"(pair(a0, a1)));
    unpair(r, a0, a1);
}

// The largest of a warp's values (a NaN gives way): for 32 heads less work than their maxima by
// shuffles (64 heads over 2,048 x 2,048 fp16 keys 242 us against 246, 32 over bf16 keys with scores of
// deviation 16 199 against 207), for 16 as much.
__device__ __forceinline__ float warp_max(float v)
{
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// Two f16 values as e4m3 (low byte: the first); they become 16 times what is left of them.
__device__ __forceinline__ uint32_t e4m3_split(uint32_t& h)
{
    const uint16_t code = __nv_cvt_halfraw2_to_fp8x2(*reinterpret_cast<const __half2_raw*>(&h),
                                                     __NV_SATFINITE, __NV_E4M3);
    const __half2 back(__nv_cvt_fp8x2_to_halfraw2(code, __NV_E4M3));
    const __half2 rest = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&h), back),
                                 __float2half2_rn(16.0f));
    h = *reinterpret_cast<const uint32_t*>(&rest);
    return code;
}

// Eight e4m3 codes (low byte first) as bf16, which holds every one of them.
__device__ __forceinline__ uint4 bf16_of_e4m3x8(uint32_t lo, uint32_t hi)
{
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h(__nv_cvt_fp8x2_to_halfraw2(
            static_cast<__nv_fp8x2_storage_t>((i < 2 ? lo : hi) >> (16 * (i & 1))), __NV_E4M3));
        const float2 f = __half22float2(h);
        r[i] = pack2<__nv_bfloat16>(f.x, f.y);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

template <int D, int NH, int MODE, bool kRange>
__global__ void __launch_bounds__(AttnCfg<D, NH, MODE>::kThreads, 1)
attention_tc_kernel(const __grid_constant__ AttnParams p)
{
    using C = AttnCfg<D, NH, MODE>;
    using T = typename std::conditional<MODE == kModeBf16 || MODE == kModeFp8Bf16, __nv_bfloat16,
                                        __half>::type;
    constexpr int HN = C::kHeads;
    extern __shared__ __align__(1024) uint8_t sm[];
    uint8_t* stages = sm;                                      // k and v of kTiles tiles
    uint8_t* pbuf = stages + C::kTiles * C::kTileBytes;        // [2] weights
    uint8_t* qbuf = pbuf + 2 * C::kPBytes;                     // [2] queries
    // [2 warpgroups][4 quadrants][HN] sums of an item, [2][HN] running maxima
    float* sums = reinterpret_cast<float*>(qbuf + 2 * C::kQBytes);
    float* maxima = sums + C::kStats / 4;
    float* qscale = maxima + C::kMax / 4;                      // [kScaleItems][NH], [NH] of scratch
    float* kscale = qscale + C::kQScale / 4;                   // [2 kTiles][128]
    float* vscale = kscale + (C::kFp8 ? C::kStages * kAttnTile : 0);
    uint8_t* valid = reinterpret_cast<uint8_t*>(vscale + (C::kFp8 ? C::kStages * kAttnTile : 0));
    uint64_t* kv_full = reinterpret_cast<uint64_t*>(valid + C::kStages * kAttnTile);
    uint64_t* kv_empty = kv_full + C::kStages;
    uint64_t* q_full = kv_empty + C::kStages;
    uint64_t* q_empty = q_full + 2;
    uint64_t* s_full = q_empty + 2;
    uint64_t* s_empty = s_full + 2;
    uint64_t* p_full = s_empty + 2;
    uint64_t* p_empty = p_full + 2;
    uint64_t* o_full = p_empty + 2;
    uint64_t* o_empty = o_full + 2;
    uint64_t* f_full = o_empty + 2;                            // sums and maxima
    uint64_t* f_empty = f_full + 1;
    uint64_t* drained = f_empty + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 2);
    volatile int* ab = reinterpret_cast<volatile int*>(tmem_slot + 1);   // a wait gave up

    const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x / 32), 0);
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(kv_full + i, C::kFp8 ? 2 : 1);
            mbar_init(kv_empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full + i, 4);
            mbar_init(q_empty + i, 1);
            mbar_init(s_full + i, 1);
            mbar_init(s_empty + i, C::kTileWarps);
            mbar_init(p_full + i, C::kTileWarps);
            mbar_init(p_empty + i, 1);
            mbar_init(o_full + i, 1);
            mbar_init(o_empty + i, 4);
        }
        mbar_init(f_full, 8);
        mbar_init(f_empty, 4);
        mbar_init(drained, 1);
        mbar_init(drained + 1, 1);
        // the swizzled tiles need their 1024-byte boundaries
        *ab = (smem_u32(sm) & 1023u) != 0;
        fence_mbar_init();
    }
    if (warp == C::kMmaWarp) {
        tmem_alloc(tmem_slot, C::kTmem);
        tmem_relinquish();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_s = *tmem_slot, tmem_o = tmem_s + 2 * C::kSCols;
    pdl_wait_then_release();
    // The status word is cleared by the call itself; a wait that gives up sets it a whole
    // wait budget later.
    if (blockIdx.x == 0 && threadIdx.x == 0)
        *p.status = *ab ? kStatusBadArg : 0u;

    const int total = p.rows * p.Hkv * p.head_tiles * p.splits;
    // A short loop in place: the roles' loops together have to stay in the instruction cache, and
    // a call would keep the compiler from giving the roles different register counts.
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (mbar_try_wait(bar, parity))
            return true;
#pragma unroll 1
        for (int i = 0; i < kWaitTries && *ab == 0; ++i)
            if (mbar_try_wait_sleep(bar, parity, 1000u))
                return true;
        *ab = kGaveUp;
        return false;
    };
    // Tiles, numbered over the block's items, use the score and weight buffers alternately.

    if (warp < 8) {
        // ---------------------------------------------------------------- softmax
        if (C::kTrade)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftmaxRegs));
        // Thread = one key of a tile (a TMEM lane) x HN heads.
        const int wg = warp / 4, quad = warp & 3, key = 32 * quad + lane, bar_id = 1 + wg;
        const uint32_t lanes = static_cast<uint32_t>(32 * quad) << 16;
        const int head0 = C::kAlternate ? 0 : HN * wg;
        float* mx = maxima + wg * HN;
        // Weights are kept relative to a running maximum that is replaced only where a score
        // passes it by kSlack: most tiles need no exchange over the keys and no rescaling of
        // the accumulated output.  bf16 weights and fp32 sums have room, so there an item goes by 0
        // instead of its maxima until a score leaves +-32 (an exchange for each item's first tile
        // cost a tenth of its time): weights of 2^32 at most over values below 2^80 leave a list of
        // 65,536 keys finite, and values above 2^-84 keep their bits.  (+-64 left them 2^-52 to
        // 2^48 and took as long where scores have a deviation of 4, 177 us, 188 for 199 at 16; +-16
        // took 188 and 230.)  fp16 weights have to stay
        // below 2^16 and end at 2^-24: they go by 2^-7 of the maximum, so that it has weight 2^7 to
        // 2^15 and the others their 11 bits down to 2^-21 of it, some to 2^-31 (by the maximum
        // itself a list's small weights were lost from 2^-25 of it on).
        constexpr bool kZeroStart = C::kWide;
        constexpr float kSlack = C::kWide ? 32.0f : 15.0f;
        constexpr float kBelow = C::kWide ? 0.0f : 7.0f;
        // the thread's heads in a row of the weights, and the row's part of them as scratch
        constexpr int kOwn = HN * 2;                     // bytes of a term
        auto scratch = [&](int b, int i) {               // float i of 4 HN
            constexpr int per = kOwn / 4;
            return reinterpret_cast<float*>(
                pbuf + b * C::kPBytes +
                swizzled<C::kPRow>(i / per * C::kPRow + head0 * 2 + i % per * 4));
        };
        // A reference this far below zero is taken anew from the next tile's scores as they are:
        // subtracted from a score near zero and added back it would round it away (to 2^-12 at
        // the limit, to nothing at a reference of -3e38).
        constexpr float kFar = -4096.0f;
        bool bad = false;
        int n = 0, iq = 0;                               // tiles and items before this item
        int entries = item_entries<kRange>(p, blockIdx.x, total);
        for (int item = blockIdx.x; item < total; item += gridDim.x) {
            const AttnItem w = attn_item<kRange>(p, item, entries);
            entries = item_entries<kRange>(p, item + gridDim.x, total);
            const int count = w.tiles - w.tile;
            if (count == 0)
                continue;
            float l[HN];
#pragma unroll
            for (int i = 0; i < HN; ++i)
                l[i] = 0.0f;
            // first: no key yet, so no maximum (and weights and sums of nothing but zeros); based: mx
            // holds the maxima; far: one of them is below kFar
            bool first = true, leave = false, based = !kZeroStart, far = false;
#pragma unroll 1
            for (int j = C::kAlternate ? (wg ^ n) & 1 : 0; j < count; j += C::kAlternate ? 2 : 1) {
                const int b = (n + j) & 1, u = (n + j) >> 1;
                bad |= !wait(s_full + b, u & 1);
                tc_fence_after();
                float x[HN];
#pragma unroll
                for (int c = 0; c < HN; c += 16)
                    tmem_ld_32x32b_x16(tmem_s + lanes + b * C::kSCols + head0 + c, x + c);
                if (C::kFp8) {
#pragma unroll
                    for (int k = 1; k < C::kQTerms; ++k) {
#pragma unroll
                        for (int c = 0; c < HN; c += 16) {
                            float r[16];
                            tmem_ld_32x32b_x16(
                                tmem_s + lanes + b * C::kSCols + k * NH + head0 + c, r);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; i += 2)
                                add2_scaled(x[c + i], x[c + i + 1], r[i], r[i + 1],
                                            k == 1 ? 0.0625f : 0.00390625f);
                        }
                    }
                }
                tmem_wait_ld();
                tc_fence_before();
                if (C::kFp8) {
                    const float* qs = qscale + iq % kScaleItems * NH + head0;
#pragma unroll
                    for (int i = 0; i < HN; i += 4) {
                        const float4 f = *reinterpret_cast<const float4*>(qs + i);
                        mul2(x[i], x[i + 1], f.x, f.y);
                        mul2(x[i + 2], x[i + 3], f.z, f.w);
                    }
                }
                const int ring = (n + j) % C::kStages * kAttnTile + key;
                const bool ok = valid[ring] != 0;
                // a tile without a key leaves everything as it is
                const bool some =
                    !first ||
                    __any_sync(0xFFFFFFFFu,
                               reinterpret_cast<const uint32_t*>(valid + (ring - key))[lane] != 0u);
                float ks = p.scale_log2, vs = 1.0f;
                if (C::kFp8) {
                    ks = ok ? kscale[ring] : 0.0f;
                    vs = vscale[ring];
                }
                const bool all = __all_sync(0xFFFFFFFFu, ok);
                if (lane == 0)
                    mbar_arrive(s_empty + b);
                // Exponents, relative to the running maximum where there is one.
                float over = -INFINITY;
                const bool raw = first || !based || far;
                if (raw) {
#pragma unroll
                    for (int i = 0; i < HN; i += 2) {
                        mul2(x[i], x[i + 1], ks, ks);
                        if (kZeroStart)
                            over = fmaxf(over, fmaxf(fabsf(x[i]), fabsf(x[i + 1])));
                    }
                    over = ok ? over : -INFINITY;
                } else {
#pragma unroll
                    for (int i = 0; i < HN; i += 4) {
                        const float4 m = *reinterpret_cast<const float4*>(mx + i);
                        fma2(x[i], x[i + 1], ks, ks, -m.x, -m.y);
                        fma2(x[i + 2], x[i + 3], ks, ks, -m.z, -m.w);
                        over = fmaxf(over, fmaxf(fmaxf(x[i], x[i + 1]), fmaxf(x[i + 2], x[i + 3])));
                    }
                    over = ok ? over : -INFINITY;
                }
                if (!all) {
#pragma unroll
                    for (int i = 0; i < HN; ++i)
                        x[i] = ok ? x[i] : -INFINITY;
                }
                bool waited = false;
                if ((raw && based && some) || bar_any(over > kSlack || bad, bar_id, 128)) {
                    waited = true;
                    // (maxima of the item before have been read)
                    if (first || !based)
                        bad |= !wait(f_empty, (iq & 1) ^ 1);
                    // the products so far are complete, the buffer is free
                    bad |= !wait(p_empty + b, (u & 1) ^ 1);
                    if (!C::kAlternate && !first)
                        bad |= !wait(p_empty + (b ^ 1), ((n + j - 1) >> 1) & 1);
                    if (!raw) {
#pragma unroll
                        for (int i = 0; i < HN; i += 4) {
                            const float4 m = *reinterpret_cast<const float4*>(mx + i);
                            add2(x[i], x[i + 1], m.x, m.y);
                            add2(x[i + 2], x[i + 3], m.z, m.w);
                        }
                    }
                    if (HN == 32) {
#pragma unroll
                        for (int c = 0; c < HN; c += 4) {
                            float4 r;
                            r.x = warp_max(x[c]);
                            r.y = warp_max(x[c + 1]);
                            r.z = warp_max(x[c + 2]);
                            r.w = warp_max(x[c + 3]);
                            if (lane == 0)
                                *reinterpret_cast<float4*>(scratch(b, quad * HN + c)) = r;
                        }
                    } else {
                        const float r = reduce16<true>(x);
                        if ((lane & 1) == 0)
                            *scratch(b, quad * HN + lane / 2) = r;
                    }
                    if (!bar_all(!bad, bar_id, 128)) {
                        leave = true;
                        break;
                    }
                    float mn = 0.0f;
                    if (key < HN) {
                        const float old = first ? -3.0e38f : based ? mx[key] : 0.0f;
                        mn = fmaxf(
                            old, fmaxf(fmaxf(*scratch(b, key), *scratch(b, HN + key)),
                                       fmaxf(*scratch(b, 2 * HN + key), *scratch(b, 3 * HN + key))) -
                                     kBelow);
                        *scratch(b, key) = ex2(old - mn);
                        mx[key] = mn;
                    }
                    far = bar_any(mn < kFar, bar_id, 128);
#pragma unroll
                    for (int i = 0; i < HN; i += 4) {
                        const float4 m = *reinterpret_cast<const float4*>(mx + i);
                        add2(x[i], x[i + 1], -m.x, -m.y);
                        add2(x[i + 2], x[i + 3], -m.z, -m.w);
                    }
                    if (!first) {
                        tc_fence_after();
#pragma unroll
                        for (int i = 0; i < HN; i += 4) {
                            const float4 f = *reinterpret_cast<const float4*>(scratch(b, i));
                            mul2(l[i], l[i + 1], f.x, f.y);
                            mul2(l[i + 2], l[i + 3], f.z, f.w);
                        }
#pragma unroll 1
                        for (int c = 0; c < HN; c += 8) {
                            const float4 f0 = *reinterpret_cast<const float4*>(scratch(b, c));
                            const float4 f1 = *reinterpret_cast<const float4*>(scratch(b, c + 4));
                            const uint32_t at =
                                tmem_o + lanes +
                                ((iq & 1) * C::kAccs + (C::kAlternate ? b : 0)) * C::kOCols + head0 +
                                c;
                            float v[8];
                            tmem_ld_32x32b_x8(at, v);
                            tmem_wait_ld();
                            v[0] *= f0.x;
                            v[1] *= f0.y;
                            v[2] *= f0.z;
                            v[3] *= f0.w;
                            v[4] *= f1.x;
                            v[5] *= f1.y;
                            v[6] *= f1.z;
                            v[7] *= f1.w;
                            tmem_st_32x32b_x8(at, v);
                        }
                        tmem_wait_st();
                        tc_fence_before();
                        bar_all(true, bar_id, 128);      // the factors have been read
                    }
                    based = true;
                }
                first = !some;
#pragma unroll
                for (int i = 0; i < HN; ++i)
                    x[i] = ex2(x[i]);
#pragma unroll
                for (int i = 0; i < HN; i += 2)
                    add2(l[i], l[i + 1], x[i], x[i + 1]);
                if (C::kFp8) {
#pragma unroll
                    for (int i = 0; i < HN; i += 2)
                        mul2(x[i], x[i + 1], vs, vs);
                }
                if (!waited)
                    bad |= !wait(p_empty + b, (u & 1) ^ 1);
                using W = typename std::conditional<C::kWide, __nv_bfloat16, __half>::type;
                uint8_t* prow = pbuf + b * C::kPBytes;
#pragma unroll
                for (int k = 0; k < C::kPTerms; ++k) {
#pragma unroll
                    for (int c = 0; c < HN; c += 8) {
                        uint32_t h[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float &lo = x[c + 2 * i], &hi = x[c + 2 * i + 1];
                            h[i] = pack2<W>(lo, hi);
                            if (k + 1 < C::kPTerms)          // what is left of them
                                add2(lo, hi, -__uint_as_float(h[i] << 16),
                                     -__uint_as_float(h[i] & 0xFFFF0000u));
                        }
                        *reinterpret_cast<uint4*>(
                            prow + k * C::kPTile +
                            swizzled<C::kPRow>(key * C::kPRow + 2 * (head0 + c))) =
                            make_uint4(h[0], h[1], h[2], h[3]);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(p_full + b);
            }
            if (leave)
                break;
            if (first || !based) {                       // no key of this item, or no maxima
                bad |= !wait(f_empty, (iq & 1) ^ 1);
                if (key < HN)
                    mx[key] = first ? -3.0e38f : 0.0f;
            }
#pragma unroll
            for (int c = 0; c < HN; c += 16) {
                const float r = reduce16<false>(l + c);
                if ((lane & 1) == 0)
                    sums[(wg * 4 + quad) * HN + c + lane / 2] = r;
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(f_full);
            n += count;
            ++iq;
        }
        __syncwarp();
        if (C::kTrade)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kLaunchRegs));
    } else if (warp < C::kGatherWarp) {
        // --------------------------------------------------------------- epilogue
        // Thread = one element (of D) of NH heads.
        const int quad = warp & 3, dim = 32 * quad + lane;
        const uint32_t lanes = static_cast<uint32_t>(32 * quad) << 16;
        const bool parts = p.splits > 1, write = D == 128 || dim < D;
        // The queries of an item, one item ahead: they are converted (e4m3 caches) or copied into
        // the operand's layout by these warps, which have little else to do.
        int q_item = blockIdx.x, nq = 0;                 // next item to load, items loaded
        int q_entries = item_entries<kRange>(p, blockIdx.x, total);
        auto load_queries = [&] {
            AttnItem w;
            for (;; q_item += gridDim.x) {
                if (q_item >= total)
                    return true;
                w = attn_item<kRange>(p, q_item, q_entries);
                q_entries = item_entries<kRange>(p, q_item + gridDim.x, total);
                if (w.tiles > w.tile)
                    break;
            }
            q_item += gridDim.x;
            // (agreed on by the four warps: they meet below)
            if (!bar_all(wait(q_empty + (nq & 1), ((nq >> 1) & 1) ^ 1), 3, 128))
                return false;
            const uint8_t* q =
                p.q + w.t * p.q_row + (int64_t)(w.g * p.group + w.ht * NH) * p.q_head;
            const int heads = min(NH, p.group - w.ht * NH);
            uint8_t* dst = qbuf + (nq & 1) * C::kQBytes;
            const int from = threadIdx.x - 32 * 8;       // of the 128 threads
            if (!C::kFp8) {
                constexpr int kPerRow = C::kRow / 16;
#pragma unroll 1
                for (int i = from; i < C::kQBytes / 16; i += 128) {
                    const int h = i / kPerRow, c = i % kPerRow;
                    const uint32_t off = (c / 8) * (NH * 128) + h * 128 + (c % 8) * 16;
                    cp_async16(smem_u32(dst) + swizzled<128>(off),
                               h < heads ? q + h * p.q_head + c * 16 : q, h < heads);
                }
                cp_async_commit();
                cp_async_wait<0>();
            } else {
                // The queries as sums of e4m3 terms, each 1/16 of the scale of the one before: two
                // hold the 8 bits of a bf16 element, three the 11 of an fp16 one, down to 2^-22 of
                // its head's largest.  One scale for all heads, which would leave nothing of a head
                // 2^-22 of its neighbour's size, spared the softmax a product (64 heads over 2,048 x
                // 2,048 keys: 280 us against 302); a flag for heads of one size took as long.
                constexpr int kGroup = D / 16;           // lanes of a vector, 16 elements each
                const int c = lane % kGroup;
                float* mul = qscale + kScaleItems * NH;  // of a head, by the lanes that read it
                {
                    // the heads' largest magnitudes, all of their elements asked for at once (a
                    // vector after another 6 % more: 4,096 rows of 64 heads, 512 keys each)
                    using T2 = typename std::conditional<MODE == kModeFp8Bf16, __nv_bfloat162,
                                                         __half2>::type;
                    constexpr int kIter = (NH * kGroup + 127) / 128;
                    uint4 in[kIter][2];
#pragma unroll
                    for (int k = 0; k < kIter; ++k) {
                        const int h = from / kGroup + k * (128 / kGroup);
                        in[k][0] = in[k][1] = make_uint4(0u, 0u, 0u, 0u);
                        if (h < heads) {
                            const uint4* at =
                                reinterpret_cast<const uint4*>(q + h * p.q_head) + 2 * c;
                            in[k][0] = at[0];
                            in[k][1] = at[1];
                        }
                    }
#pragma unroll
                    for (int k = 0; k < kIter; ++k) {
                        const int h = from / kGroup + k * (128 / kGroup);
                        const T2* two = reinterpret_cast<const T2*>(in[k]);
                        T2 m = __habs2(two[0]);
#pragma unroll
                        for (int i = 1; i < 8; ++i)
                            m = __hmax2(m, __habs2(two[i]));
                        float amax = fmaxf(value(m.x), value(m.y));
#pragma unroll
                        for (int d = kGroup / 2; d > 0; d >>= 1)
                            amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d));
                        // a power of two that takes amax to 128..256, so that no element is
                        // rounded (any of an infinite one, whose head is NaN whatever it is)
                        const int ex = static_cast<int>(__float_as_uint(amax) >> 23);
                        const int up = amax > 0.0f ? min(max(261 - ex, 1), 254) : 127;
                        const float f = __uint_as_float(static_cast<uint32_t>(up) << 23);
                        if (c == 0 && h < NH) {
                            mul[h] = f;
                            qscale[nq % kScaleItems * NH + h] = p.scale_log2 / f;
                        }
                    }
                    __syncwarp();
                }
                // (heads that are none are zeros: the tile's scores are those of all its heads)
#pragma unroll 1
                for (int h = from / kGroup; h < NH; h += 128 / kGroup) {
                    uint4 in[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
                    if (h < heads) {
                        const uint4* at = reinterpret_cast<const uint4*>(q + h * p.q_head) + 2 * c;
                        in[0] = at[0];
                        in[1] = at[1];
                    }
                    const T* e = reinterpret_cast<const T*>(in);
                    const float f = mul[h];
                    uint32_t v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        // (+ 0 x: an infinite element makes its head NaN)
                        float a = value(e[2 * i]), b = value(e[2 * i + 1]), a0 = a, b0 = b;
                        mul2(a, b, f, f);
                        fma2(a0, b0, 0.0f, 0.0f, a, b);
                        v[i] = pack2<__half>(a0, b0);
                    }
#pragma unroll
                    for (int k = 0; k < C::kQTerms; ++k) {
                        uint32_t o[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t lo = e4m3_split(v[2 * i]);
                            o[i] = lo | e4m3_split(v[2 * i + 1]) << 16;
                        }
                        *reinterpret_cast<uint4*>(
                            dst + swizzled<C::kAtom>((k * NH + h) * C::kRow + c * 16)) =
                            make_uint4(o[0], o[1], o[2], o[3]);
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(q_full + (nq & 1));
            ++nq;
            return true;
        };
        int n = 0, iq = 0;                               // tiles and items before this item
        int entries = item_entries<kRange>(p, blockIdx.x, total);
        for (int item = blockIdx.x; item < total; item += gridDim.x) {
            const AttnItem w = attn_item<kRange>(p, item, entries);
            entries = item_entries<kRange>(p, item + gridDim.x, total);
            const int tiles = w.tiles - w.tile, head0 = w.ht * NH;
            // The next item's queries (and before the first item its own).  Not for items without
            // tiles: the place waited for is that of the item before this one, which has left
            // it by now; a later one's would wait for this very warp.
            bool loaded = true;
#pragma unroll 1
            for (int k = tiles == 0 ? 0 : iq == 0 ? 2 : 1; k > 0; --k)
                loaded = loaded && load_queries();
            if (!loaded)
                break;
            const int heads = parts ? NH : min(NH, p.group - head0);
            uint8_t* out =
                p.out + w.t * p.out_row + (int64_t)(w.g * p.group + head0) * p.out_head + 2 * dim;
            // (A cluster's parts stay in shared memory, for a block's one item: the sums and maxima
            // where softmax, which is done with the keys by then, read what it had to know of
            // them; the output in the stages once the last product is complete.)
            float* part = (p.cluster ? reinterpret_cast<float*>(stages)
                                     : p.part_o + (int64_t)item * NH * D) + dim;
            float2* part_ml = p.cluster ? reinterpret_cast<float2*>(valid)
                                        : reinterpret_cast<float2*>(p.part_ml) + (int64_t)item * NH;
            // Factors of the accumulators, for head `lane` (+ 32): the weight of its maximum,
            // over the sum.
            float fa[(NH + 31) / 32], fb = 0.0f;
            bool ok = tiles == 0 || wait(f_full, iq & 1);
#pragma unroll
            for (int k = 0; k < (NH + 31) / 32; ++k) {
                const int h = lane + 32 * k, i = C::kAlternate ? h % HN : lane;
                float m = -3.0e38f, l = 0.0f;
                fa[k] = 1.0f;
                if (tiles > 0) {
                    const float* s = sums + (C::kAlternate ? 0 : k) * 4 * HN + i;
                    m = maxima[(C::kAlternate ? 0 : k) * HN + i];
                    l = (s[0] + s[HN]) + (s[2 * HN] + s[3 * HN]);
                    if (C::kAlternate) {
                        const float m2 = maxima[HN + i];
                        const float l2 = (s[4 * HN] + s[5 * HN]) + (s[6 * HN] + s[7 * HN]);
                        const float mn = fmaxf(m, m2);
                        fa[k] = ex2(m - mn);
                        fb = ex2(m2 - mn);
                        m = mn;
                        l = l * fa[k] + l2 * fb;
                    }
                }
                if (quad == 0 && h < heads) {
                    if (parts)
                        part_ml[h] = make_float2(m, l);
                    else if (p.lse)
                        p.lse[(int64_t)w.t * p.Hq + w.g * p.group + head0 + h] =
                            (m + __log2f(l)) * 0.693147180559945309f;
                }
                const float inv = parts ? 1.0f : l == 0.0f ? 0.0f : __fdividef(1.0f, l);
                fa[k] *= inv;
                fb *= inv;
            }
            if (tiles > 0) {
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(f_empty);
                ok = ok && wait(o_full + (iq & 1), (iq >> 1) & 1);
                if (!__all_sync(0xFFFFFFFFu, ok))
                    break;
                tc_fence_after();
            }
            // 16 heads at a time, 8 of small groups (8 heads of 64: 8 % less; 32 of 128 in
            // eights 7 % more)
            constexpr int kStep = NH == 16 ? 8 : 16;
            auto load = [](uint32_t at, float* v) {
                if (kStep == 8)
                    tmem_ld_32x32b_x8(at, v);
                else
                    tmem_ld_32x32b_x16(at, v);
            };
#pragma unroll 1
            for (int h0 = 0; h0 < heads; h0 += kStep) {
                float o[kStep];
#pragma unroll
                for (int i = 0; i < kStep; ++i)
                    o[i] = 0.0f;
#pragma unroll 1
                for (int a = 0; a < C::kAccs && tiles > 0; ++a) {
                    if (tiles == 1 && C::kAlternate && a != (n & 1))
                        continue;                        // it was not written
                    const uint32_t at =
                        tmem_o + lanes + ((iq & 1) * C::kAccs + a) * C::kOCols + h0;
                    const float fac = a > 0 ? fb : NH > 32 && h0 >= 32 ? fa[NH / 64] : fa[0];
                    float v[kStep];
                    load(at, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < kStep; ++i) {
                        const float s = __shfl_sync(0xFFFFFFFFu, fac, (h0 + i) & 31);
                        o[i] = s != 0.0f ? fmaf(v[i], s, o[i]) : o[i];
                    }
                }
                if (!write)
                    continue;
                if (parts) {
                    float* to = part + h0 * D;
#pragma unroll
                    for (int i = 0; i < kStep; ++i)
                        to[i * D] = o[i];
                } else {
                    uint8_t* to = out + h0 * p.out_head;
#pragma unroll
                    for (int i = 0; i < kStep; ++i) {
                        if (h0 + i < heads)
                            *reinterpret_cast<T*>(to) = static_cast<T>(o[i]);
                        to += p.out_head;
                    }
                }
            }
            if (tiles > 0) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(o_empty + (iq & 1));
                n += tiles;
                ++iq;
            }
        }
    } else {
        if (C::kTrade)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kFeedRegs));
        if (warp < C::kMmaWarp) {
            // ---------------------------------------------------------------- gather
            // Two warps fill a place of the ring: one its keys and one its values, or (e4m3 caches,
            // whose values are converted by the warp that copied them) each both of 64 keys.  A
            // warp looks up its keys' slots, waits for the place, copies the vectors (zeros for
            // keys that are none), waits for its own copies and signals.  The other places'
            // warps keep the memory system busy meanwhile.  A warp sees every phase of the
            // barriers it waits on.  It reads the list entries of its next tile while its copies are
            // under way and the pages after them.  (2,048 rows x 2,048 e4m3 keys: 16, 32 and 64 heads
            // 188, 209 and 278 us; a warp for all of a tile's values 233, 265 and 313.  16-bit keys
            // both ways round: 160, 183 and 265 against 151, 184 and 234.)
            constexpr bool kBoth = C::kFp8;
            const int pw = warp - C::kGatherWarp, place = pw / 2;
            const bool is_v = !kBoth && (pw & 1);
            const int first_key = kBoth ? (pw & 1) * 64 : 0;
            constexpr int kOwnKeys = kBoth ? 2 : 4;          // of a lane
            constexpr int kPerRow = C::kRow / 16;            // copies of 16 bytes a vector takes
            constexpr int kSpan = kOwnKeys * kPerRow;        // keys of a group of kPerRow lanes
            const int chunk = lane % kPerRow, row0 = first_key + lane / kPerRow * kSpan;
            // a vector's 16 bytes in its row (of kAtom bytes, further ones in a next tile of rows)
            constexpr int kNext = kAttnTile * C::kAtom;
            const uint32_t place_at = smem_u32(stages + place * C::kTileBytes);
            const uint32_t copy_at =
                place_at + (is_v ? C::kKStage : 0) + row0 * C::kAtom + (chunk * 16 / C::kAtom) * kNext + (chunk * 16) % C::kAtom;
            // Values of e4m3 caches are copied to where the second half of their own bf16 row goes
            // (rows of 64: one half or the other), read back by the lane that copied them and
            // written as bf16 over the row.  Four lanes of every eight are a row of the pair ahead
            // or behind, which spreads the eight over the banks: they read and write 16 bytes of
            // even chunks in a row of an even and one of an odd swizzle.
            const int flip = C::kFp8 ? (lane >> 2) & 1 : 0;
            const uint32_t v_row =
                (place_at + C::kKStage + row0 * 128) ^ swizzle_of<128>(flip * 128);
            const uint32_t v_codes = (v_row + (D == 128 ? kAttnTile * 128 : 0)) ^
                                     ((D == 128 ? 0 : flip * 64) + chunk * 16);
            const uint32_t v_values = (v_row + chunk / 4 * (kAttnTile * 128)) ^ chunk % 4 * 32;
            AttnItem w;
            w.tile = w.tiles = w.n_sel = w.t = w.g = 0;
            int item = blockIdx.x - gridDim.x, skip = place;    // tiles to the warp's next one
            int entries = item_entries<kRange>(p, blockIdx.x, total);
            int r = 0, base = 0, most = 0, len = 0, g = 0;
            // the lane's keys of a tile: row0 + kPerRow i + chunk
            int32_t entry[kOwnKeys], key[kOwnKeys], page[kOwnKeys];
            auto advance = [&] {                             // to the warp's next tile; its entries
                w.tile += skip;
                bool fresh = false;
                while (w.tile >= w.tiles) {
                    skip = w.tile - w.tiles;
                    item += gridDim.x;
                    if (item >= total)
                        return false;
                    w = attn_item<kRange>(p, item, entries);
                    entries = item_entries<kRange>(p, item + gridDim.x, total);
                    w.tile += skip;
                    fresh = true;
                }
                skip = C::kTiles;
                if (fresh) {
                    r = request_of(p.row_begin, p.num_requests, w.t);
                    base = p.key_begin[r];
                    most = p.key_begin[r + 1] - base;
                    len = kRange ? w.len : p.clen[w.t];      // (used after the copies' wait)
                }
                const int32_t* sel = p.sel + w.t * p.ld_sel;
                // (keys past the first ones under a window are these many further on)
                const int past = kRange ? w.len - w.n_sel : 0;
                const int firsts = kRange ? p.sinks : 0;
#pragma unroll
                for (int i = 0; i < kOwnKeys; ++i) {
                    const int e =
                        (w.tile * kAttnTile + row0 + kPerRow * i + chunk) >> p.block_shift;
                    if constexpr (kRange)
                        entry[i] = e >= w.n_sel ? -1 : e < firsts ? e : e + past;
                    else
                        entry[i] = e < w.n_sel ? sel[e] : -1;
                }
                return true;
            };
            auto locate = [&] {                              // keys and pages of the entries
                const int32_t* table = p.table + r * p.ld_table;
#pragma unroll
                for (int i = 0; i < kOwnKeys; ++i) {
                    const int pos = w.tile * kAttnTile + row0 + kPerRow * i + chunk;
                    const int64_t k = ((int64_t)entry[i] << p.block_shift) +
                                      (pos & ((1 << p.block_shift) - 1));
                    const bool in = entry[i] >= 0 && k < min(len, most);
                    key[i] = static_cast<int32_t>(k);
                    page[i] = in ? 0 : -1;
                    if (p.page == 0) {
                        key[i] += base;
                    } else if (in) {
                        const int pg = quotient(key[i], p.by_page);
                        page[i] = table[pg];
                        key[i] -= pg * p.page;
                    }
                }
                g = w.g;
            };
            // (one copy of each step, for the instruction cache: the first round only looks up)
            for (int u = -1;; ++u) {
                if (u >= 0) {
                    int32_t slot[kOwnKeys];
                    bool whole = true;
#pragma unroll
                    for (int i = 0; i < kOwnKeys; ++i) {
                        const int64_t at = (int64_t)page[i] * p.page + key[i];
                        slot[i] = page[i] >= 0 && at < p.num_slots ? static_cast<int32_t>(at) : -1;
                        whole = whole && slot[i] >= 0;
                    }
                    whole = __all_sync(0xFFFFFFFFu, whole);
                    if (!__all_sync(0xFFFFFFFFu, wait(kv_empty + 2 * place + is_v, (u & 1) ^ 1)))
                        break;
                    if (!is_v) {
                        // What the softmax has to know of the keys.  No barrier guards the place, last
                        // read for the tile n - 2 kTiles: the scores of tile n - kTiles have freed the
                        // stage, and were issued after those of tile n - kTiles - 2 were read.
                        const int ring = (u * C::kTiles + place) % C::kStages * kAttnTile;
#pragma unroll
                        for (int i = 0; i < kOwnKeys; ++i) {
                            const int k = ring + row0 + kPerRow * i + chunk;
                            valid[k] = slot[i] >= 0;
                            if (C::kFp8) {
                                const int64_t at = (int64_t)max(slot[i], 0) * p.Hkv + g;
                                cp_async4(smem_u32(kscale + k), p.k_scale + at, slot[i] >= 0);
                                cp_async4(smem_u32(vscale + k), p.v_scale + at, slot[i] >= 0);
                            }
                        }
                    }
                    // A span's keys are spread over its lanes: slot i of lane k is key
                    // kPerRow i + k.  (eight rows at a time, for the instruction cache)
                    auto copy = [&](const uint8_t* src, uint32_t stride, uint32_t to, int turn,
                                    auto width) {
                        constexpr int kW = decltype(width)::value;
                        const int from = (lane & ~(kPerRow - 1)) ^ turn;
                        auto pick = [&](int i) {
                            const int32_t lo = i & 1 ? slot[1] : slot[0];
                            const int32_t hi = i & 1 ? slot[kOwnKeys - 1] : slot[kOwnKeys - 2];
                            return kOwnKeys > 2 && (i & 2) ? hi : lo;
                        };
                        if (whole) {
#pragma unroll 1
                            for (int row = 0; row < kSpan; row += 8) {
                                const int32_t a = pick(row / kPerRow);
                                const int32_t b = kPerRow < 8 ? pick(row / kPerRow + 1) : a;
                                const uint32_t dst = to + row * kW;
                                const int lane0 = from ^ row % kPerRow;
#pragma unroll
                                for (int x = 0; x < 8; ++x) {
                                    const uint32_t s = __shfl_sync(
                                        0xFFFFFFFFu, x < kPerRow ? a : b, lane0 ^ x % kPerRow);
                                    cp_async16(dst ^ swizzle_of<kW>(x * kW),
                                               src + (uint64_t)s * stride);
                                }
                            }
                        } else {
#pragma unroll 1
                            for (int row = 0; row < kSpan; ++row) {
                                const int32_t s = __shfl_sync(0xFFFFFFFFu, pick(row / kPerRow),
                                                              from ^ row % kPerRow);
                                cp_async16((to + row / 8 * 8 * kW) ^ swizzle_of<kW>(row % 8 * kW),
                                           src + (uint64_t)(uint32_t)max(s, 0) * stride, s >= 0);
                            }
                        }
                        cp_async_commit();
                    };
                    copy((is_v ? p.v : p.k) + chunk * 16 + g * (is_v ? p.v_head : p.k_head),
                         static_cast<uint32_t>(is_v ? p.v_slot : p.k_slot), copy_at, 0,
                         std::integral_constant<int, C::kAtom>());
                    if (kBoth) {
                        if (!__all_sync(0xFFFFFFFFu, wait(kv_empty + 2 * place + 1, (u & 1) ^ 1)))
                            break;
                        copy(p.v + chunk * 16 + g * p.v_head, static_cast<uint32_t>(p.v_slot),
                             v_codes, flip, std::integral_constant<int, 128>());
                    }
                }
                const bool more = advance();
                if (u >= 0) {
                    if (kBoth) {
                        cp_async_wait<1>();
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(kv_full + 2 * place);
                    }
                    cp_async_wait<0>();
                    if (C::kFp8) {
#pragma unroll 1
                        for (int row = 0; row < kSpan; row += 4) {
                            const uint32_t at = row / 8 * 1024;
                            const uint32_t four = swizzle_of<128>((row & 4) * 128);
                            uint4 codes[4];
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                codes[x] =
                                    lds128((v_codes + at) ^ four ^ swizzle_of<128>(x * 128));
                            __syncwarp();                    // (the rows have been read)
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                const uint32_t to =
                                    (v_values + at) ^ four ^ swizzle_of<128>(x * 128);
                                sts128(to, bf16_of_e4m3x8(codes[x].x, codes[x].y));
                                sts128(to ^ 16, bf16_of_e4m3x8(codes[x].z, codes[x].w));
                            }
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(kv_full + 2 * place + (kBoth || is_v));
                }
                if (!more)
                    break;
                locate();
            }
            cp_async_wait<0>();                              // (of a wait that gave up)
        } else {
            // --------------------------------------------------------------------- MMA
            // One elected lane of a warp for the scores, and of another for the products: each
            // waits and issues.  (One thread for both took 1,400 cycles a tile for its own instructions.)
            constexpr int kK = 32 / C::kEb;                 // contraction elements of a score MMA
            const bool scores = warp == C::kMmaWarp;
            if (elect_one()) {
                int n = 0, iq = 0, st = 0;                  // tile n's place in the ring
                uint32_t phase = 0;                         // and the uses of that place
                bool ok = true;
                int entries = item_entries<kRange>(p, blockIdx.x, total);
                for (int item = blockIdx.x; item < total && ok; item += gridDim.x) {
                    const AttnItem w = attn_item<kRange, true>(p, item, entries);
                    entries = item_entries<kRange>(p, item + gridDim.x, total);
                    const int count = w.tiles - w.tile;
                    if (count == 0)
                        continue;
                    if (scores) {                           // S = Q K
                        constexpr uint32_t idesc =
                            idesc_dense(128, C::kQRows, MODE == kModeBf16 ? 1 : 0, false, false);
                        const uint64_t q_desc =
                            smem_desc(smem_u32(qbuf + (iq & 1) * C::kQBytes), C::kAtom, 16,
                                          8 * C::kAtom);
                        ok = wait(q_full + (iq & 1), (iq >> 1) & 1);
                        for (int j = 0; j < count && ok; ++j, ++n) {
                            ok = wait(kv_full + 2 * st, phase) &&
                                 wait(s_empty + (n & 1), ((n >> 1) & 1) ^ 1);
                            if (!ok)
                                break;
                            tc_fence_after();
                            const uint64_t k_desc = smem_desc(smem_u32(stages + st * C::kTileBytes),
                                                              C::kAtom, 16, 8 * C::kAtom);
#pragma unroll
                            for (int k = 0; k < D / kK; ++k) {
                                const int atom = k * 32 / C::kAtom, in = (k * 32) % C::kAtom;
                                (C::kFp8 ? mma_f8f6f4 : mma_f16)(
                                    tmem_s + (n & 1) * C::kSCols,
                                    k_desc + (atom * (kAttnTile * C::kAtom) + in) / 16,
                                    q_desc + (atom * (C::kQRows * C::kAtom) + in) / 16, idesc, k > 0);
                            }
                            mma_commit(s_full + (n & 1));
                            mma_commit(kv_empty + 2 * st);
                            if (++st == C::kTiles) {
                                st = 0;
                                phase ^= 1;
                            }
                        }
                        if (ok)
                            mma_commit(q_empty + (iq & 1));
                    } else {                                // O += P V
                        constexpr uint32_t idesc =
                            idesc_dense(128, C::kOCols, C::kWide ? 1 : 0, true, true);
                        // v rows are keys: both operands are read along their rows.  D = 64 takes
                        // the same 64 elements for both halves of the 128 output rows.
                        constexpr uint32_t lbo = D == 64 ? 0 : kAttnTile * 128;
                        ok = wait(o_empty + (iq & 1), ((iq >> 1) & 1) ^ 1);
                        for (int j = 0; j < count && ok; ++j, ++n) {
                            const int b = n & 1;
                            ok = wait(kv_full + 2 * st + 1, phase) &&
                                 wait(p_full + b, (n >> 1) & 1);
                            if (!ok)
                                break;
                            tc_fence_after();
                            const uint64_t v_desc = smem_desc(
                                smem_u32(stages + st * C::kTileBytes + C::kKStage), 128, lbo, 1024);
                            const uint64_t p_desc =
                                smem_desc(smem_u32(pbuf + b * C::kPBytes), C::kPRow, 0,
                                          8 * C::kPRow);
                            const uint32_t d =
                                tmem_o + ((iq & 1) * C::kAccs + (C::kAlternate ? b : 0)) * C::kOCols;
                            // an empty accumulator
                            const bool fresh = C::kAlternate ? j < 2 : j == 0;
#pragma unroll
                            for (int k = 0; k < C::kPTerms * kAttnTile / 16; ++k)
                                mma_f16(d, v_desc + k % (kAttnTile / 16) * 128,
                                        p_desc + k * C::kPRow, idesc, !fresh || k > 0);
                            mma_commit(p_empty + b);
                            mma_commit(kv_empty + 2 * st + 1);
                            if (++st == C::kTiles) {
                                st = 0;
                                phase ^= 1;
                            }
                        }
                        if (ok)
                            mma_commit(o_full + (iq & 1));
                    }
                    ++iq;
                }
                // what was issued, and its arrivals, end before the memory goes
                uint64_t* mine = drained + (scores ? 0 : 1);
                mma_commit(mine);
                for (int i = 0; i < kWaitTries && !mbar_try_wait_sleep(mine, 0, 1000u); ++i)
                    ;
            }
        }
        __syncwarp();
        if (C::kTrade)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kLaunchRegs));
    }
    __syncthreads();
    if (threadIdx.x == 0 && *ab == kGaveUp)
        atomicOr(p.status, kStatusTimeout);
    if (p.cluster) {
        // The blocks of a row's splits are a cluster and have an item each: every block joins its
        // share of the heads from all blocks' parts.
        cluster_sync();
        const AttnItem w = attn_item<kRange>(p, blockIdx.x, p.num_sel);
        const int heads = min(NH, p.group - w.ht * NH), head0 = w.g * p.group + w.ht * NH;
        constexpr int kPer = D / 4;                      // threads of a head, four elements each
        const int d = threadIdx.x % kPer * 4;
        const uint32_t parts = smem_u32(stages), ml = smem_u32(valid);
        for (int h = w.split + threadIdx.x / kPer * p.splits; h < heads;
             h += C::kThreads / kPer * p.splits) {
            float2 stat[kMaxCluster];                    // maximum and sum
            float4 v[kMaxCluster];
#pragma unroll
            for (int r = 0; r < kMaxCluster; ++r) {
                stat[r] = make_float2(-3.0e38f, 0.0f);
                if (r < p.splits) {
                    stat[r] = ld_cluster2(cluster_address(ml + 8 * h, r));
                    v[r] = ld_cluster4(cluster_address(parts + (h * D + d) * 4, r));
                }
            }
            float m = stat[0].x, l = 0.0f;
#pragma unroll
            for (int r = 1; r < kMaxCluster; ++r)
                m = fmaxf(m, stat[r].x);
            float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int r = 0; r < kMaxCluster; ++r) {
                const float f = ex2(stat[r].x - m);
                l = fmaf(stat[r].y, f, l);
                if (r < p.splits && f != 0.0f) {
                    o.x = fmaf(v[r].x, f, o.x);
                    o.y = fmaf(v[r].y, f, o.y);
                    o.z = fmaf(v[r].z, f, o.z);
                    o.w = fmaf(v[r].w, f, o.w);
                }
            }
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            T* out = reinterpret_cast<T*>(p.out + w.t * p.out_row +
                                          (int64_t)(head0 + h) * p.out_head) + d;
            out[0] = static_cast<T>(o.x * inv);
            out[1] = static_cast<T>(o.y * inv);
            out[2] = static_cast<T>(o.z * inv);
            out[3] = static_cast<T>(o.w * inv);
            if (p.lse && d == 0)
                p.lse[(int64_t)w.t * p.Hq + head0 + h] =
                    (m + log2f(l)) * 0.693147180559945309f;
        }
        cluster_sync();                                  // no block leaves while it is read
    }
    if (warp == C::kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem_s, C::kTmem);
    }
}

// Rows split over more blocks than a cluster joins: the partial outputs of a row and head, weighted
// by their maxima.  One warp per (row, query head): the maxima and sums of all splits in one read,
// the parts four at a time (read one after another, 16 parts took 8 us).
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
    const int64_t first = ((t * p.Hkv + g) * p.head_tiles + hg / nh) * p.splits * nh + hg % nh;
    const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
    float2 v[kMaxSplits / 32];
    float m = -3.0e38f, l = 0.0f;
#pragma unroll
    for (int k = 0; k < kMaxSplits / 32; ++k) {
        const int s = lane + 32 * k;
        v[k] = s < p.splits ? ml[first + (int64_t)s * nh] : make_float2(-3.0e38f, 0.0f);
        m = fmaxf(m, v[k].x);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
#pragma unroll
    for (int k = 0; k < kMaxSplits / 32; ++k) {
        v[k].x = ex2(v[k].x - m);
        l = fmaf(v[k].y, v[k].x, l);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
    constexpr int N = D / 32;            // elements of a lane, neighbours
    const float* part = p.part_o + first * D + N * lane;
    float o[N] = {};
    for (int s0 = 0; s0 < p.splits; s0 += 4) {
        float in[4][N];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float* at = part + (int64_t)min(s0 + k, p.splits - 1) * nh * D;
            if (N == 4)
                *reinterpret_cast<float4*>(in[k]) = *reinterpret_cast<const float4*>(at);
            else
                *reinterpret_cast<float2*>(in[k]) = *reinterpret_cast<const float2*>(at);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float f = __shfl_sync(0xFFFFFFFFu, s0 < 32 ? v[0].x : v[kMaxSplits / 32 - 1].x,
                                        (s0 + k) & 31);
            if (s0 + k < p.splits && f != 0.0f)
#pragma unroll
                for (int e = 0; e < N; ++e)
                    o[e] = fmaf(in[k][e], f, o[e]);
        }
    }
    T* out = reinterpret_cast<T*>(p.out + t * p.out_row + h * p.out_head) + N * lane;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int e = 0; e < N; ++e)
        out[e] = static_cast<T>(o[e] * inv);
    if (p.lse && lane == 0)
        p.lse[i] = (m + log2f(l)) * 0.693147180559945309f;
}

template <int D, int NH, int MODE, bool kRange>
cudaError_t attention_tc(const AttnParams& p, cudaStream_t st)
{
    using C = AttnCfg<D, NH, MODE>;
    static std::atomic<uint64_t> ready;
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e == cudaSuccess)
        e = once_per_device(ready, device, [] {
            // the warpgroups' trade has to add up against what a block is launched with
            cudaFuncAttributes a;
            cudaError_t r = cudaFuncGetAttributes(&a, attention_tc_kernel<D, NH, MODE, kRange>);
            if (r == cudaSuccess && C::kTrade && a.numRegs != C::kLaunchRegs)
                r = cudaErrorLaunchOutOfResources;
            return r != cudaSuccess
                       ? r
                       : cudaFuncSetAttribute(attention_tc_kernel<D, NH, MODE, kRange>,
                                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                                              C::kSmem);
        });
    if (e != cudaSuccess)
        return e;
    const int items = p.rows * p.Hkv * p.head_tiles * p.splits;
    const unsigned blocks = p.cluster ? items : std::min(items, device_sms());
    return launch_pdl_cluster(attention_tc_kernel<D, NH, MODE, kRange>, dim3(blocks), dim3(C::kThreads),
                              C::kSmem, st, p.cluster ? p.splits : 1, p);
}

template <int D, int MODE, bool kRange>
cudaError_t attention_heads(const AttnParams& p, int nh, cudaStream_t st)
{
    cudaError_t e;
    if (nh == 16)
        e = attention_tc<D, 16, MODE, kRange>(p, st);
    else if (MODE == kModeFp8Fp16 || nh == 32)
        e = attention_tc<D, 32, MODE, kRange>(p, st);
    else if constexpr (MODE != kModeFp8Fp16)
        e = attention_tc<D, 64, MODE, kRange>(p, st);
    if (e != cudaSuccess || p.splits == 1 || p.cluster)
        return e;
    using T = typename std::conditional<MODE == kModeBf16 || MODE == kModeFp8Bf16, __nv_bfloat16,
                                        __half>::type;
    count_launch();
    const unsigned blocks = static_cast<unsigned>(((int64_t)p.rows * p.Hq + 3) / 4);
    return launch_pdl(attention_join_kernel<T, D>, dim3(blocks), dim3(128), 0, st, p, nh);
}

template <int MODE, bool kRange>
cudaError_t attention_mode(const AttnParams& p, int D, int nh, cudaStream_t st)
{
    return D == 64 ? attention_heads<64, MODE, kRange>(p, nh, st)
                   : attention_heads<128, MODE, kRange>(p, nh, st);
}

template <bool kRange>
cudaError_t attention_any(const AttnParams& p, int D, int dtype, bool fp8, cudaStream_t st)
{
    const int nh = attention_heads_per_tile(p.group, dtype, fp8);
    if (dtype == IDX_BF16)
        return fp8 ? attention_mode<kModeFp8Bf16, kRange>(p, D, nh, st)
                   : attention_mode<kModeBf16, kRange>(p, D, nh, st);
    return fp8 ? attention_mode<kModeFp8Fp16, kRange>(p, D, nh, st)
               : attention_mode<kModeFp16, kRange>(p, D, nh, st);
}

}  // namespace
}  // namespace idx
