// Causal attention of new tokens over the cached keys of their requests: all of them, or a sliding
// window and the first few.
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

// A work item is a key/value head and 256 rows of a request.  Rows are (token, query head of the
// group) pairs in that order, so that a group of any size fills the tensor cores' 128 rows and its heads
// read each key once.  Per tile of 128 keys and each of the item's two tiles of 128 rows
//     S [rows x keys] = Q K^T,   P = exp2(S scale log2(e) - reference),   O += P V
// with S, P and O in TMEM: a softmax thread owns a row, so its maximum and sum are its own, and P goes
// back over S as the product's first operand.  A tile's keys are two halves of 64, each with scores of
// its own: while one half is weighed, the product and the next scores of the other run.  The reference
// follows the row's maximum only when that has grown by kSlack, so that O is seldom rescaled.
//
// Which keys: row by row those of [len - window, len) and [0, sinks).  An item walks a list of
// consecutive places: the sinks, then from the first key that any of its rows sees to the last.  Every
// block gets an equal run of all items' key tiles, which may begin and end inside an item (256 items
// on 152 SMs: 824 us where whole ones took 880); cut items are joined by a kernel of their own.
//
// Roles: four warps load keys and values (converting e4m3), two load queries (one of them lists the
// items), two issue the products, two warpgroups do softmax and outputs.  All waits are bounded.
//
// Roundings: scores, maxima, sums and outputs are fp32.  Weights are rounded to the values' type, which
// the tensor cores take at twice tf32's rate and half its bytes: roundings of 2^-8 of a weight at most, of
// either sign, so that a bf16 output is off by 0.0024 of its size where fp32 weights leave 0.0017, the
// output's own rounding.
//
// Measured (GB300): 2,048 tokens behind 29,951, 4 x 8 heads of 128, bf16: 710 us (1.46 PFLOP/s, 78 % of the
// measured matrix rate); three prompts of 2,389 to 7,167 tokens, 8 x 4 heads of 64, fp16: 412 us (0.8
// PFLOP/s); 16,384 tokens under a window of 1,024, 8 x 8 heads of 128, e4m3: 632 us (0.87 PFLOP/s).  What
// bounds it: a half's chain in its softmax warp (wait, read, maximum, 64 exponentials, store: about 1,000
// cycles, of which the exponentials alone are 256), under which the MMAs run (60 % of the tensor pipe at
// heads of 128); an item's end and beginning, some 6,000 cycles.  Over e4m3 caches a tile of heads of 128
// takes 2.9 us with both row tiles and 2.4 with one (16-bit ones 2.3 and 1.8): not the scales that every
// softmax thread reads alone, which would halve; how much the loading warps' conversions cost is not
// measured.  Tried without gain: four softmax
// warpgroups of a half each (their registers leave room for reading the scores twice only: 515 us for
// the prompts where two took 465), the next half's scores read ahead (they are seldom there yet, 554),
// turns between the two warps of an SM's quarter (507).

constexpr int kModeBf16 = 0, kModeFp16 = 1, kModeFp8Bf16 = 2, kModeFp8Fp16 = 3;
constexpr int kWaitTries = 1 << 22;     // of about a microsecond at most
constexpr int kGaveUp = 2;
constexpr int kSmemLimit = 232448;
constexpr int kRows = kCausalRows;      // of an item
constexpr int kInfos = 4;               // items listed: the one that is weighed, and ahead
constexpr int kKeyRing = 8;             // tiles whose keys' validity and scales are kept

template <int D, int MODE>
struct Cfg {
    static constexpr bool kFp8 = MODE >= kModeFp8Bf16;
    // Operands: scores in the queries' type, whose 8 or 11 bits hold every e4m3 value; products over
    // e4m3 caches in bf16, because a weight times its value's scale needs an fp32 number's range, of
    // two terms under fp16 queries, whose outputs have 11 bits.
    static constexpr bool kHalfS = MODE == kModeFp16 || MODE == kModeFp8Fp16;
    static constexpr bool kHalfP = MODE == kModeFp16;
    static constexpr int kPTerms = MODE == kModeFp8Fp16 ? 2 : 1;
    static constexpr int kAtom = 128 * 128;             // 128 rows of 64 elements
    static constexpr int kStage = 128 * D * 2;          // keys or values of a tile
    static constexpr int kQ = 2 * kStage;
    static constexpr int kRaw = kFp8 ? 128 * D : 0;     // codes of a tile
    static constexpr int kRaws = kFp8 ? (D == 64 ? 6 : 3) : 0;
    static constexpr int kStages = kFp8 ? (D == 64 ? 4 : 3) : (D == 64 ? 8 : 5);
    // loads under way before one is waited for
    static constexpr int kLag = kFp8 ? kRaws - 1 : 2;
    static constexpr int kKeyInfo = kKeyRing * (32 + (kFp8 ? 2 * 128 * 4 : 0));
    static constexpr int kBars = 2 * kStages + 2 + 4 + 4 + 4 + 2 * kInfos + 2;
    static constexpr int kSmem = kQ + kStages * kStage + kRaws * kRaw + kKeyInfo + kInfos * 64 +
                                 8 * kBars + 16;
    static_assert(kSmem <= kSmemLimit, "tiles do not fit");
    static_assert(kFp8 || kLag <= kStages - 3, "a load is signalled before its place is waited for");
    static_assert(kKeyRing >= kStages / 2 + 2, "key ring");
    // Registers: what is traded was launched with, 512 threads of 128.  The softmax holds a half's scores
    // and weights, and two outputs' columns at an item's end; loading warps convert four e4m3 vectors at a
    // time.  (176, 64 and 96 the same over 16-bit caches, 676 us against 657 under a window of e4m3 keys;
    // 200, 56 and 56 838.)  fp16 over e4m3, whose weights have two terms, spills 100 bytes a thread at heads
    // of 128 and 52 at 64; the split was not tried for it.
    static constexpr int kThreads = 512, kLaunchRegs = 128;
    static constexpr int kSoftmaxRegs = 184, kFeedRegs = 56, kLoadRegs = 88;
    static_assert(2 * kSoftmaxRegs + kFeedRegs + kLoadRegs <= 4 * kLaunchRegs, "registers");
    static constexpr int kTmemO = 256;                  // columns: scores (and weights), then outputs
};

struct Item {
    int r, g, i0, rows;      // request, key/value head, first (token, head) row and how many
    int sinks, off, n;       // places of the list below sinks are keys; others are off keys on; places
    int tile, tiles;         // tiles [tile, tiles) of the list; tile < 0: no more items
    int part;                // where a part of an item goes, -1: the whole item
    int base, keys;          // the request's first packed key and its keys
    int inner, outer;        // places that every row sees: [inner, outer)
    int pad[2];
    // Whether a row may be blind to a key of the tile that others see.
    __device__ __forceinline__ bool edge(int t) const { return t * 128 < inner || t * 128 + 128 > outer; }
};
static_assert(sizeof(Item) == 64, "item");

__device__ __forceinline__ int quotient(int n, const Divisor& d)
{
    return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * d.mul) >> d.shift);
}

__device__ __forceinline__ constexpr uint32_t swizzled(uint32_t off)
{
    return off ^ (((off >> 7) & 7u) << 4);
}

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
__device__ __forceinline__ void fma2(float& a, float& b, uint64_t s, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pair(a, b)), "l"(s), "l"(c));
    unpair(r, a, b);
}
__device__ __forceinline__ void mul2(float& a, float& b, uint64_t s)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair(a, b)), "l"(s));
    unpair(r, a, b);
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

template <bool kHalf>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    uint32_t r;
    if (kHalf)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two e4m3 codes (low half) as two fp16 or bf16 numbers, exactly.
template <bool kHalf>
__device__ __forceinline__ uint32_t of_e4m3x2(uint32_t codes)
{
    const __half2 h(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes), __NV_E4M3));
    if (kHalf)
        return *reinterpret_cast<const uint32_t*>(&h);
    const float2 f = __half22float2(h);
    return pack2<false>(f.x, f.y);
}

template <bool kHalf>
__device__ __forceinline__ uint4 of_e4m3x8(uint32_t lo, uint32_t hi)
{
    return make_uint4(of_e4m3x2<kHalf>(lo & 0xFFFFu), of_e4m3x2<kHalf>(lo >> 16),
                      of_e4m3x2<kHalf>(hi & 0xFFFFu), of_e4m3x2<kHalf>(hi >> 16));
}

// Two fp16 or bf16 numbers, zeros for those that are not finite.
template <bool kHalf>
__device__ __forceinline__ uint32_t finite2(uint32_t two)
{
    constexpr uint32_t kExponent = kHalf ? 0x7C00u : 0x7F80u;
    return two & (((two & kExponent) != kExponent ? 0xFFFFu : 0u) |
                  ((two >> 16 & kExponent) != kExponent ? 0xFFFF0000u : 0u));
}

// o += those of a cached vector's elements [d, d + 16) that are not finite.  Whether any o is a number.
template <int MODE>
__device__ __forceinline__ bool add_not_finite(float (&o)[16], const uint8_t* v, int d)
{
    using T = typename std::conditional<MODE == kModeFp16, __half, __nv_bfloat16>::type;
    constexpr bool kFp8 = MODE >= kModeFp8Bf16;
    uint4 w[kFp8 ? 1 : 2];
#pragma unroll
    for (int k = 0; k < (kFp8 ? 1 : 2); ++k)
        w[k] = reinterpret_cast<const uint4*>(v)[kFp8 ? d / 16 : d / 8 + k];
    bool some = false;
#pragma unroll
    for (int q = 0; q < 16; ++q) {
        if (kFp8) {
            if ((reinterpret_cast<const uint8_t*>(w)[q] & 0x7Fu) == 0x7Fu)
                o[q] = NAN;
        } else {
            const float f = static_cast<float>(reinterpret_cast<const T*>(w)[q]);
            o[q] += isfinite(f) ? 0.0f : f;
        }
        some = some || o[q] == o[q];
    }
    return some;
}

// The low n bits (none below 0, all above 31).
__device__ __forceinline__ uint32_t below(int n)
{
    return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u;
}

template <int D, int MODE>
__global__ void __launch_bounds__(512, 1)
causal_kernel(const __grid_constant__ CausalParams p)
{
    using C = Cfg<D, MODE>;
    extern __shared__ __align__(1024) uint8_t sm[];
    uint8_t* qbuf = sm;                                      // [2 row tiles]
    uint8_t* stages = qbuf + C::kQ;
    uint8_t* raws = stages + C::kStages * C::kStage;
    uint2* valid = reinterpret_cast<uint2*>(raws + C::kRaws * C::kRaw);     // [kKeyRing][2] bits
    uint2* bad = valid + 2 * kKeyRing;                                      // of values, edge tiles
    float* kscale = reinterpret_cast<float*>(bad + 2 * kKeyRing);           // [kKeyRing][128]
    float* vscale = kscale + (C::kFp8 ? kKeyRing * 128 : 0);
    Item* infos = reinterpret_cast<Item*>(vscale + (C::kFp8 ? kKeyRing * 128 : 0));
    uint64_t* kv_full = reinterpret_cast<uint64_t*>(infos + kInfos);
    uint64_t* kv_empty = kv_full + C::kStages;
    uint64_t* q_full = kv_empty + C::kStages;
    uint64_t* q_empty = q_full + 1;
    uint64_t* s_full = q_empty + 1;                          // [2 halves of the keys][2 row tiles]
    uint64_t* p_full = s_full + 4;
    uint64_t* pv_done = p_full + 4;
    uint64_t* info_full = pv_done + 4;
    uint64_t* info_empty = info_full + kInfos;
    uint64_t* drained = info_empty + kInfos;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 2);
    volatile int* ab = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x / 32), 0);
    const int lane = threadIdx.x & 31;
    constexpr int kMmaWarp = 8, kQWarp = 10, kLoadWarp = 12;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(kv_full + i, 4);
            mbar_init(kv_empty + i, 2);
        }
        mbar_init(q_full, 2);
        mbar_init(q_empty, 2);
        for (int i = 0; i < 4; ++i) {
            mbar_init(s_full + i, 1);
            mbar_init(p_full + i, 4);
            mbar_init(pv_done + i, 1);
        }
        for (int i = 0; i < kInfos; ++i) {
            mbar_init(info_full + i, 1);
            mbar_init(info_empty + i, 8 + 2 + 2 + 4);
        }
        mbar_init(drained, 1);
        mbar_init(drained + 1, 1);
        *ab = (smem_u32(sm) & 1023u) != 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    if (threadIdx.x == 32 * kQWarp && p.q_boxes)
        tma_prefetch_desc(&p.q_map);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait_then_release();
    // (a wait that gives up sets the status a whole wait budget after this)
    if (blockIdx.x == 0 && threadIdx.x == 0)
        *p.status = *ab ? kStatusBadArg : 0u;

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
    // The block's it-th item; false at the end of the list or where a wait gave up.
    auto item_of = [&](int it, Item& w) {
        if (!wait(info_full + it % kInfos, (it / kInfos) & 1))
            return false;
        w = infos[it % kInfos];
        return w.tile >= 0;
    };

    if (warp < 8) {
        // ---------------------------------------------------------------- softmax
        // Thread = one row of one of the two row tiles.
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftmaxRegs));
        const int wg = warp / 4, quad = warp & 3;
        const uint32_t lanes = static_cast<uint32_t>(32 * quad) << 16;
        const uint32_t s_row = tmem + lanes + 128 * wg;
        const uint32_t o_at = tmem + lanes + C::kTmemO + D * wg;
        // Weights go by a reference that is replaced once a score passes it by kSlack.  fp16 weights
        // end at 2^-24: theirs is 2^-7 of the maximum, so that they keep their 11 bits down to
        // 2^-21 of it and the largest stays below 2^16.
        constexpr float kSlack = C::kHalfP ? 15.0f : 8.0f;
        constexpr float kBelow = C::kHalfP ? 7.0f : 0.0f;
        uint32_t su = 0;                                     // half tiles so far
        int n = 0;                                           // tiles before this item
        const int i = 128 * wg + 32 * quad + lane;           // row of an item
        // The next item and the thread's row of it, one item ahead: its length is on its way while the
        // item before is written.
        Item w;
        int t = 0, head = 0, row_len = 0, it = 0;
        auto fetch = [&] {
            if (it > 0 && lane == 0)
                mbar_arrive(info_empty + (it - 1) % kInfos);
            const bool more = __all_sync(0xFFFFFFFFu, item_of(it, w));
            if (!more)
                return false;
            __syncwarp();
            ++it;
            const int token = quotient(w.i0 + i, p.by_group);
            head = w.i0 + i - token * p.group + w.g * p.group;
            t = p.row_begin[w.r] + token;
            row_len = i < w.rows ? p.clen[t] : 0;
            return true;
        };
        bool more = fetch();
        while (more) {
            const int count = max(w.tiles - w.tile, 0);
            if (128 * wg >= w.rows) {
                n += count;
                more = fetch();
                continue;
            }
            const bool mine = i < w.rows;
            // places of the list that the row sees: below a, and from c to b
            // (rows that are none see everything, so that nothing is masked for them)
            const int len = max(0, min(row_len, w.keys));
            const int a = min(len, p.sinks), b = mine ? len - w.off : 0x7FFFFFFF;
            const int c = p.window > 0 ? max(0, len - p.window) - w.off : 0;
            float m = -INFINITY, l = 0.0f;                   // reference and sum
            bool ok = true;
            // halves of which the row lost a value, a bit for as many neighbours as 32 bits need
            uint32_t lost = 0;
            const auto bit_of = [&](int h) {
                return 1u << (h >> max(0, 27 - __clz(2 * count - 1)));
            };
            const auto seen = [&](int e) {                   // of 32 places from e on
                return below(a - e) | (below(b - e) & ~below(c - e));
            };
            // A half's weights from its scores in x.  Once for tiles that all rows see and once for the
            // others, whose masks in the same code would cost all tiles a sixth of their time.
            const auto weigh = [&](float(&x)[64], int ring, int half) {
                const uint32_t s_at = s_row + 64 * half;
                if (C::kFp8) {                               // scores times their key's scale
                    const float4* ks =
                        reinterpret_cast<const float4*>(kscale + ring * 128 + 64 * half);
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float4 f = ks[k];
                        mul2(x[4 * k], x[4 * k + 1], pair(f.x, f.y));
                        mul2(x[4 * k + 2], x[4 * k + 3], pair(f.z, f.w));
                    }
                }
                float t4[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    t4[k] = max3(x[16 * k], x[16 * k + 1], x[16 * k + 2]);
#pragma unroll
                    for (int q = 3; q < 15; q += 2)
                        t4[k] = max3(t4[k], x[16 * k + q], x[16 * k + q + 1]);
                    t4[k] = fmaxf(t4[k], x[16 * k + 15]);
                }
                float top = fmaxf(max3(t4[0], t4[1], t4[2]), t4[3]);
                if (!C::kFp8)
                    top *= p.scale_log2;
                // A new reference for rows whose scores have passed the old one.
                const bool raise = top > m + kSlack || (m == -INFINITY && top > -INFINITY);
                if (__any_sync(0xFFFFFFFFu, raise)) {
                    const float to = raise ? top - kBelow : m;
                    const float f = m == -INFINITY ? 0.0f : ex2(m - to);
                    if (__any_sync(0xFFFFFFFFu, raise && m > -INFINITY)) {
                        // the products so far are complete (these scores told of all but the last)
                        ok = __all_sync(0xFFFFFFFFu, wait(pv_done + 2 * (half ^ 1) + wg,
                                                          ((su - 1) >> 1) & 1));
                        tc_fence_after();
                        const float g = m == -INFINITY ? 1.0f : f;
#pragma unroll 1
                        for (int k = 0; k < D; k += 16) {
                            float v[16];
                            tmem_ld_32x32b_x16(o_at + k, v);
                            tmem_wait_ld();
#pragma unroll
                            for (int q = 0; q < 16; ++q)
                                v[q] *= g;
                            tmem_st_32x32b_x8(o_at + k, v);
                            tmem_st_32x32b_x8(o_at + k + 8, v + 8);
                        }
                    }
                    l *= f;
                    m = to;
                }
                const float ref = m == -INFINITY ? 0.0f : m;
                const uint64_t mul = pair(p.scale_log2, p.scale_log2), sub = pair(-ref, -ref);
                const float2* vs = reinterpret_cast<const float2*>(vscale + ring * 128 + 64 * half);
                uint32_t r[32], rest[C::kPTerms > 1 ? 32 : 1];
                uint64_t sum[4] = {};
#pragma unroll
                for (int q = 0; q < 64; q += 2) {
                    float lo = x[q], hi = x[q + 1];
                    if (C::kFp8)
                        unpair(add2(pair(lo, hi), sub), lo, hi);
                    else
                        fma2(lo, hi, mul, sub);
                    lo = ex2(lo);
                    hi = ex2(hi);
                    sum[q / 2 % 4] = add2(sum[q / 2 % 4], pair(lo, hi));
                    if (C::kFp8) {
                        const float2 f = vs[q / 2];
                        mul2(lo, hi, pair(f.x, f.y));
                    }
                    r[q / 2] = pack2<C::kHalfP>(lo, hi);
                    if constexpr (C::kPTerms > 1)            // what is left of them
                        rest[q / 2] = pack2<false>(lo - __uint_as_float(r[q / 2] << 16),
                                                   hi - __uint_as_float(r[q / 2] & 0xFFFF0000u));
                }
                tmem_st_32x32b_x32(s_at, r);
                if constexpr (C::kPTerms > 1)
                    tmem_st_32x32b_x32(s_at + 32, rest);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(p_full + 2 * half + wg);
                float s0, s1;
                unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), s0, s1);
                l += s0 + s1;
            };
#pragma unroll 1
            for (int h = 0; h < 2 * count; ++h, ++su) {
                const int half = su & 1, ring = (n + h / 2) % kKeyRing;
                const uint32_t s_at = s_row + 64 * half;
                ok = wait(s_full + 2 * half + wg, (su >> 1) & 1);
                if (!__all_sync(0xFFFFFFFFu, ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int e0 = w.tile * 128 + 64 * h;
                float x[64];
                tmem_ld_32x32b_x32(s_at, x);
                tmem_ld_32x32b_x32(s_at + 32, x + 32);
                const uint2 keys = valid[2 * ring + half];
                const bool edge = w.edge(w.tile + h / 2);
                tmem_wait_ld();
                if (edge || (keys.x & keys.y) != 0xFFFFFFFFu) {
                    uint64_t blind = 0;                      // values that are not finite
                    if (edge) {
                        const int load = 2 * (n + h / 2) + 1;
                        ok = __all_sync(0xFFFFFFFFu, wait(kv_full + load % C::kStages,
                                                          (load / C::kStages) & 1));
                        const uint2 v = bad[2 * ring + half];
                        blind = v.x | static_cast<uint64_t>(v.y) << 32;
                    }
                    const bool whole = (e0 + 64 <= a || (e0 >= c && e0 + 64 <= b)) && blind == 0 &&
                                       (keys.x & keys.y) == 0xFFFFFFFFu;
                    if (!__all_sync(0xFFFFFFFFu, whole)) {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int e = e0 + 32 * k;
                            const uint32_t see = seen(e) & (k == 0 ? keys.x : keys.y);
                            if ((see & static_cast<uint32_t>(blind >> (32 * k))) != 0u)
                                lost |= bit_of(h);
#pragma unroll
                            for (int q = 0; q < 32; ++q)
                                x[32 * k + q] = (see >> q) & 1u ? x[32 * k + q] : -INFINITY;
                        }
                    }
                    weigh(x, ring, half);
                } else {
                    weigh(x, ring, half);
                }
            }
            if (!ok)
                break;
            n += count;
            lost = mine ? lost : 0u;
            if (__any_sync(0xFFFFFFFFu, lost != 0u)) {
                // Values that are not finite, of keys that some rows do not see, were taken out of their
                // tiles: rows that see one get it in its column here, from the cache.
                const uint32_t parity = ((su - 1) >> 1) & 1;
                ok = wait(pv_done + wg, parity) && wait(pv_done + 2 + wg, parity);
                if (!__all_sync(0xFFFFFFFFu, ok))
                    break;
                tc_fence_after();
                const Item& s = infos[(it - 1) % kInfos];
                const uint8_t* vh = p.v + s.g * p.v_head;
                const int32_t* table = p.table + s.r * p.ld_table;
#pragma unroll 1
                for (int d = 0; d < D; d += 16) {
                    float o[16];
                    tmem_ld_32x32b_x16(o_at + d, o);
                    tmem_wait_ld();
#pragma unroll 1
                    bool left = lost != 0u;                  // until no column is a number
#pragma unroll 1
                    for (int h = 0; left && h < 2 * count; ++h) {
                        if (!(lost & bit_of(h)) || !s.edge(s.tile + h / 2))
                            continue;
#pragma unroll 1
                        for (int e = s.tile * 128 + 64 * h, end = e + 64; left && e < end; ++e) {
                            if (!(e < a || (e >= c && e < b)))
                                continue;
                            int64_t slot = e < s.sinks ? e : e + s.off;
                            if (p.page > 0) {
                                const int pg = quotient(static_cast<int>(slot), p.by_page);
                                const int page = table[pg];
                                slot = page < 0 ? -1 : slot + ((int64_t)page - pg) * p.page;
                            } else {
                                slot += s.base;
                            }
                            if (slot < 0 || slot >= p.num_slots)
                                continue;
                            left = add_not_finite<MODE>(o, vh + slot * p.v_slot, d);
                        }
                    }
                    __syncwarp();
                    tmem_st_32x32b_x8(o_at + d, o);
                    tmem_st_32x32b_x8(o_at + d + 8, o + 8);
                }
                tmem_wait_st();
            }
            // ---- output
            const int part = w.part, out_t = t, out_head = head;
            more = fetch();
            if (count > 0) {
                const uint32_t parity = ((su - 1) >> 1) & 1;
                ok = wait(pv_done + wg, parity) && wait(pv_done + 2 + wg, parity);
                if (!__all_sync(0xFFFFFFFFu, ok))
                    break;
                tc_fence_after();
            }
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            const float lse = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
            const int64_t at = (int64_t)part * kRows + i;
            uint8_t* out = p.out + out_t * p.out_row + out_head * p.out_head;
            if (mine && part >= 0)
                p.part_lse[at] = lse;
            else if (mine && p.lse)
                p.lse[(int64_t)out_t * p.Hq + out_head] = lse;
            // (the next columns are read while these are written)
            float v[2][32];
            if (count > 0)
                tmem_ld_32x32b_x32(o_at, v[0]);
#pragma unroll
            for (int k = 0; k < D; k += 32) {
                float(&o)[32] = v[(k / 32) & 1];
                if (count > 0) {
                    tmem_wait_ld();
                    if (k + 32 < D)
                        tmem_ld_32x32b_x32(o_at + k + 32, v[(k / 32 + 1) & 1]);
                }
                if (part >= 0) {
                    if (mine && l != 0.0f) {
#pragma unroll
                        for (int q = 0; q < 32; q += 8) {
                            uint32_t r[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                r[e] = __float_as_uint(o[q + e] * inv);
                            stg256(p.part_o + at * D + k + q, r);
                        }
                    }
                } else if (mine) {
                    uint32_t r[16];
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        r[q] = l == 0.0f ? 0u : pack2<C::kHalfS>(o[2 * q] * inv, o[2 * q + 1] * inv);
                    if (p.out_vec) {
                        stg256(out + 2 * k, r);
                        stg256(out + 2 * k + 32, r + 8);
                    } else {
#pragma unroll
                        for (int q = 0; q < 16; ++q) {
                            reinterpret_cast<uint16_t*>(out + 2 * k)[2 * q] = r[q] & 0xFFFFu;
                            reinterpret_cast<uint16_t*>(out + 2 * k)[2 * q + 1] = r[q] >> 16;
                        }
                    }
                }
                __syncwarp();
            }
            tc_fence_before();
        }
        __syncwarp();
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kLaunchRegs));
    } else if (warp >= kLoadWarp) {
        // ------------------------------------------------------- keys and values
        // A warp takes 32 keys of every tile, a lane looks one of them up.  Copies are signalled
        // kLag loads later, once they have landed; e4m3 codes land in a ring of their own and are
        // converted by the lane that copied them.
        if (C::kLoadRegs < C::kLaunchRegs)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kLoadRegs));
        constexpr int kEb = C::kFp8 ? 1 : 2;
        constexpr int kPer = D * kEb / 16;                   // copies of a vector
        constexpr int kAtOnce = 32 / kPer;                   // vectors of a warp's instruction
        const int row0 = 32 * (warp - kLoadWarp), chunk = lane % kPer, sub = lane / kPer;
        int st = 0, phase = 1, raw = 0;                      // next place, its empty parity
        int done_st = 0, done_raw = 0;                       // next place to signal
        int n = 0;                                           // tiles so far
        bool ok = true;
        // Signal the oldest load (its copies have landed).
        auto signal = [&](bool is_v, bool edge, int ring) {
            if (C::kFp8) {
                // into the place, once its last reader has left it
                ok = __all_sync(0xFFFFFFFFu, ok && wait(kv_empty + st, phase));
                if (!ok)
                    return;
                const uint32_t from = smem_u32(raws + done_raw * C::kRaw) + row0 * D + lane * 16;
                const uint32_t to = smem_u32(stages + st * C::kStage);
                auto convert = [&](auto half) {
                    constexpr bool kHalf = decltype(half)::value;
#pragma unroll
                    for (int k = 0; k < kPer; k += 4) {
                        uint4 w[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            w[q] = lds128(from + (k + q) * 512);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int row = row0 + (k + q) * kAtOnce + sub;
                            const uint32_t off = (chunk / 4) * C::kAtom + row * 128 + (chunk % 4) * 32;
                            sts128(to + swizzled(off), of_e4m3x8<kHalf>(w[q].x, w[q].y));
                            sts128(to + swizzled(off + 16), of_e4m3x8<kHalf>(w[q].z, w[q].w));
                        }
                    }
                };
                if (is_v || !C::kHalfS)
                    convert(std::false_type());
                else
                    convert(std::true_type());
                if (++st == C::kStages) {
                    st = 0;
                    phase ^= 1;
                }
                done_raw = done_raw + 1 == C::kRaws ? 0 : done_raw + 1;
            }
            if (is_v && edge) {
                // A weight of 0 times a value that is not finite would be NaN in rows that do not see
                // the key: such values become zeros, and rows that see the key are told.
                __syncwarp();
                uint8_t* v = stages + done_st * C::kStage + (row0 + lane) * 128;
                using T2 = typename std::conditional<C::kHalfP, __half2, __nv_bfloat162>::type;
                const T2 none = {0.0f, 0.0f};
                T2 sum = none;
#pragma unroll 4
                for (int x = 0; x < D / 8; ++x) {
                    const uint4 w = *reinterpret_cast<const uint4*>(
                        v + (x / 8) * C::kAtom + (((x ^ lane) & 7) << 4));
                    const T2* two = reinterpret_cast<const T2*>(&w);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        sum = __hfma2(two[k], none, sum);
                }
                const float2 f = {static_cast<float>(sum.x), static_cast<float>(sum.y)};
                const bool not_finite = !(f.x == 0.0f && f.y == 0.0f);
                const uint32_t bits = __ballot_sync(0xFFFFFFFFu, not_finite);
                if (not_finite)
#pragma unroll 1
                    for (int x = 0; x < D / 4; ++x) {
                        uint2* two =
                            reinterpret_cast<uint2*>(v + (x / 16) * C::kAtom + (x & 15) * 8);
                        *two = make_uint2(finite2<C::kHalfP>(two->x), finite2<C::kHalfP>(two->y));
                    }
                if (lane == 0)
                    reinterpret_cast<uint32_t*>(bad + 2 * ring)[warp - kLoadWarp] = bits;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(kv_full + done_st);
            done_st = done_st + 1 == C::kStages ? 0 : done_st + 1;
        };
        for (int it = 0; ok; ++it) {
            Item w;
            if (!__all_sync(0xFFFFFFFFu, item_of(it, w)))
                break;
            __syncwarp();
            if (lane == 0)
                mbar_arrive(info_empty + it % kInfos);
            const int32_t* table = p.table + w.r * p.ld_table;
            const uint8_t* kh = p.k + w.g * p.k_head + chunk * 16;
            const uint8_t* vh = p.v + w.g * p.v_head + chunk * 16;
            // the lane's key of a tile: its page and place there
            int page = -1, rest = 0;
            auto look = [&](int tile) {
                const int e = tile * 128 + row0 + lane;
                page = -1;
                rest = e < w.sinks ? e : e + w.off;
                if (e < w.n) {
                    page = 0;
                    if (p.page > 0) {
                        const int pg = quotient(rest, p.by_page);
                        page = table[pg];
                        rest -= pg * p.page;
                    } else {
                        rest += w.base;
                    }
                }
            };
            int loads = 0, signalled = 0;                    // of this item
            const int n0 = n;
            auto signal_next = [&] {
                signal(signalled & 1, w.edge(w.tile + signalled / 2),
                       (n0 + signalled / 2) % kKeyRing);
                ++signalled;
            };
            if (w.tile < w.tiles)
                look(w.tile);
            for (int tile = w.tile; tile < w.tiles && ok; ++tile, ++n) {
                const int64_t at = (int64_t)page * p.page + rest;
                const int32_t slot = page >= 0 && at < p.num_slots ? static_cast<int32_t>(at) : -1;
                const uint32_t bits = __ballot_sync(0xFFFFFFFFu, slot >= 0);
                // (scales of keys that a row sees are positive and finite; others leave -inf and 0 as
                // they are)
                float ks = 1.0f, vs = 1.0f;
                if (C::kFp8 && slot >= 0) {
                    ks = p.k_scale[(int64_t)slot * p.Hkv + w.g];
                    vs = p.v_scale[(int64_t)slot * p.Hkv + w.g];
                    ks = ks > 0.0f && ks < INFINITY ? ks : 1.0f;
                    vs = vs > 0.0f && vs < INFINITY ? vs : 1.0f;
                }
                ks = fmaxf(ks * p.scale_log2, 1.17549435e-38f);      // (0 times -inf is none)
                if (tile + 1 < w.tiles)
                    look(tile + 1);
#pragma unroll 1
                for (int is_v = 0; is_v < 2; ++is_v) {
                    uint32_t to;
                    if (!C::kFp8) {
                        // no place yet: what has been asked for is signalled before the wait
                        if (!__all_sync(0xFFFFFFFFu, mbar_test_wait(kv_empty + st, phase))) {
                            if (signalled < loads)
                                cp_async_wait<0>();
                            while (signalled < loads)
                                signal_next();
                            ok = __all_sync(0xFFFFFFFFu, wait(kv_empty + st, phase));
                            if (!ok)
                                break;
                        }
                        to = smem_u32(stages + st * C::kStage);
                        if (++st == C::kStages) {
                            st = 0;
                            phase ^= 1;
                        }
                    } else {
                        to = smem_u32(raws + raw * C::kRaw) + row0 * D + lane * 16;
                        raw = raw + 1 == C::kRaws ? 0 : raw + 1;
                    }
                    const uint8_t* src = is_v ? vh : kh;
                    const uint32_t stride = static_cast<uint32_t>(is_v ? p.v_slot : p.k_slot);
                    // (16-bit vectors: chunk x of row y of eight is at x ^ y)
                    if (!C::kFp8)
                        to += (chunk / 8) * C::kAtom + (row0 + sub) * 128 + ((chunk ^ sub) % 8) * 16;
#pragma unroll
                    for (int k = 0; k < kPer; ++k) {
                        const int32_t s = __shfl_sync(0xFFFFFFFFu, slot, k * kAtOnce + sub);
                        const uint32_t at = C::kFp8 ? to + k * 512
                                                    : (to ^ (k * kAtOnce % 8 * 16)) +
                                                          k * kAtOnce * 128;
                        cp_async16(at, src + static_cast<uint64_t>(static_cast<uint32_t>(max(s, 0))) * stride,
                                   s >= 0);
                    }
                    cp_async_commit();
                    ++loads;
                    if (loads - signalled > C::kLag) {
                        cp_async_wait<C::kLag>();
                        signal_next();
                    }
                    if (is_v == 0) {
                        // (the ring's place was last read for a tile whose keys have left their stage)
                        const int ring = n % kKeyRing;
                        if (lane == 0)
                            reinterpret_cast<uint32_t*>(valid + 2 * ring)[warp - kLoadWarp] = bits;
                        if (C::kFp8) {
                            kscale[ring * 128 + row0 + lane] = ks;
                            vscale[ring * 128 + row0 + lane] = vs;
                        }
                    }
                }
            }
            // The item's last loads: the next item may be a long wait away.
            if (ok) {
                cp_async_wait<0>();
                while (signalled < loads && ok)
                    signal_next();
            }
        }
        cp_async_wait<0>();                                  // (of a wait that gave up)
        __syncwarp();
        if (C::kLoadRegs < C::kLaunchRegs)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kLaunchRegs));
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kFeedRegs));
        if (warp >= kQWarp) {
            // ------------------------------------------------- items and queries
            // Both warps load queries; the first lists the items, two ahead of those it loads for.
            // The block's share of all items' key tiles, as it was planned: from the first's on.
            int item = p.cut_item[blockIdx.x], begin = p.cut_tile[blockIdx.x];
            const int last_item = p.cut_item[blockIdx.x + 1], end = p.cut_tile[blockIdx.x + 1];
            int listed = 0;
            bool more = true;
            auto list = [&] {
                const int it = listed++;
                Item w = {};
                w.tile = -1;
                more = item < last_item || (item == last_item && begin < end);
                if (!__all_sync(0xFFFFFFFFu,
                                wait(info_empty + it % kInfos, ((it / kInfos) & 1) ^ 1))) {
                    more = false;
                    return;
                }
                if (more) {
                    const int d = quotient(item, p.by_hkv);
                    w.g = item - d * p.Hkv;
                    int lo = 0, hi = p.num_requests - 1;     // the request of row tile d
                    while (lo < hi) {
                        const int mid = (lo + hi + 1) >> 1;
                        if (p.tile_begin[mid] <= d)
                            lo = mid;
                        else
                            hi = mid - 1;
                    }
                    w.r = lo;
                    w.i0 = (d - p.tile_begin[lo]) * kRows;
                    const int row0 = p.row_begin[lo], tokens = p.row_begin[lo + 1] - row0;
                    w.rows = min(kRows, tokens * p.group - w.i0);
                    w.base = p.key_begin[lo];
                    w.keys = p.key_begin[lo + 1] - w.base;
                    const int t0 = quotient(w.i0, p.by_group);
                    const int t1 = quotient(w.i0 + w.rows - 1, p.by_group);
                    // the rows' longest and shortest length, their windows' first and last beginning
                    int most = 0, fewest = 0x7FFFFFFF, least = 0x7FFFFFFF, latest = 0;
                    for (int t = t0 + lane; t <= t1; t += 32) {
                        const int len = max(0, min(p.clen[row0 + t], w.keys));
                        const int lo = p.window > 0 ? max(0, len - p.window) : 0;
                        most = max(most, len);
                        fewest = min(fewest, len);
                        latest = max(latest, lo);
                        if (len > 0)
                            least = min(least, lo);
                    }
                    most = __reduce_max_sync(0xFFFFFFFFu, most);
                    fewest = __reduce_min_sync(0xFFFFFFFFu, fewest);
                    latest = __reduce_max_sync(0xFFFFFFFFu, latest);
                    least = min(__reduce_min_sync(0xFFFFFFFFu, least), most);
                    if (least > p.sinks) {
                        w.sinks = p.sinks;
                        w.off = least - p.sinks;
                    }
                    w.n = most - w.off;
                    w.inner = latest - w.off;
                    w.outer = fewest - w.off;
                    const int tiles = (w.n + 127) / 128;
                    const int planned =
                        causal_tiles(w.keys, tokens, t0, t1, p.window, p.sinks);
                    const int to = item == last_item ? end : planned;
                    // the part's share of the tiles that there are
                    w.tile = static_cast<int>((int64_t)begin * tiles / planned);
                    w.tiles = static_cast<int>((int64_t)to * tiles / planned);
                    const int place = 2 * static_cast<int>(blockIdx.x);
                    w.part = begin > 0 ? place : to < planned ? place + 1 : -1;
                }
                if (lane == 0) {
                    infos[it % kInfos] = w;
                    mbar_arrive(info_full + it % kInfos);
                }
                ++item;
                begin = 0;
            };
            constexpr int kPer = D / 8;                      // copies of a vector
            const int from = threadIdx.x - 32 * kQWarp;      // of 64 threads
            // x / group as the high word of a product, exact for x group < 2^32
            const uint32_t q_row = static_cast<uint32_t>(p.q_row);
            const uint32_t q_head = static_cast<uint32_t>(p.q_head);
            const uint32_t group_inv = p.group > 1 ? 0xFFFFFFFFu / p.group + 1 : 0u;
            uint32_t u = 0;
            for (int it = 0;; ++it) {
                while (warp == kQWarp && more && listed < it + 3)
                    list();
                Item w;
                if (!__all_sync(0xFFFFFFFFu, item_of(it, w)))
                    break;
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(info_empty + it % kInfos);
                if (w.tile >= w.tiles)
                    continue;
                if (!__all_sync(0xFFFFFFFFu, wait(q_empty, (u & 1) ^ 1)))
                    break;
                ++u;
                if (p.q_boxes) {
                    // A box is a row tile's 128 (token, head) pairs, in the tile's own order.  Tokens past
                    // the request's are another's or zeros, rows that are none.  (By cp.async, 256 rows of
                    // 128 took 10,000 cycles beside the softmax, most of an item's beginning.)
                    const int x = warp - kQWarp;
                    if (lane == 0 && 128 * x < w.rows) {
                        const int token = p.row_begin[w.r] + quotient(w.i0 + 128 * x, p.by_group);
                        mbar_arrive_expect_tx(q_full, C::kStage);
#pragma unroll
                        for (int k = 0; k < D / 64; ++k)
                            tma_load_3d(qbuf + x * C::kStage + k * C::kAtom, &p.q_map, q_full, 64 * k,
                                        w.g * p.group, token);
                    } else if (lane == 0) {
                        mbar_arrive(q_full);
                    }
                    __syncwarp();
                    continue;
                }
                const int rows = w.rows > 128 ? 256 : 128;
                // row x of the item: (token, head of the group), counted from the first row's token
                constexpr int kStep = 64 / kPer;
                const int chunk = from % kPer, first = from / kPer;
                const int t0 = quotient(w.i0, p.by_group), h0 = w.i0 - t0 * p.group;
                const uint8_t* src = p.q + (int64_t)(p.row_begin[w.r] + t0) * p.q_row +
                                     (int64_t)(w.g * p.group) * p.q_head + chunk * 16;
                const uint32_t to = smem_u32(qbuf) + (chunk / 8) * C::kAtom;
#pragma unroll 8
                for (int x = first; x < rows; x += kStep) {
                    const uint32_t token = group_inv ? __umulhi(h0 + x, group_inv) : h0 + x;
                    const uint32_t head = h0 + x - token * p.group;
                    const uint8_t* at = src + static_cast<uint64_t>(token) * q_row +
                                        static_cast<uint64_t>(head) * q_head;
                    // (row tiles are kStage apart)
                    const uint32_t off = (x / 128) * C::kStage + x % 128 * 128 + (((chunk ^ x) & 7) << 4);
                    cp_async16(to + off, x < w.rows ? at : p.q, x < w.rows);
                }
                cp_async_commit();
                cp_async_wait<0>();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(q_full);
            }
        } else {
            // --------------------------------------------------------- products
            // A warp for each row tile, an elected lane issues everything, in this order: the next
            // scores of a half go over the weights whose product was issued just before.
            if (elect_one()) {
                constexpr uint32_t s_desc = idesc_dense(128, 64, C::kHalfS ? 0 : 1, false, false);
                constexpr uint32_t o_desc = idesc_dense(128, D, C::kHalfP ? 0 : 1, false, true);
                const int rt = warp - kMmaWarp;
                const uint32_t s_at = tmem + 128 * rt, o_at = tmem + C::kTmemO + D * rt;
                const uint64_t q = smem_desc(smem_u32(qbuf + rt * C::kStage), 128, 16, 1024);
                const uint64_t kd = smem_desc(smem_u32(stages), 128, 16, 1024);
                const uint64_t vd = smem_desc(smem_u32(stages), 128, C::kAtom, 1024);
                uint32_t u = 0, pu = 0;                      // items, weight tiles so far
                int st = 0, phase = 0;
                bool ok = true;
                auto next = [&](int& s) {                    // a place of the ring and the next one
                    s = st;
                    const bool r = wait(kv_full + st, phase);
                    if (++st == C::kStages) {
                        st = 0;
                        phase ^= 1;
                    }
                    return r;
                };
                auto scores = [&](int half, int place) {
                    const uint64_t k = kd + (place * C::kStage + half * 8192) / 16;
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        const int at = ((i / 4) * C::kAtom + (i % 4) * 32) / 16;
                        mma_f16(s_at + 64 * half, q + at, k + at, s_desc, i > 0);
                    }
                    mma_commit(s_full + 2 * half + rt);
                };
                auto products = [&](int half, int place, bool more) {
                    if (!wait(p_full + 2 * half + rt, pu & 1))
                        return false;
                    tc_fence_after();
                    const uint64_t v = vd + (place * C::kStage + half * 8192) / 16;
#pragma unroll
                    for (int i = 0; i < 4 * C::kPTerms; ++i)
                        mma_f16_tmem(o_at, s_at + 64 * half + 32 * (i / 4) + 8 * (i % 4),
                                     v + i % 4 * 128, o_desc, more || i > 0);
                    mma_commit(pv_done + 2 * half + rt);
                    return true;
                };
                for (int it = 0; ok; ++it) {
                    Item w;
                    if (!item_of(it, w))
                        break;
                    mbar_arrive(info_empty + it % kInfos);
                    const int count = w.tiles - w.tile;
                    if (count <= 0)
                        continue;
                    int ks, vs;
                    ok = wait(q_full, u & 1);
                    ++u;
                    if (128 * rt >= w.rows) {                // no such rows: hand everything on
                        mbar_arrive(q_empty);
                        for (int j = 0; j < 2 * count && ok; ++j) {
                            ok = next(ks);
                            mbar_arrive(kv_empty + ks);
                        }
                        continue;
                    }
                    ok = ok && next(ks);
                    if (!ok)
                        break;
                    tc_fence_after();
                    scores(0, ks);
                    scores(1, ks);
                    mma_commit(kv_empty + ks);
                    if (count == 1)
                        mma_commit(q_empty);
                    for (int j = 0; j < count; ++j, ++pu) {
                        const bool last = j + 1 == count;
                        ok = next(vs) && products(0, vs, j > 0);
                        if (ok && !last) {
                            ok = next(ks);
                            tc_fence_after();
                            if (ok)
                                scores(0, ks);
                        }
                        ok = ok && products(1, vs, true);
                        if (!ok)
                            break;
                        mma_commit(kv_empty + vs);
                        if (!last) {
                            scores(1, ks);
                            mma_commit(kv_empty + ks);
                            if (j + 2 == count)
                                mma_commit(q_empty);
                        }
                    }
                }
                // what was issued, and its arrivals, end before the memory goes
                mma_commit(drained + rt);
                for (int i = 0; i < kWaitTries && !mbar_try_wait_sleep(drained + rt, 0, 1000u); ++i)
                    ;
            }
        }
        __syncwarp();
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kLaunchRegs));
    }
    __syncthreads();
    if (threadIdx.x == 0 && *ab == kGaveUp)
        atomicOr(p.status, kStatusTimeout);
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Items that end in another block than they began: their parts, weighted by their log-sum-exps.  The
// grid's x is such an item, a warp takes a row, or (W = 4, items of many parts) a block, whose warps take
// every fourth part: 38 parts of 128 rows one after another took a warp 12 us.  Parts without a key
// were not written and are not read.
template <typename T, int D, int W>
__global__ void __launch_bounds__(128)
causal_join_kernel(const __grid_constant__ CausalParams p)
{
    pdl_wait_then_release();
    const int cut = p.first_cut[blockIdx.x], item = p.cut_item[cut];
    int end = cut + 1;                                       // the blocks [cut - 1, end) share it
    while (end < p.blocks && p.cut_item[end] == item && p.cut_tile[end] > 0)
        ++end;
    const int d = quotient(item, p.by_hkv), g = item - d * p.Hkv;
    int r = 0, hi = p.num_requests - 1;
    while (r < hi) {
        const int mid = (r + hi + 1) >> 1;
        if (p.tile_begin[mid] <= d)
            r = mid;
        else
            hi = mid - 1;
    }
    const int i0 = (d - p.tile_begin[r]) * kRows, row0 = p.row_begin[r];
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int i = blockIdx.y * (4 / W) + warp / W;
    if (i >= min(kRows, (p.row_begin[r + 1] - row0) * p.group - i0))
        return;                                              // (with W = 4 the whole block)
    const int token = quotient(i0 + i, p.by_group);
    const int64_t t = row0 + token;
    const int head = i0 + i - token * p.group + g * p.group;
    const int parts = end - cut + 1;
    // (the first part is its block's last item, the others are their blocks' first)
    auto place = [&](int s) { return (int64_t)(2 * (cut - 1 + s) + (s == 0)) * kRows + i; };
    constexpr int kEach = kCausalBlocks / 32 + 1;
    float f[kEach], m = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const int s = lane + 32 * k;
        f[k] = s < parts ? p.part_lse[place(s)] : -INFINITY;
        m = fmaxf(m, f[k]);
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, x));
    const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        f[k] = exp2f((f[k] - ref) * 1.4426950408889634f);
        sum += f[k];
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1)
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, x);
    constexpr int N = D / 32;
    float o[N] = {};
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        for (int s0 = 32 * k + warp % W; s0 < min(parts, 32 * k + 32); s0 += 4 * W) {
            float in[4][N], w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                // (0 past the parts, and past this 32)
                const int s = s0 + W * q;
                w[q] = __shfl_sync(0xFFFFFFFFu, f[k], s & 31);
                w[q] = s < 32 * k + 32 ? w[q] : 0.0f;
                if (w[q] == 0.0f)
                    continue;
                const float* at = p.part_o + place(s) * D + N * lane;
                if (N == 4)
                    *reinterpret_cast<float4*>(in[q]) = *reinterpret_cast<const float4*>(at);
                else
                    *reinterpret_cast<float2*>(in[q]) = *reinterpret_cast<const float2*>(at);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int e = 0; e < N; ++e)
                    o[e] = w[q] != 0.0f ? fmaf(in[q][e], w[q], o[e]) : o[e];
        }
    }
    if constexpr (W > 1) {
        __shared__ float both[W][D];
#pragma unroll
        for (int e = 0; e < N; ++e)
            both[warp][N * lane + e] = o[e];
        __syncthreads();
        if (warp > 0)
            return;
#pragma unroll
        for (int e = 0; e < N; ++e)
            for (int q = 1; q < W; ++q)
                o[e] += both[q][N * lane + e];
    }
    T* out = reinterpret_cast<T*>(p.out + t * p.out_row + head * p.out_head) + N * lane;
    const float inv = sum > 0.0f ? 1.0f / sum : sum;
#pragma unroll
    for (int e = 0; e < N; ++e)
        out[e] = static_cast<T>(o[e] * inv);
    if (p.lse && lane == 0)
        p.lse[t * p.Hq + head] = m == -INFINITY ? m : ref + log2f(sum) * 0.693147180559945309f;
}

template <int D, int MODE>
cudaError_t causal(const CausalParams& p, cudaStream_t st)
{
    using C = Cfg<D, MODE>;
    static std::atomic<uint64_t> ready;
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e == cudaSuccess)
        e = once_per_device(ready, device, [] {
            // the warpgroups' trade has to add up against what a block is launched with
            cudaFuncAttributes a;
            cudaError_t r = cudaFuncGetAttributes(&a, causal_kernel<D, MODE>);
            if (r == cudaSuccess && a.numRegs != C::kLaunchRegs)
                r = cudaErrorLaunchOutOfResources;
            return r != cudaSuccess
                       ? r
                       : cudaFuncSetAttribute(causal_kernel<D, MODE>,
                                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                                              C::kSmem);
        });
    if (e != cudaSuccess)
        return e;
    e = launch_pdl(causal_kernel<D, MODE>, dim3(p.blocks), dim3(C::kThreads), C::kSmem, st, p);
    if (e != cudaSuccess || !p.joined)
        return e;
    using T = typename std::conditional<C::kHalfS, __half, __nv_bfloat16>::type;
    count_launch();
    if (p.blocks > 4 * p.joined)
        return launch_pdl(causal_join_kernel<T, D, 4>, dim3(p.joined, p.most_rows), dim3(128), 0, st, p);
    return launch_pdl(causal_join_kernel<T, D, 1>, dim3(p.joined, (p.most_rows + 3) / 4), dim3(128), 0,
                      st, p);
}

template <int MODE>
cudaError_t causal_mode(const CausalParams& p, int D, cudaStream_t st)
{
    return D == 64 ? causal<64, MODE>(p, st) : causal<128, MODE>(p, st);
}

}  // namespace

cudaError_t launch_causal(const CausalParams& p, int D, int dtype, bool fp8, cudaStream_t st)
{
    if (dtype == IDX_BF16)
        return fp8 ? causal_mode<kModeFp8Bf16>(p, D, st) : causal_mode<kModeBf16>(p, D, st);
    return fp8 ? causal_mode<kModeFp8Fp16>(p, D, st) : causal_mode<kModeFp16>(p, D, st);
}

}  // namespace idx
