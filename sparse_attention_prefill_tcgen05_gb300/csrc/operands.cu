// Rotary positions and the quantised operands and caches the indexer and the sparse
// attention read: rotation, quantising rows into cache slots, reading them back.
//
// Every kernel here reads its input once and writes its output once; what bounds them is
// HBM traffic (large calls) or launch latency (small ones).
#include <algorithm>
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "indexer.h"
#include "elements.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace idx {
namespace {

constexpr int kThreads = 256;
constexpr int kAppendRows = 1024;   // rows of a block: kThreads / 2 groups of eight vectors at most

// Cosine and sine (times the amplitude) of a pair's turn at a position.  position * inc
// modulo 2^64 is the angle in 2^-64 turns, exactly; its top 32 bits are a quarter turn q and
// a remainder of at most an eighth of a turn, which becomes radians with one rounding (its
// upper bits and its lowest six are exact in fp32, 2 pi 2^-32 is two numbers).  On that range
// the Taylor series of sine and cosine to the ninth and tenth power leave 2e-9, so the error
// is some units in fp32's last place, below 1.5e-7, at every position (a 32-bit product of
// position and frequency would be off by 0.03 rad at position 487,935).
__device__ __forceinline__ float2 turn(const RopeParams& rp, int32_t pos, uint64_t inc)
{
    const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(pos)) * inc;
    const uint32_t top = static_cast<uint32_t>(phase >> 32);
    const uint32_t q = (top + 0x20000000u) >> 30;
    const int32_t rest = static_cast<int32_t>(top - (q << 30));
    constexpr double kUnit = 6.283185307179586 / 4294967296.0;
    constexpr float kHi = static_cast<float>(kUnit), kLo = static_cast<float>(kUnit - kHi);
    const float upper = static_cast<float>(rest & ~63), lower = static_cast<float>(rest & 63);
    const float z = fmaf(upper, kHi, fmaf(upper, kLo, lower * kHi));
    const float y = z * z;
    float s = fmaf(y, 1.0f / 362880.0f, -1.0f / 5040.0f);
    s = fmaf(y, s, 1.0f / 120.0f);
    s = fmaf(y, s, -1.0f / 6.0f);
    s = fmaf(z * y, s, z);
    float c = fmaf(y, -1.0f / 3628800.0f, 1.0f / 40320.0f);
    c = fmaf(y, c, -1.0f / 720.0f);
    c = fmaf(y, c, 1.0f / 24.0f);
    c = fmaf(y, c, -0.5f);
    c = fmaf(y, c, 1.0f);
    const float cq = (q & 1u) ? s : c, sq = (q & 1u) ? c : s;
    const float ca = ((q + 1u) & 2u) ? -rp.amplitude : rp.amplitude;
    const float sa = (((q & 2u) != 0u) != (rp.inverse != 0)) ? -rp.amplitude : rp.amplitude;
    return make_float2(cq * ca, sq * sa);
}

// A vector's 16 elements of one thread: unit u of the rotated part holds eight pairs, as
// eight elements at `a` and their partners at `b` (half layout) or as sixteen neighbours
// (interleaved; b = a + 8).  The units after those hold the elements left alone, eight from
// their first half and eight from their second, so that neighbouring threads read
// neighbouring 16 bytes; the last may have only one eight (b < 0).
struct Unit {
    int a, b;       // element offsets of the two groups of eight
    bool rotated;
};

__device__ __forceinline__ Unit unit_of(int rot, int offset, int interleaved, int u, int D)
{
    Unit r;
    const int nrot = rot / 16;
    r.rotated = u < nrot;
    if (r.rotated) {
        r.a = offset + (interleaved ? 16 * u : 8 * u);
        r.b = interleaved ? r.a + 8 : r.a + rot / 2;
    } else {
        const int rest = D - rot;
        const int e = 8 * (u - nrot), f = e + (rest + 15) / 16 * 8;   // among those left alone
        r.a = e < offset ? e : e + rot;
        r.b = f >= rest ? -1 : f < offset ? f : f + rot;
    }
    return r;
}
__device__ __forceinline__ Unit unit_of(const RopeParams& rp, int u, int D)
{
    return unit_of(rp.rot, rp.offset, rp.interleaved, u, D);
}

// What a block of the kernels below does: vectors (row, head) of up to `rows` rows and
// `heads` heads, `lanes` threads each (one unit a thread), as many at once as the block has
// groups of lanes, and a few per group with their loads in flight together.
struct Tiling {
    int32_t rows, heads, lanes, groups;
    int32_t batch;               // vectors a group takes
    int32_t angle_rows;          // rows whose angles the block's threads take at a time
    uint32_t by_heads, by_lanes, by_pairs;   // for quotient()
};

// q / d for q and d up to 2^16 as the high word of q * reciprocal(d); d = 1 has none.
__device__ __forceinline__ int quotient(uint32_t q, uint32_t reciprocal)
{
    return reciprocal ? __umulhi(q, reciprocal) : q;
}
uint32_t reciprocal(int d)
{
    return d == 1 ? 0u : static_cast<uint32_t>(((1ull << 32) + d - 1) / d);
}

constexpr int kAngles = 2048;    // cosines and sines a block keeps

// The angles of a block's rows, once for all heads: those of two neighbouring pairs of row r
// as one 16-byte word (their cosines, their sines), where the thread of their unit finds its
// four words without bank conflicts.  A thread takes one pair for every angle_rows-th row.
__device__ __forceinline__ void block_angles(const RopeParams& rp, const Tiling& t,
                                             const int32_t* positions, int rows, float* cs)
{
    const int pairs = rp.rot / 2, units = rp.rot / 16;
    int r = quotient(threadIdx.x, t.by_pairs);
    const int i = threadIdx.x - r * pairs;
    if (r >= t.angle_rows)
        return;
    // a plain load: as an indexed constant, lanes of different pairs would take turns
    const uint64_t* table = rp.inc;
    asm volatile("" : "+l"(table));
    const uint64_t inc = table[i];
    float* o = cs + ((i % 8) / 2 * units + i / 8) * 4 + (i & 1);
    for (; r < rows; r += t.angle_rows) {
        const float2 v = turn(rp, positions[r], inc);
        o[r * 2 * pairs] = v.x;
        o[r * 2 * pairs + 2] = v.y;
    }
}

// A unit's 16 elements turned by its eight angles (`cs`: the row's, u: the unit).
__device__ __forceinline__ void rotate16(const RopeParams& rp, const float* cs, int u,
                                         float (&a)[8], float (&b)[8])
{
    const int units = rp.rot / 16;
    const float4* p = reinterpret_cast<const float4*>(cs) + u;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float4 v = p[k * units];
        const uint64_t c = pack(v.x, v.y), s = pack(v.z, v.w), ns = pack(-v.z, -v.w);
        if (rp.interleaved) {
            float(&w)[8] = k < 2 ? a : b;
            const int e = 4 * (k & 1);
            const uint64_t x = pack(w[e], w[e + 2]), y = pack(w[e + 1], w[e + 3]);
            unpack(fma2(x, c, mul2(y, ns)), w[e], w[e + 2]);
            unpack(fma2(x, s, mul2(y, c)), w[e + 1], w[e + 3]);
        } else {
            const uint64_t x = pack(a[2 * k], a[2 * k + 1]), y = pack(b[2 * k], b[2 * k + 1]);
            unpack(fma2(x, c, mul2(y, ns)), a[2 * k], a[2 * k + 1]);
            unpack(fma2(x, s, mul2(y, c)), b[2 * k], b[2 * k + 1]);
        }
    }
}

// ------------------------------------------------------------------------- rotation

// Each unit is read once, turned in fp32 and written once; HBM bounds it.  The vectors of a
// thread are loaded together before the angles are computed, and a head's cosines come from
// shared memory instead of every thread's own.  16,384 x 32 x 128 bf16, all turned: 41 us
// (6.6 TB/s), 64 rows 2.3 us; four vectors in flight took 42 and 2.9 us, one 44 and 2.1 us,
// angles per thread (eight heads each) 52 us.
constexpr int kRopeBatch = 2;

template <typename T>
__global__ void __launch_bounds__(kThreads)
rope_kernel(const __grid_constant__ RopeParams rp, const __grid_constant__ RopeCall c,
            const __grid_constant__ Tiling t)
{
    __shared__ __align__(16) float sm_angles[2 * kAngles];
    pdl_wait_then_release();
    const int groups = t.groups, g = quotient(threadIdx.x, t.by_lanes);
    const int l = threadIdx.x - g * t.lanes;
    const int r0 = blockIdx.x * t.rows, h0 = blockIdx.y * t.heads;
    const int rows = min(t.rows, c.rows - r0), heads = min(t.heads, c.heads - h0);
    const Unit u = unit_of(rp, l, c.D);
    const bool mine = g < groups && (u.rotated || c.x != c.out);
    const T* x = static_cast<const T*>(c.x) + r0 * c.x_row + h0 * c.x_head;
    T* out = static_cast<T*>(c.out) + r0 * c.out_row + h0 * c.out_head;
    constexpr int kB = kRopeBatch;
    Eight<T> wa[kB], wb[kB];
    int row[kB], head[kB];
#pragma unroll
    for (int j = 0; j < kB; ++j) {
        const uint32_t q = j * groups + g;
        row[j] = quotient(q, t.by_heads);
        head[j] = q - row[j] * t.heads;
        if (!mine || row[j] >= rows || head[j] >= heads) {
            row[j] = -1;
            continue;
        }
        const T* p = x + row[j] * c.x_row + head[j] * c.x_head;
        wa[j].load(p + u.a);
        if (u.b >= 0)
            wb[j].load(p + u.b);
    }
    block_angles(rp, t, c.positions + r0, rows, sm_angles);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kB; ++j) {
        if (row[j] < 0)
            continue;
        float a[8], b[8];
        wa[j].values(a);
        wb[j].values(b);
        if (u.rotated)
            rotate16(rp, sm_angles + row[j] * rp.rot, l, a, b);
        T* p = out + row[j] * c.out_row + head[j] * c.out_head;
        store8(p + u.a, a);
        if (u.b >= 0)
            store8(p + u.b, b);
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
            const float2 cs = turn(rp, c.positions[t], rp.inc[e]);
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

// The largest of four groups.
__device__ __forceinline__ float largest4(const float* groups)
{
    const float4 g = *reinterpret_cast<const float4*>(groups);
    return fmaxf(fmaxf(g.x, g.y), fmaxf(g.z, g.w));
}

__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8], float inv)
{
    uint32_t r = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        r |= static_cast<uint32_t>(
                 __nv_cvt_float2_to_fp4x2(make_float2(v[2 * j] * inv, v[2 * j + 1] * inv),
                                          __NV_E2M1, cudaRoundNearest) &
                 0xFFu)
             << (8 * j);
    return r;
}

// Biased exponent floor(log2(amax)) - 2 of an e2m1 block, clamped to ue8m0's 0..254; 127
// for a zero block.  A subnormal amax has an exponent below the clamp anyway.
__device__ __forceinline__ uint32_t e2m1_exponent(float amax)
{
    if (!(amax > 0.0f))
        return 127u;
    const int e = min(static_cast<int>(__float_as_uint(amax) >> 23), 254) - 2;
    return static_cast<uint32_t>(max(e, 0));
}

// 2^(127 - e) for a biased exponent e in 0..252 (the exponents e2m1_exponent returns).
__device__ __forceinline__ float exp2_neg(uint32_t e) { return __uint_as_float((254u - e) << 23); }

// The same tiling, `lanes` a power of two; a group takes its vectors one after another, the next
// one's loads under way.  The largest magnitude of a vector (e4m3) by a shuffle reduction over
// its lanes.  An e2m1 scale covers 32 neighbours, four groups of eight that any lanes may hold:
// the groups' maxima meet in shared memory, the values stay where they are (exchanging the values
// took 2.4 times as long).
//
// Instructions bound it, not bytes (some 290 per warp and 512 elements: widening, turning, maxima,
// quotients, narrowing; without rotation and quotients it runs at 5.9 TB/s).  16,384 x 32 x
// 128 bf16 with 64 turned: e4m3 45 us, e2m1 42 us (4.5 and 4.0 TB/s).  Blocks of 64 registers,
// four an SM: at 40 and six the loop took 52 and 58 us, and without it, a vector a group, whose
// set-up is a third of its instructions, it was 50 and 53 us at best.
template <typename T, bool kFp4>
__global__ void __launch_bounds__(kThreads, 4)
cache_write_kernel(const __grid_constant__ RopeParams rp,
                   const __grid_constant__ CacheWriteCall c, const __grid_constant__ Tiling t)
{
    __shared__ __align__(16) float sm_angles[2 * kAngles];
    __shared__ __align__(16) float sm_groups[kFp4 ? kThreads * 2 : 1];   // maxima of eight
    pdl_wait_then_release();
    const int g = quotient(threadIdx.x, t.by_lanes);
    const int l = threadIdx.x - g * t.lanes;
    const int r0 = blockIdx.x * t.rows, h0 = blockIdx.y * t.heads;
    const int rows = min(t.rows, c.rows - r0), heads = min(t.heads, c.heads - h0);
    const Unit u = unit_of(rp, l, c.D);
    const bool unit = l < c.D / 16;
    const T* x = static_cast<const T*>(c.x) + r0 * c.x_row + h0 * c.x_head;
    Eight<T> wa, wb;
    int row = quotient(g, t.by_heads), head = g - row * t.heads, slot = -1;
    auto load = [&] {
        slot = -1;
        if (row < rows && head < heads) {
            slot = c.slots ? c.slots[r0 + row] : r0 + row;
            if (unit) {
                const T* p = x + row * c.x_row + head * c.x_head;
                wa.load(p + u.a);
                wb.load(p + u.b);
            }
        }
    };
    load();
    if (rp.rot > 0) {
        block_angles(rp, t, c.positions + r0, rows, sm_angles);
        __syncthreads();
    }
    float* maxima = sm_groups + (kFp4 ? (threadIdx.x - l) * 2 : 0);
    const int row_step = quotient(t.groups, t.by_heads), head_step = t.groups - row_step * t.heads;
#pragma unroll 1
    for (int j = 0;;) {
        // a skipped row's lanes stay in the shuffles of the warp's other rows
        const bool on = unit && slot >= 0 && slot < c.num_slots;
        const int64_t vec = (int64_t)slot * c.heads + h0 + head;
        const int angles = row * rp.rot;
        float a[8] = {}, b[8] = {}, ma = 0.0f, mb = 0.0f;
        if (on) {
            wa.values(a);
            wb.values(b);
        }
        if (++j < t.batch) {
            row += row_step;
            head += head_step;
            if (head >= t.heads) {
                head -= t.heads;
                ++row;
            }
            load();
        }
        if (on) {
            if (u.rotated)
                rotate16(rp, sm_angles + angles, l, a, b);
            ma = largest(a);
            mb = largest(b);
        }
        if (kFp4) {
            if (on) {
                maxima[u.a / 8] = ma;
                maxima[u.b / 8] = mb;
            }
            __syncwarp();
            if (on) {
                const uint32_t ea = e2m1_exponent(largest4(maxima + u.a / 32 * 4));
                const uint32_t eb = e2m1_exponent(largest4(maxima + u.b / 32 * 4));
                uint8_t* o = c.codes + vec * (c.D / 2);
                *reinterpret_cast<uint32_t*>(o + u.a / 2) = e2m1x8(a, exp2_neg(ea));
                *reinterpret_cast<uint32_t*>(o + u.b / 2) = e2m1x8(b, exp2_neg(eb));
                uint8_t* sc = static_cast<uint8_t*>(c.scales) + vec * (c.D / 32);
                if (u.a % 32 == 0)
                    sc[u.a / 32] = static_cast<uint8_t>(ea);
                if (u.b % 32 == 0)
                    sc[u.b / 32] = static_cast<uint8_t>(eb);
            }
            __syncwarp();
        } else {
            float m = fmaxf(ma, mb);
            for (int d = t.lanes / 2; d > 0; d >>= 1)
                m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
            if (on) {
                const float s = e4m3_scale(m);
                const float inv = 1.0f / s;
                uint8_t* o = c.codes + vec * c.D;
                if (m == INFINITY) {
                    finite8(a);
                    finite8(b);
                }
                *reinterpret_cast<uint2*>(o + u.a) = e4m3x8(a, s, inv);
                *reinterpret_cast<uint2*>(o + u.b) = e4m3x8(b, s, inv);
                if (l == 0)
                    static_cast<float*>(c.scales)[vec] = s;
            }
        }
        if (j >= t.batch)
            break;
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
            const float2 cs = turn(rp, c.positions[t], rp.inc[p]);
            const float xa = v[a], xb = v[b];
            v[a] = fmaf(xa, cs.x, -xb * cs.y);
            v[b] = fmaf(xa, cs.y, xb * cs.x);
        }
        __syncwarp();
        for (int e = l; e < c.D; e += 32)
            v[e] = v[e] == v[e] ? v[e] : 0.0f;
        __syncwarp();
        const int64_t vec = (int64_t)slot * c.heads + h;
        float m = 0.0f;
        if (kFp4) {
            // lane l: the 32 elements of block l
            const int b = l < c.D / 32 ? l : 0;
            for (int e = 0; e < 32; ++e)
                m = fmaxf(m, fabsf(v[32 * b + e]));
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
                m = fmaxf(m, fabsf(v[e]));
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
                finite8(w);
                *reinterpret_cast<uint2*>(c.codes + vec * c.D + 8 * l) = e4m3x8(w, s, inv);
            }
        }
        __syncwarp();
    }
}

// ---------------------------------------------------------------------- cache append

// Slot of a row's new key: through the request's page table, at its place among the packed keys,
// or as given.  -1 where there is none.
__device__ __forceinline__ int32_t append_slot(const AppendCall& c, int t)
{
    int64_t slot;
    if (c.slots) {
        slot = c.slots[t];
    } else {
        int lo = 0, hi = c.num_requests - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (c.row_begin[mid] <= t)
                lo = mid;
            else
                hi = mid - 1;
        }
        const int32_t j = c.positions[t], base = c.key_begin[lo];
        if (j < 0 || j >= c.key_begin[lo + 1] - base)
            return -1;
        if (c.page > 0) {
            const int32_t pg = c.table[lo * c.ld_table + j / c.page];
            slot = pg < 0 ? -1 : (int64_t)pg * c.page + j % c.page;
        } else {
            slot = base + j;
        }
    }
    return slot >= 0 && slot < c.num_slots ? static_cast<int32_t>(slot) : -1;
}

// Keys (blocks of z = 0, turned) and values (z = 1, as they are) of the same rows, in one launch:
// the rotation's tiling, or for e4m3 the cache writes'.  The first vectors' loads are under way
// while the block's threads look up its rows' slots (position, page, slot: two reads one after the
// other) and compute its angles; a group then takes a few vectors, the next one's loads under
// way.  16,384 rows of 4 heads of 128 to e4m3: 16 us over one cache after another (14 over the same one, which
// the L2 holds; 10 to bf16), instructions as for the cache writes (0.7 of the issue slots); batches that
// leave two to twelve blocks an SM take as long, 24 took 20.  64 rows of 8 heads: 9 us, the call on the
// host.
template <typename T, typename C>
__global__ void __launch_bounds__(kThreads, 4)
append_kernel(const __grid_constant__ RopeParams rp, const __grid_constant__ AppendCall c,
              const __grid_constant__ Tiling t)
{
    constexpr bool kFp8 = sizeof(C) == 1;
    __shared__ __align__(16) float sm_angles[2 * kAngles];
    __shared__ int32_t sm_slots[kAppendRows];
    pdl_wait_then_release();
    const bool is_v = blockIdx.z != 0;
    const int rot = is_v ? 0 : rp.rot;
    const int g = quotient(threadIdx.x, t.by_lanes);
    const int l = threadIdx.x - g * t.lanes;
    const int r0 = blockIdx.x * t.rows, h0 = blockIdx.y * t.heads;
    const int rows = min(t.rows, c.rows - r0), heads = min(t.heads, c.heads - h0);
    const Unit u = unit_of(rot, is_v ? 0 : rp.offset, rp.interleaved, l, c.D);
    const bool unit = g < t.groups && l < rot / 16 + (c.D - rot + 15) / 16;
    const int64_t x_row = is_v ? c.v_row : c.k_row, x_head = is_v ? c.v_head : c.k_head;
    const T* x = static_cast<const T*>(is_v ? c.v : c.k) + r0 * x_row + h0 * x_head;
    C* cache = static_cast<C*>(is_v ? c.v_cache : c.k_cache);
    float* scales = is_v ? c.v_scale : c.k_scale;
    const int64_t to_slot = is_v ? c.vc_slot : c.kc_slot, to_head = is_v ? c.vc_head : c.kc_head;
    Eight<T> wa, wb;
    int row = quotient(g, t.by_heads), head = g - row * t.heads;
    bool here = false;
    auto load = [&] {
        here = unit && row < rows && head < heads;
        if (here) {
            const T* p = x + row * x_row + head * x_head;
            wa.load(p + u.a);
            if (u.b >= 0)
                wb.load(p + u.b);
        }
    };
    load();
    for (int i = threadIdx.x; i < rows; i += kThreads)
        sm_slots[i] = append_slot(c, r0 + i);
    if (rot > 0)
        block_angles(rp, t, c.positions + r0, rows, sm_angles);
    __syncthreads();
    const int row_step = quotient(t.groups, t.by_heads), head_step = t.groups - row_step * t.heads;
#pragma unroll 1
    for (int j = 0;;) {
        const int32_t slot = here ? sm_slots[row] : -1;
        const bool on = slot >= 0;
        const int h = h0 + head, angles = row * rot;
        float a[8] = {}, b[8] = {};
        if (on) {
            wa.values(a);
            if (u.b >= 0)
                wb.values(b);
        }
        if (++j < t.batch) {
            row += row_step;
            head += head_step;
            if (head >= t.heads) {
                head -= t.heads;
                ++row;
            }
            load();
        }
        if (on && u.rotated)
            rotate16(rp, sm_angles + angles, l, a, b);
        if constexpr (kFp8) {
            // (a skipped row's lanes stay in the shuffles of the warp's other rows)
            float m = 0.0f;
            if (on)
                m = fmaxf(largest(a), largest(b));
            for (int d = t.lanes / 2; d > 0; d >>= 1)
                m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
            if (on) {
                const float s = e4m3_scale(m);
                const float inv = 1.0f / s;
                if (m == INFINITY) {
                    finite8(a);
                    finite8(b);
                }
                uint8_t* o = reinterpret_cast<uint8_t*>(cache) + slot * to_slot + h * to_head;
                *reinterpret_cast<uint2*>(o + u.a) = e4m3x8(a, s, inv);
                *reinterpret_cast<uint2*>(o + u.b) = e4m3x8(b, s, inv);
                if (l == 0)
                    scales[(int64_t)slot * c.heads + h] = s;
            }
        } else if (on) {
            C* o = cache + slot * to_slot + h * to_head;
            store8(o + u.a, a);
            if (u.b >= 0)
                store8(o + u.b, b);
        }
        if (j >= t.batch)
            break;
    }
}

// Any rotation, size and alignment: one warp per (row, head, keys or values).
template <typename T, typename C>
__global__ void __launch_bounds__(kThreads)
append_any_kernel(const __grid_constant__ RopeParams rp, const __grid_constant__ AppendCall c)
{
    __shared__ float sm[kThreads / 32][kMaxHeadDim];
    pdl_wait_then_release();
    float* v = sm[threadIdx.x / 32];
    const int l = threadIdx.x & 31;
    const int64_t n = 2 * (int64_t)c.rows * c.heads;
    for (int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; i < n;
         i += (int64_t)gridDim.x * (kThreads / 32)) {
        const bool is_v = i & 1;
        const int t = static_cast<int>((i >> 1) / c.heads), h = static_cast<int>((i >> 1) % c.heads);
        const int32_t slot = append_slot(c, t);
        if (slot < 0)
            continue;
        const T* x = is_v ? static_cast<const T*>(c.v) + t * c.v_row + h * c.v_head
                          : static_cast<const T*>(c.k) + t * c.k_row + h * c.k_head;
        for (int e = l; e < c.D; e += 32)
            v[e] = Elt<T>::load(x[e]);
        __syncwarp();
        for (int p = l; p < (is_v ? 0 : rp.rot / 2); p += 32) {
            const int a = rp.offset + (rp.interleaved ? 2 * p : p);
            const int b = rp.interleaved ? a + 1 : a + rp.rot / 2;
            const float2 cs = turn(rp, c.positions[t], rp.inc[p]);
            const float xa = v[a], xb = v[b];
            v[a] = fmaf(xa, cs.x, -xb * cs.y);
            v[b] = fmaf(xa, cs.y, xb * cs.x);
        }
        __syncwarp();
        C* o = is_v ? static_cast<C*>(c.v_cache) + slot * c.vc_slot + h * c.vc_head
                    : static_cast<C*>(c.k_cache) + slot * c.kc_slot + h * c.kc_head;
        if constexpr (sizeof(C) == 1) {
            float m = 0.0f;
            for (int e = l; e < c.D; e += 32) {
                v[e] = v[e] == v[e] ? v[e] : 0.0f;
                m = fmaxf(m, fabsf(v[e]));
            }
            for (int d = 16; d > 0; d >>= 1)
                m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
            __syncwarp();
            const float s = e4m3_scale(m);
            const float inv = 1.0f / s;
            if (l == 0)
                (is_v ? c.v_scale : c.k_scale)[(int64_t)slot * c.heads + h] = s;
            if (l < c.D / 8) {
                float w[8];
                for (int k = 0; k < 8; ++k)
                    w[k] = v[8 * l + k];
                finite8(w);
                *reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(o) + 8 * l) = e4m3x8(w, s, inv);
            }
        } else {
            for (int e = l; e < c.D; e += 32)
                o[e] = Elt<C>::store(v[e]);
        }
        __syncwarp();
    }
}

// ------------------------------------------------------------------------ read back

// The values of eight e4m3 or e2m1 codes.
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

// A thread takes eight codes (whose values a 16-bit type stores with one instruction, a warp's
// side by side) of each of four stretches, all loads under way before the first store; HBM
// bounds it.  524,288 rows of 128 to bf16: e4m3 33 us (6.1 TB/s), e2m1 34 us; two stretches 35 and
// 34 us, eight 34 and 38, one 43 and 40; one thread per 16 bytes of codes 35 and 38.
constexpr int kReadBatch = 4;

template <typename T, bool kFp4>
__global__ void __launch_bounds__(kThreads)
cache_read_kernel(const __grid_constant__ CacheReadCall c, int chunks)
{
    pdl_wait_then_release();
    using Codes = typename std::conditional<kFp4, uint32_t, uint2>::type;
    const int64_t n = (int64_t)c.rows * chunks;
    const int per_vec = c.D / 8;
    for (int64_t i0 = (int64_t)blockIdx.x * kThreads * kReadBatch + threadIdx.x; i0 < n;
         i0 += (int64_t)gridDim.x * kThreads * kReadBatch) {
        int32_t slot[kReadBatch];
        int k[kReadBatch];
        Codes w[kReadBatch];
        float s[kReadBatch];
#pragma unroll
        for (int j = 0; j < kReadBatch; ++j) {
            const int64_t i = i0 + j * kThreads;
            slot[j] = -1;
            if (i < n) {
                int64_t t;
                if (n <= UINT32_MAX) {
                    t = static_cast<uint32_t>(i) / static_cast<uint32_t>(chunks);
                    k[j] = static_cast<uint32_t>(i) - static_cast<uint32_t>(t) * chunks;
                } else {
                    t = i / chunks;
                    k[j] = static_cast<int>(i - t * chunks);
                }
                slot[j] = c.slots ? c.slots[t] : static_cast<int32_t>(t);
            }
        }
#pragma unroll
        for (int j = 0; j < kReadBatch; ++j) {
            if (slot[j] < 0 || slot[j] >= c.num_slots) {
                w[j] = Codes{};
                s[j] = 1.0f;
                continue;
            }
            const int64_t at = (int64_t)slot[j] * chunks + k[j];
            w[j] = __ldg(reinterpret_cast<const Codes*>(c.codes) + at);
            if constexpr (kFp4)
                s[j] = ldexpf(
                    1.0f, static_cast<int>(__ldg(static_cast<const uint8_t*>(c.scales) + at / 4)) -
                              127);
            else
                s[j] = __ldg(static_cast<const float*>(c.scales) + (int64_t)slot[j] * c.heads +
                             k[j] / per_vec);
        }
#pragma unroll
        for (int j = 0; j < kReadBatch; ++j) {
            const int64_t i = i0 + j * kThreads;
            if (i >= n)
                break;
            float v[8];
            if constexpr (kFp4)
                e2m1_values(w[j], v);
            else
                e4m3_values(w[j], v);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] *= s[j];
            store8(static_cast<T*>(c.out) + i * 8, v);
        }
    }
}

// Codes and scales as they are.  A row outside the cache reads as zero codes of scale 1.  16 bytes of
// codes a thread, one read at a time: 152,048 rows of 128 in e4m3 10.4 us (3.9 TB/s read and
// written), e2m1 4.7 us (4.5); 524,288 rows 36 us (3.9) and 13.3 us (5.5).  Its division per 16 bytes and
// the read's latency bound it, not HBM.
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

// A key a thread, its request by a search of the batch's key offsets: 152,048 keys 1.7 us, 524,288
// of two requests 2.7 us, little above a launch.
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

// The tiling of a call.
Tiling tiling(const RopeParams& rp, int rows, int heads, int lanes, int batch)
{
    Tiling t = {};
    t.lanes = lanes;
    t.groups = kThreads / lanes;
    t.heads = std::min(heads, t.groups * batch);
    t.rows = std::min(rows, t.groups * batch / t.heads);
    t.by_lanes = reciprocal(lanes);
    if (rp.rot > 0) {
        t.rows = std::min(t.rows, kAngles / (rp.rot / 2));
        t.angle_rows = kThreads / (rp.rot / 2);
        t.by_pairs = reciprocal(rp.rot / 2);
    }
    t.batch = (t.rows * t.heads + t.groups - 1) / t.groups;
    t.by_heads = reciprocal(t.heads);
    return t;
}

dim3 tiles(const Tiling& t, int rows, int heads)
{
    return dim3(static_cast<unsigned>((rows + t.rows - 1) / t.rows),
                static_cast<unsigned>((heads + t.heads - 1) / t.heads));
}

template <typename T>
cudaError_t rope_of(const RopeParams& rp, const RopeCall& c, cudaStream_t st)
{
    if (whole_units(rp) && c.D % 8 == 0 && vector_rows(c.x, c.x_row, c.x_head, c.dtype) &&
        vector_rows(c.out, c.out_row, c.out_head, c.dtype)) {
        const int units = rp.rot / 16 + (c.D - rp.rot + 15) / 16;
        const Tiling t = tiling(rp, c.rows, c.heads, units, kRopeBatch);
        return launch_pdl(rope_kernel<T>, tiles(t, c.rows, c.heads), dim3(kThreads), 0, st, rp, c,
                          t);
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
        // Several vectors a group, up to eight, where that leaves six blocks an SM (rows of 32
        // heads to e4m3, a product for the quotient: 16,384 rows 42 us in eights, 61 one by one; 4,096 rows 12.6 in fours,
        // 13.6 in eights, 15.7 one by one; 1,024 rows 5.0 one by one, 6.3 in threes).
        const int64_t blocks = ((int64_t)c.rows * c.heads * lanes + kThreads - 1) / kThreads;
        const int batch = static_cast<int>(
            std::max<int64_t>(1, std::min<int64_t>(8, blocks / (6 * device_sms()))));
        const Tiling t = tiling(rp, c.rows, c.heads, lanes, batch);
        return launch_pdl(cache_write_kernel<T, kFp4>, tiles(t, c.rows, c.heads), dim3(kThreads), 0,
                          st, rp, c, t);
    }
    const int64_t n = (int64_t)c.rows * c.heads;
    const unsigned blocks = static_cast<unsigned>(
        std::min<int64_t>((n + kThreads / 32 - 1) / (kThreads / 32), 152 * 16));
    return launch_pdl(cache_write_any_kernel<T, kFp4>, dim3(blocks), dim3(kThreads), 0, st, rp, c);
}

template <typename T, typename C>
cudaError_t append_of(const RopeParams& rp, const AppendCall& c, cudaStream_t st)
{
    constexpr bool kFp8 = sizeof(C) == 1;
    const bool whole =
        whole_units(rp) && c.D % 8 == 0 && vector_rows(c.k, c.k_row, c.k_head, c.dtype) &&
        vector_rows(c.v, c.v_row, c.v_head, c.dtype) &&
        (kFp8 || (vector_rows(c.k_cache, c.kc_slot, c.kc_head, IDX_BF16) &&
                  vector_rows(c.v_cache, c.vc_slot, c.vc_head, IDX_BF16)));
    if (whole) {
        // threads of a vector: for the maximum over it (e4m3) a power of two (rot_dim is a multiple
        // of 16, so turned keys take as many units as values)
        int lanes = kFp8 ? 2 : std::max(2, (c.D + 15) / 16);
        while (kFp8 && lanes * 16 < c.D)
            lanes *= 2;
        const int64_t blocks = (2 * (int64_t)c.rows * c.heads * lanes + kThreads - 1) / kThreads;
        const int batch = static_cast<int>(
            std::max<int64_t>(1, std::min<int64_t>(8, blocks / (6 * device_sms()))));
        const Tiling t = tiling(rp, c.rows, c.heads, lanes, batch);
        dim3 grid = tiles(t, c.rows, c.heads);
        grid.z = 2;
        return launch_pdl(append_kernel<T, C>, grid, dim3(kThreads), 0, st, rp, c, t);
    }
    const int64_t n = 2 * (int64_t)c.rows * c.heads;
    const unsigned blocks = static_cast<unsigned>(
        std::min<int64_t>((n + kThreads / 32 - 1) / (kThreads / 32), 152 * 16));
    return launch_pdl(append_any_kernel<T, C>, dim3(blocks), dim3(kThreads), 0, st, rp, c);
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

cudaError_t launch_append(const RopeParams& rp, const AppendCall& c, cudaStream_t st)
{
    if (c.rows <= 0)
        return cudaSuccess;
    if (c.cache_dtype == IDX_CODES)
        return c.dtype == IDX_BF16   ? append_of<__nv_bfloat16, uint8_t>(rp, c, st)
               : c.dtype == IDX_FP16 ? append_of<__half, uint8_t>(rp, c, st)
                                     : append_of<float, uint8_t>(rp, c, st);
    if (c.dtype == IDX_FP32)
        return c.cache_dtype == IDX_BF16 ? append_of<float, __nv_bfloat16>(rp, c, st)
                                         : append_of<float, __half>(rp, c, st);
    return c.dtype == IDX_BF16 ? append_of<__nv_bfloat16, __nv_bfloat16>(rp, c, st)
                               : append_of<__half, __half>(rp, c, st);
}

cudaError_t launch_cache_read(const CacheReadCall& c, cudaStream_t st)
{
    if (c.rows <= 0)
        return cudaSuccess;
    const dim3 block(kThreads);
    if (c.out_dtype == IDX_CODES) {
        const int whole = c.heads * (c.fp4 ? c.D / 32 : c.D / 16);   // 16 bytes each
        return launch_pdl(cache_copy_kernel, dim3(stride_blocks((int64_t)c.rows * whole)), block, 0,
                          st, c, whole);
    }
    const int chunks = c.heads * (c.D / 8);
    const dim3 grid(stride_blocks(((int64_t)c.rows * chunks + kReadBatch - 1) / kReadBatch));
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
