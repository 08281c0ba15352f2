// Host side of the operators around the indexer: rotary positions, quantised caches and
// attention over the selected keys.  Argument checks, launches; no device memory is
// allocated and nothing synchronizes.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <new>

#include "indexer.h"
#include "internal.h"

using namespace idx;

struct indexer_rope_s {
    int32_t D = 0;
    RopeParams p;
};

struct indexer_attention_s {
    indexer_attention_spec spec;
    AttnParams p;                // everything but the operands of a call
    size_t part_floats = 0;      // partial vectors
    size_t ws_bytes = 0;
};

struct indexer_causal_s {
    indexer_causal_spec spec;
    CausalParams p;              // everything but the operands of a call
    AttnParams rows;             // the same for rows one by one
    bool by_rows = false;        // which of the two
    int64_t max_pages = 0;       // of the longest request
    size_t part_floats = 0;      // partial vectors
    size_t ws_bytes = 0;
};

namespace {

constexpr int kPlanSms = 152;    // SMs the splits are planned for
constexpr int kClusterBlocks = 144;   // blocks in clusters of 4 that run at once

bool is_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool dense_type(int dtype) { return dtype == IDX_BF16 || dtype == IDX_FP16 || dtype == IDX_FP32; }

size_t type_bytes(int dtype) { return dtype == IDX_FP32 ? 4 : 2; }

int finish(cudaError_t e) { return e == cudaSuccess ? IDX_OK : IDX_ERR_CUDA; }

// A frequency in radians per position as the phase a position adds, in 2^-64 turns, modulo one
// turn.  1 / 2 pi is two doubles and their product with the frequency too, so that the phase of
// position 2^31 has the frequency's own rounding (2^-53 of it, 1.2e-7 rad at one radian a position)
// and no other.
uint64_t phase_increment(double radians)
{
    constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;
    const double turns = radians * kHi;
    const double rest = std::fma(radians, kHi, -turns) + radians * kLo;
    return static_cast<uint64_t>(std::ldexp(turns - std::floor(turns), 64)) +
           static_cast<uint64_t>(static_cast<int64_t>(std::nearbyint(std::ldexp(rest, 64))));
}

// Where a call's items do not fill the SMs, the tiles of a row are split.  Two or four splits
// that all run at once are a cluster, which joins them through its shared memory; more are
// joined from the workspace by a kernel of its own.  The number that ends first by measured
// times: 0.65 us a tile, 2 an item, 1.4 for a cluster's join, 1.1 for the kernel's, 0.15 for each
// part of a row and the parts' bytes at 4 TB/s.  Fitted to 231 calls (16, 32 and 64 heads of 128, 8
// and 32 of 64, one or four to a cached head, 16-bit and e4m3 caches, both query types; 1 to 200
// rows of 4 to 64 tiles), each timed whole, in 2 to 64 parts and in clusters of 2 and 4: the chosen
// number takes 0.5 % longer than the best on average, 12 % at most.  (One row of 64 tiles, 32 heads
// of 128: 47 us whole, 17.5 in 4, 12.3 in 16, which are chosen, 16.9 in 64.  64 rows of 16 tiles of
// e4m3: 13.9 in a cluster of 2, 18.8 whole.)  A cluster of 8 does not run on all SMs at once
// (16 rows 17.5 us against 10.4 in four).
double row_splits(AttnParams& p, int64_t items, int64_t tiles, int D, int nh)
{
    double best = INFINITY;
    for (int64_t n = 1; n <= std::min<int64_t>(tiles, kMaxSplits) && items * n <= (1 << 30); ++n) {
        const int64_t per = (tiles + n - 1) / n;
        if ((tiles + per - 1) / per != n)
            continue;
        const double waves = static_cast<double>((items * n + kPlanSms - 1) / kPlanSms);
        const bool cluster = (n == 2 || n == kMaxCluster) && items * n <= kClusterBlocks;
        const double bytes = 4.0 * D * nh * (items * n);
        const double join = n == 1 ? 0.0 : cluster ? 1.4 : 1.1 + 0.15 * n + 1e-6 / 4 * bytes;
        const double cost = waves * (0.65 * per + 2.0) + join;
        if (cost < best) {
            best = cost;
            p.cluster = cluster;
            p.splits = static_cast<int32_t>(n);
            p.split_tiles = static_cast<int32_t>(per);
        }
    }
    return best;
}

// The tiled form of causal attention: what each block takes, and its time in microseconds.  An item
// costs its key tiles and as much as kItemTiles of them for its queries and outputs; every block gets
// an equal run of that, cut where it ends inside an item, or else at the nearest item's end.  (16 rows over
// 32,768 keys, 4 x 8 heads of 128: 25 us on 152 blocks, 84 row by row; 2,048 keys 12.9 on 64 blocks.)
double causal_cuts(CausalParams& p)
{
    constexpr double kItemTiles = 2.0, kTileUs = 2.0, kJoinUs = 5.0, kPartUs = 0.04;
    int64_t row_tiles = 0;
    for (int r = 0; r < p.num_requests; ++r) {
        p.tile_begin[r] = static_cast<int32_t>(row_tiles);
        const int64_t rows = (int64_t)(p.row_begin[r + 1] - p.row_begin[r]) * p.group;
        p.most_rows = static_cast<int32_t>(
            std::max<int64_t>(p.most_rows, std::min<int64_t>(rows, kCausalRows)));
        row_tiles += (rows + kCausalRows - 1) / kCausalRows;
    }
    p.tile_begin[p.num_requests] = static_cast<int32_t>(row_tiles);
    const int64_t items = row_tiles * p.Hkv;
    if (items > (1 << 26))
        return INFINITY;
    // Every item's tiles: the same for all heads of a row tile.
    const auto walk = [&](auto visit) {
        for (int r = 0; r < p.num_requests; ++r) {
            const int tokens = p.row_begin[r + 1] - p.row_begin[r];
            const int keys = p.key_begin[r + 1] - p.key_begin[r];
            for (int d = p.tile_begin[r]; d < p.tile_begin[r + 1]; ++d) {
                const int i0 = (d - p.tile_begin[r]) * kCausalRows;
                const int i1 = std::min(i0 + kCausalRows, tokens * p.group) - 1;
                visit(d, causal_tiles(keys, tokens, i0 / p.group, i1 / p.group, p.window, p.sinks));
            }
        }
    };
    double total = 0.0;
    int64_t tiles = 0;
    walk([&](int, int n) {
        total += p.Hkv * (n + kItemTiles);
        tiles += (int64_t)p.Hkv * n;
    });
    double best = INFINITY;
    // Whole items, or at least four tiles a block, two or one.
    for (int cut = 0; cut < 8; cut = cut ? 2 * cut : 1) {
        CausalParams c = p;
        c.blocks = static_cast<int32_t>(std::min<int64_t>(
            kCausalBlocks,
            cut ? std::max<int64_t>(1, cut * tiles / 4) : std::max<int64_t>(1, items)));
        const double share = total / c.blocks;
        c.joined = 0;
        c.cut_item[0] = c.cut_tile[0] = 0;
        int b = 1;
        double done = 0.0, longest = 0.0, begun = 0.0;
        walk([&](int d, int n) {
            for (int g = 0; g < p.Hkv; ++g) {
                const int item = d * p.Hkv + g;
                const double cost = n + kItemTiles;
                while (b < c.blocks && b * share < done + cost) {
                    const double in = b * share - done - kItemTiles;
                    int at = cut ? static_cast<int>(in + 0.5) : 0;
                    if (!cut && b * share - done >= cost / 2)
                        break;                               // (after it)
                    at = std::min(std::max(at, 0), n);
                    if (cut && c.cut_item[b - 1] == item)
                        at = std::max(at, c.cut_tile[b - 1] + 1);   // (no part is empty)
                    if (at >= n)
                        break;
                    c.cut_item[b] = item;
                    c.cut_tile[b] = at;
                    if (at > 0 && (c.joined == 0 || c.cut_item[c.first_cut[c.joined - 1]] != item))
                        c.first_cut[c.joined++] = b;
                    const double here = done + (at > 0 ? at + kItemTiles : 0.0);
                    longest = std::max(longest, here - begun);
                    begun = done + (at > 0 ? at : 0.0);
                    ++b;
                }
                done += cost;
            }
        });
        longest = std::max(longest, done - begun);
        for (; b <= c.blocks; ++b) {
            c.cut_item[b] = static_cast<int32_t>(items);
            c.cut_tile[b] = 0;
        }
        const double parts = c.joined ? static_cast<double>(c.blocks) / c.joined : 0.0;
        const double time = longest * kTileUs + (c.joined ? kJoinUs + kPartUs * parts : 0.0);
        if (time < best) {
            best = time;
            p = c;
        }
    }
    return best;
}

// The form for rows one by one, and its time.
double causal_rows(AttnParams& q, const CausalParams& p, const indexer_causal_spec& s, bool fp8)
{
    std::memset(&q, 0, sizeof(q));
    q.scale_log2 = static_cast<float>(s.scale * 1.4426950408889634);
    q.rows = p.rows;
    q.Hq = p.Hq;
    q.Hkv = p.Hkv;
    q.group = p.group;
    q.num_slots = p.num_slots;
    q.page = p.page;
    q.by_page = p.by_page;
    q.window = p.window;
    q.sinks = p.sinks;
    q.num_requests = p.num_requests;
    std::copy(p.row_begin, p.row_begin + p.num_requests + 1, q.row_begin);
    std::copy(p.key_begin, p.key_begin + p.num_requests + 1, q.key_begin);
    const int nh = attention_heads_per_tile(p.group, s.dtype, fp8);
    q.head_tiles = (p.group + nh - 1) / nh;
    const int64_t items = (int64_t)p.rows * p.Hkv * q.head_tiles;
    int64_t most = 1;
    for (int r = 0; r < p.num_requests; ++r) {
        int64_t keys = p.key_begin[r + 1] - p.key_begin[r];
        if (p.window > 0)
            keys = std::min<int64_t>(keys, (int64_t)p.window + p.sinks);
        if (p.row_begin[r + 1] > p.row_begin[r])
            most = std::max(most, (keys + kAttnTile - 1) / kAttnTile);
    }
    if (items > (1 << 30))
        return INFINITY;
    const double cost = row_splits(q, items, most, s.D, nh);
    q.by_splits = divisor(q.splits);
    q.by_head_tiles = divisor(q.head_tiles);
    q.by_hkv = divisor(q.Hkv);
    return cost;
}

}  // namespace

extern "C" {

int indexer_rope_create(const indexer_rope_spec* s, indexer_rope_t* out)
{
    if (!out)
        return IDX_ERR_INVALID_ARG;
    *out = nullptr;
    if (!s || s->D < 2 || s->D > kMaxHeadDim || s->rot_dim < 2 || s->rot_dim % 2 != 0 ||
        s->rot_dim > s->D || s->rot_offset < 0 || s->rot_offset > s->D - s->rot_dim ||
        (s->layout != IDX_ROPE_HALF && s->layout != IDX_ROPE_INTERLEAVED) || !(s->base > 0.0) ||
        !std::isfinite(s->base) || !(s->factor >= 1.0) || !std::isfinite(s->factor) ||
        !std::isfinite(s->amplitude))
        return IDX_ERR_INVALID_ARG;
    if (s->factor > 1.0 && s->original_len > 0.0 &&
        (!std::isfinite(s->original_len) || !(s->beta_fast > 0.0) || !(s->beta_slow > 0.0) ||
         !(s->beta_fast >= s->beta_slow) || !std::isfinite(s->beta_fast) || !(s->base > 1.0)))
        return IDX_ERR_INVALID_ARG;
    indexer_rope_s* r = new (std::nothrow) indexer_rope_s();
    if (!r)
        return IDX_ERR_INVALID_ARG;
    std::memset(&r->p, 0, sizeof(r->p));
    r->D = s->D;
    r->p.rot = s->rot_dim;
    r->p.offset = s->rot_offset;
    r->p.interleaved = s->layout == IDX_ROPE_INTERLEAVED;
    r->p.amplitude = static_cast<float>(s->amplitude);
    double lo = 0.0, hi = 0.0;
    const bool parts = s->factor > 1.0 && s->original_len > 0.0;
    if (parts) {
        // the pair that makes n turns over the original length
        const auto pair_of = [&](double n) {
            return s->rot_dim * std::log(s->original_len / (n * 6.283185307179586)) /
                   (2.0 * std::log(s->base));
        };
        lo = std::max(std::floor(pair_of(s->beta_fast)), 0.0);
        hi = std::min(std::ceil(pair_of(s->beta_slow)), s->rot_dim - 1.0);
    }
    for (int i = 0; i < s->rot_dim / 2; ++i) {
        double f = std::pow(s->base, -2.0 * i / s->rot_dim);
        if (parts) {
            const double ramp = std::min(std::max((i - lo) / std::max(hi - lo, 0.001), 0.0), 1.0);
            f = f / s->factor * ramp + f * (1.0 - ramp);
        } else {
            f /= s->factor;
        }
        r->p.inc[i] = phase_increment(f);
    }
    *out = r;
    return IDX_OK;
}

void indexer_rope_destroy(indexer_rope_t rope) { delete rope; }

int indexer_rope(indexer_rope_t rope, const void* x, int32_t dtype, int32_t rows, int32_t heads,
                 int64_t row_stride, int64_t head_stride, const int32_t* positions,
                 int32_t inverse, void* out, int64_t out_row_stride, int64_t out_head_stride,
                 void* stream)
{
    if (!rope || !dense_type(dtype) || rows < 0 || heads < 1 || heads > IDX_MAX_HEADS ||
        row_stride < 0 || head_stride < 0 || out_row_stride < 0 || out_head_stride < 0 ||
        (inverse != 0 && inverse != 1))
        return IDX_ERR_INVALID_ARG;
    if (rows > 0 &&
        (!x || !out || !positions || !is_aligned(x, type_bytes(dtype)) ||
         !is_aligned(out, type_bytes(dtype)) || !is_aligned(positions, 4) ||
         (heads > 1 && out_head_stride < rope->D) || (rows > 1 && out_row_stride < rope->D) ||
         (x == out && ((rows > 1 && row_stride != out_row_stride) ||
                       (heads > 1 && head_stride != out_head_stride)))))
        return IDX_ERR_INVALID_ARG;
    if (!device_supported())
        return IDX_ERR_UNSUPPORTED;
    if (rows == 0)
        return IDX_OK;
    RopeParams rp = rope->p;
    rp.inverse = inverse;
    const RopeCall c{x,    out,  positions,   row_stride, head_stride, out_row_stride,
                     out_head_stride, rows, heads,       rope->D,    dtype};
    count_launch();
    return finish(launch_rope(rp, c, static_cast<cudaStream_t>(stream)));
}

static bool cache_format(int format, int heads, int D, int num_slots)
{
    return (format == IDX_K_FP8_E4M3 || format == IDX_K_FP4_E2M1_UE8M0) && heads >= 1 &&
           heads <= IDX_MAX_HEADS && D >= 32 && D <= kMaxHeadDim && D % 32 == 0 && num_slots >= 0;
}

int indexer_cache_write(indexer_rope_t rope, const void* x, int32_t dtype, int32_t rows,
                        int32_t heads, int32_t D, int64_t row_stride, int64_t head_stride,
                        const int32_t* positions, const int32_t* slots, int32_t num_slots,
                        int32_t format, void* codes, void* scales, void* stream)
{
    if (!dense_type(dtype) || !cache_format(format, heads, D, num_slots) || rows < 0 ||
        row_stride < 0 || head_stride < 0 || (rope && rope->D != D))
        return IDX_ERR_INVALID_ARG;
    if (rows > 0 && (!x || !codes || !scales || (rope && !positions) ||
                     !is_aligned(x, type_bytes(dtype)) || !is_aligned(codes, 16) ||
                     !is_aligned(scales, 4) || !is_aligned(positions, 4) ||
                     !is_aligned(slots, 4) || (!slots && rows > num_slots)))
        return IDX_ERR_INVALID_ARG;
    if (!device_supported())
        return IDX_ERR_UNSUPPORTED;
    if (rows == 0)
        return IDX_OK;
    RopeParams rp;
    if (rope)
        rp = rope->p;
    else
        std::memset(&rp, 0, sizeof(rp));
    const CacheWriteCall c{x,
                           positions,
                           slots,
                           static_cast<uint8_t*>(codes),
                           scales,
                           row_stride,
                           head_stride,
                           rows,
                           heads,
                           D,
                           dtype,
                           num_slots,
                           format == IDX_K_FP4_E2M1_UE8M0};
    count_launch();
    return finish(launch_cache_write(rp, c, static_cast<cudaStream_t>(stream)));
}

int indexer_cache_read(const void* codes, const void* scales, int32_t format, int32_t num_slots,
                       int32_t heads, int32_t D, const int32_t* slots, int32_t rows,
                       int32_t out_dtype, void* out, void* out_scales, void* stream)
{
    if (!cache_format(format, heads, D, num_slots) || rows < 0 ||
        !(dense_type(out_dtype) || out_dtype == IDX_CODES))
        return IDX_ERR_INVALID_ARG;
    if (rows > 0 && (!codes || !scales || !out || !is_aligned(codes, 16) ||
                     !is_aligned(scales, 4) || !is_aligned(out, 16) || !is_aligned(slots, 4) ||
                     (!slots && rows > num_slots) ||
                     (out_dtype == IDX_CODES && (!out_scales || !is_aligned(out_scales, 4)))))
        return IDX_ERR_INVALID_ARG;
    if (!device_supported())
        return IDX_ERR_UNSUPPORTED;
    if (rows == 0)
        return IDX_OK;
    const CacheReadCall c{static_cast<const uint8_t*>(codes),
                          scales,
                          slots,
                          out,
                          out_scales,
                          rows,
                          heads,
                          D,
                          num_slots,
                          format == IDX_K_FP4_E2M1_UE8M0,
                          out_dtype};
    count_launch();
    return finish(launch_cache_read(c, static_cast<cudaStream_t>(stream)));
}

int indexer_page_slots(indexer_plan_t p, const int32_t* page_table, int64_t ld_page_table,
                       int32_t page_size, int32_t* slots, void* stream)
{
    if (!p || page_size < 1)
        return IDX_ERR_INVALID_ARG;
    const PlanView v = plan_view(p);
    if (ld_page_table < (v.max_L + (int64_t)page_size - 1) / page_size)
        return IDX_ERR_INVALID_ARG;
    if (v.Lk > 0 && (!page_table || !slots || !is_aligned(page_table, 4) || !is_aligned(slots, 4)))
        return IDX_ERR_INVALID_ARG;
    if (!device_supported())
        return IDX_ERR_UNSUPPORTED;
    if (v.Lk == 0)
        return IDX_OK;
    PageSlotParams pp;
    std::memset(&pp, 0, sizeof(pp));
    pp.table = page_table;
    pp.ld_table = ld_page_table;
    pp.slots = slots;
    pp.page = page_size;
    pp.num_requests = v.R;
    std::copy(v.key_begin, v.key_begin + v.R + 1, pp.key_begin);
    count_launch();
    return finish(launch_page_slots(pp, static_cast<cudaStream_t>(stream)));
}

int indexer_attention_create(indexer_plan_t plan, const indexer_attention_spec* s,
                             indexer_attention_t* out, size_t* ws_bytes)
{
    if (!out)
        return IDX_ERR_INVALID_ARG;
    *out = nullptr;
    if (!plan || !s || s->Hkv < 1 || s->Hq < 1 || s->Hq > IDX_MAX_HEADS ||
        s->Hq % s->Hkv != 0 || s->block < 1 || s->block > 128 ||
        (s->block & (s->block - 1)) != 0 || s->num_sel < 1 || s->num_sel > 65536 ||
        (s->dtype != IDX_BF16 && s->dtype != IDX_FP16) ||
        (s->kv_format != IDX_KV_DENSE && s->kv_format != IDX_KV_FP8_E4M3) || s->num_slots < 0 ||
        s->page_size < 0 || !(std::fabs(s->scale) <= 1e38f) || s->D < 1)
        return IDX_ERR_INVALID_ARG;
    if (s->D != 64 && s->D != 128)
        return IDX_ERR_UNSUPPORTED;
    const PlanView v = plan_view(plan);
    if ((int64_t)v.T * s->Hq > INT32_MAX)
        return IDX_ERR_INVALID_ARG;
    indexer_attention_s* a = new (std::nothrow) indexer_attention_s();
    if (!a)
        return IDX_ERR_INVALID_ARG;
    a->spec = *s;
    AttnParams& p = a->p;
    std::memset(&p, 0, sizeof(p));
    p.scale_log2 = static_cast<float>(s->scale * 1.4426950408889634);
    p.rows = v.T;
    p.Hq = s->Hq;
    p.Hkv = s->Hkv;
    p.group = s->Hq / s->Hkv;
    while ((1 << p.block_shift) < s->block)
        ++p.block_shift;
    p.num_sel = s->num_sel;
    p.num_slots = s->num_slots;
    p.page = s->page_size;
    p.by_page = divisor(std::max(1, s->page_size));
    p.num_requests = v.R;
    std::copy(v.row_begin, v.row_begin + v.R + 1, p.row_begin);
    std::copy(v.key_begin, v.key_begin + v.R + 1, p.key_begin);
    // Work items: rows x key/value heads x tiles of query heads, each over the row's key tiles.
    const int nh = attention_heads_per_tile(p.group, s->dtype, s->kv_format != IDX_KV_DENSE);
    p.head_tiles = (p.group + nh - 1) / nh;
    const int64_t tiles = (((int64_t)s->num_sel << p.block_shift) + kAttnTile - 1) / kAttnTile;
    const int64_t items = (int64_t)v.T * s->Hkv * p.head_tiles;
    if (items > (1 << 30)) {
        delete a;
        return IDX_ERR_INVALID_ARG;
    }
    row_splits(p, items, tiles, s->D, nh);
    p.by_splits = divisor(p.splits);
    p.by_head_tiles = divisor(p.head_tiles);
    p.by_hkv = divisor(p.Hkv);
    // status word, then the parts of split rows
    a->part_floats = p.splits > 1 && !p.cluster ? (size_t)(items * p.splits) * nh : 0;
    a->ws_bytes = 256 + a->part_floats * (s->D + 2) * sizeof(float);
    *out = a;
    if (ws_bytes)
        *ws_bytes = a->ws_bytes;
    return IDX_OK;
}

void indexer_attention_destroy(indexer_attention_t a) { delete a; }

int indexer_sparse_attention(indexer_attention_t a, const indexer_attention_io* io, void* ws,
                             size_t ws_bytes, void* stream)
{
    if (!a || !io)
        return IDX_ERR_INVALID_ARG;
    const indexer_attention_spec& s = a->spec;
    const bool fp8 = s.kv_format == IDX_KV_FP8_E4M3;
    const int64_t kb = fp8 ? 1 : 2;       // bytes of a cached element
    if (a->p.rows > 0) {
        const bool strides_ok =
            io->q_row >= 0 && io->q_head >= 0 && io->k_slot >= 0 && io->k_head >= 0 &&
            io->v_slot >= 0 && io->v_head >= 0 && io->out_row >= 0 && io->out_head >= 0 &&
            (io->q_row * 2) % 16 == 0 && (io->q_head * 2) % 16 == 0 &&
            (io->k_slot * kb) % 16 == 0 && (io->k_head * kb) % 16 == 0 &&
            (io->v_slot * kb) % 16 == 0 && (io->v_head * kb) % 16 == 0 &&
            kb * io->k_slot <= UINT32_MAX && kb * io->v_slot <= UINT32_MAX &&
            (s.Hq == 1 || io->out_head >= s.D) && (a->p.rows == 1 || io->out_row >= s.D);
        if (!strides_ok || !io->q || !io->out || !io->sel || !io->compress_len ||
            (s.num_slots > 0 && (!io->k || !io->v)) || !is_aligned(io->q, 16) ||
            !is_aligned(io->k, 16) || !is_aligned(io->v, 16) || !is_aligned(io->out, 2) ||
            !is_aligned(io->sel, 4) || !is_aligned(io->sel_count, 4) ||
            !is_aligned(io->compress_len, 4) || !is_aligned(io->page_table, 4) ||
            !is_aligned(io->lse, 4) || !is_aligned(io->k_scale, 4) || !is_aligned(io->v_scale, 4) ||
            io->ld_sel < s.num_sel ||
            (fp8 && s.num_slots > 0 && (!io->k_scale || !io->v_scale)))
            return IDX_ERR_INVALID_ARG;
        if (s.page_size > 0) {
            int max_L = 0;
            for (int r = 0; r < a->p.num_requests; ++r)
                max_L = std::max(max_L, a->p.key_begin[r + 1] - a->p.key_begin[r]);
            if (!io->page_table ||
                io->ld_page_table < (max_L + (int64_t)s.page_size - 1) / s.page_size)
                return IDX_ERR_INVALID_ARG;
        }
    }
    if (a->p.rows > 0) {
        if (!ws || !is_aligned(ws, 256))
            return IDX_ERR_INVALID_ARG;
        if (ws_bytes < a->ws_bytes)
            return IDX_ERR_WORKSPACE;
    }
    if (!device_supported())
        return IDX_ERR_UNSUPPORTED;
    if (a->p.rows == 0)
        return IDX_OK;
    AttnParams p = a->p;
    p.q = static_cast<const uint8_t*>(io->q);
    p.k = static_cast<const uint8_t*>(io->k);
    p.v = static_cast<const uint8_t*>(io->v);
    p.out = static_cast<uint8_t*>(io->out);
    p.k_scale = io->k_scale;
    p.v_scale = io->v_scale;
    p.sel = io->sel;
    p.sel_count = io->sel_count;
    p.clen = io->compress_len;
    p.table = io->page_table;
    p.lse = io->lse;
    p.q_row = 2 * io->q_row;
    p.q_head = 2 * io->q_head;
    p.k_slot = kb * io->k_slot;
    p.k_head = kb * io->k_head;
    p.v_slot = kb * io->v_slot;
    p.v_head = kb * io->v_head;
    p.out_row = 2 * io->out_row;
    p.out_head = 2 * io->out_head;
    p.ld_sel = io->ld_sel;
    p.ld_table = io->ld_page_table;
    p.status = static_cast<uint32_t*>(ws);
    p.part_ml = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + 256);
    p.part_o = p.part_ml + 2 * a->part_floats;
    count_launch();
    return finish(launch_attention(p, s.D, s.dtype, fp8, static_cast<cudaStream_t>(stream)));
}

int indexer_mask_blocks(indexer_plan_t plan, const uint8_t* cand_mask, int64_t ld_mask,
                        const int32_t* compress_len, int32_t block, int32_t* blocks,
                        int32_t num_sel, int32_t* count, void* stream)
{
    if (!plan || block < 1 || num_sel < 1)
        return IDX_ERR_INVALID_ARG;
    const PlanView v = plan_view(plan);
    if (ld_mask < (v.max_L + (int64_t)block - 1) / block ||
        (v.T > 0 && (!cand_mask || !compress_len || !blocks || !is_aligned(compress_len, 4) ||
                     !is_aligned(blocks, 4) || !is_aligned(count, 4))))
        return IDX_ERR_INVALID_ARG;
    if (!device_supported())
        return IDX_ERR_UNSUPPORTED;
    if (v.T == 0)
        return IDX_OK;
    MaskBlocksParams p;
    std::memset(&p, 0, sizeof(p));
    p.mask = cand_mask;
    p.ld_mask = ld_mask;
    p.clen = compress_len;
    p.blocks = blocks;
    p.count = count;
    p.block = block;
    p.num_sel = num_sel;
    p.rows = v.T;
    p.max_blocks = static_cast<int32_t>((v.max_L + (int64_t)block - 1) / block);
    p.num_requests = v.R;
    std::copy(v.row_begin, v.row_begin + v.R + 1, p.row_begin);
    std::copy(v.L, v.L + v.R, p.key_count);
    count_launch();
    return finish(launch_mask_blocks(p, static_cast<cudaStream_t>(stream)));
}

int indexer_causal_attention_create(indexer_plan_t plan, const indexer_causal_spec* s,
                                    indexer_causal_t* out, size_t* ws_bytes)
{
    if (!out)
        return IDX_ERR_INVALID_ARG;
    *out = nullptr;
    if (!plan || !s || s->Hkv < 1 || s->Hq < 1 || s->Hq > IDX_MAX_HEADS ||
        s->Hq % s->Hkv != 0 || s->window < 0 || s->sinks < 0 ||
        (s->dtype != IDX_BF16 && s->dtype != IDX_FP16) ||
        (s->kv_format != IDX_KV_DENSE && s->kv_format != IDX_KV_FP8_E4M3) || s->num_slots < 0 ||
        s->page_size < 0 || !(std::fabs(s->scale) <= 1e38f) || s->D < 1)
        return IDX_ERR_INVALID_ARG;
    if (s->D != 64 && s->D != 128)
        return IDX_ERR_UNSUPPORTED;
    const PlanView v = plan_view(plan);
    if ((int64_t)v.T * s->Hq > INT32_MAX)
        return IDX_ERR_INVALID_ARG;
    indexer_causal_s* a = new (std::nothrow) indexer_causal_s();
    if (!a)
        return IDX_ERR_INVALID_ARG;
    a->spec = *s;
    CausalParams& p = a->p;
    std::memset(&p, 0, sizeof(p));
    const bool fp8 = s->kv_format == IDX_KV_FP8_E4M3;
    p.scale_log2 = static_cast<float>(s->scale * 1.4426950408889634);
    // (a masked score is -inf, which 0 would make NaN; 2^-100 leaves all weights alike as 0 does)
    if (p.scale_log2 == 0.0f)
        p.scale_log2 = 0x1p-100f;
    p.rows = v.T;
    p.Hq = s->Hq;
    p.Hkv = s->Hkv;
    p.group = s->Hq / s->Hkv;
    // (a window as long as the longest request hides nothing)
    p.window = s->window < v.max_L ? s->window : 0;
    p.sinks = p.window > 0 ? std::min(s->sinks, v.max_L) : 0;
    p.num_slots = s->num_slots;
    p.page = s->page_size;
    p.num_requests = v.R;
    std::copy(v.row_begin, v.row_begin + v.R + 1, p.row_begin);
    std::copy(v.key_begin, v.key_begin + v.R + 1, p.key_begin);
    if (s->page_size > 0)
        a->max_pages = (v.max_L + (int64_t)s->page_size - 1) / s->page_size;
    p.by_page = divisor(std::max(1, s->page_size));
    p.by_group = divisor(p.group);
    p.by_hkv = divisor(p.Hkv);
    // (the tiled form masks and takes the largest score before the scale)
    const double tiled = s->scale < 0.0f ? INFINITY : causal_cuts(p);
    // The form that ends first.  Over 1,350 calls (1 to 32 requests of 1 to 256 rows and 256 to 32,768
    // keys; 8, 32 and 64 heads, 1 to 16 to a cached one, of 64 and 128, 16-bit and e4m3 caches), each
    // timed both ways, the chosen one takes 0.6 % longer than the better one on average, six calls more
    // than 20 %, 38 % at most (four requests of two tokens over 32,768 bf16 keys, 8 heads of 128: 122
    // us against 89 in tiles, which take 1.6 us each there, not kTileUs): rows one by one for a token
    // or two a request (64 over 16,384 keys, 4 heads of 128: 322 us against 444 in tiles), tiles from
    // about eight (2,048 rows: 0.71 ms against 8.0).  Tiles of 64 KB take the rows' form 1.3 times as
    // long as what its splits are chosen by.
    const double by_rows = causal_rows(a->rows, p, *s, fp8) * (s->D == 128 && !fp8 ? 1.3 : 1.0);
    if (tiled == INFINITY && by_rows == INFINITY) {
        delete a;
        return IDX_ERR_INVALID_ARG;
    }
    a->by_rows = by_rows < tiled;
    // status word, then the parts of what is cut
    if (a->by_rows) {
        const AttnParams& q = a->rows;
        const int nh = attention_heads_per_tile(q.group, s->dtype, fp8);
        a->part_floats = q.splits > 1 && !q.cluster
                             ? (size_t)q.rows * q.Hkv * q.head_tiles * q.splits * nh * (s->D + 2)
                             : 0;
    } else {
        a->part_floats = p.joined ? (size_t)2 * p.blocks * kCausalRows * (s->D + 1) : 0;
    }
    a->ws_bytes = 256 + a->part_floats * sizeof(float);
    *out = a;
    if (ws_bytes)
        *ws_bytes = a->ws_bytes;
    return IDX_OK;
}

void indexer_causal_attention_destroy(indexer_causal_t a) { delete a; }

int indexer_causal_attention_info(indexer_causal_t a, int32_t* tiles, int32_t* blocks,
                                  int32_t* joined)
{
    if (!a)
        return IDX_ERR_INVALID_ARG;
    if (tiles)
        *tiles = !a->by_rows;
    if (blocks)
        *blocks = a->by_rows ? 0 : a->p.blocks;
    if (joined)
        *joined = a->by_rows ? 0 : a->p.joined;
    return IDX_OK;
}

int indexer_causal_attention(indexer_causal_t a, const indexer_causal_io* io, void* ws,
                             size_t ws_bytes, void* stream)
{
    if (!a || !io)
        return IDX_ERR_INVALID_ARG;
    const indexer_causal_spec& s = a->spec;
    const bool fp8 = s.kv_format == IDX_KV_FP8_E4M3;
    const int64_t kb = fp8 ? 1 : 2;       // bytes of a cached element
    if (a->p.rows > 0) {
        const bool strides_ok =
            io->q_row >= 0 && io->q_head >= 0 && io->k_slot >= 0 && io->k_head >= 0 &&
            io->v_slot >= 0 && io->v_head >= 0 && io->out_row >= 0 && io->out_head >= 0 &&
            (io->q_row * 2) % 16 == 0 && (io->q_head * 2) % 16 == 0 &&
            (io->k_slot * kb) % 16 == 0 && (io->k_head * kb) % 16 == 0 &&
            (io->v_slot * kb) % 16 == 0 && (io->v_head * kb) % 16 == 0 &&
            2 * io->q_row <= UINT32_MAX && 2 * io->q_head <= UINT32_MAX &&
            kb * io->k_slot <= UINT32_MAX && kb * io->v_slot <= UINT32_MAX &&
            (s.Hq == 1 || io->out_head >= s.D) && (a->p.rows == 1 || io->out_row >= s.D);
        if (!strides_ok || !io->q || !io->out || !io->compress_len ||
            (s.num_slots > 0 && (!io->k || !io->v)) || !is_aligned(io->q, 16) ||
            !is_aligned(io->k, 16) || !is_aligned(io->v, 16) || !is_aligned(io->out, 2) ||
            !is_aligned(io->compress_len, 4) || !is_aligned(io->page_table, 4) ||
            !is_aligned(io->lse, 4) || !is_aligned(io->k_scale, 4) || !is_aligned(io->v_scale, 4) ||
            (fp8 && s.num_slots > 0 && (!io->k_scale || !io->v_scale)) ||
            (s.page_size > 0 && a->max_pages > 0 &&
             (!io->page_table || io->ld_page_table < a->max_pages)))
            return IDX_ERR_INVALID_ARG;
        if (!ws || !is_aligned(ws, 256))
            return IDX_ERR_INVALID_ARG;
        if (ws_bytes < a->ws_bytes)
            return IDX_ERR_WORKSPACE;
    }
    if (!device_supported())
        return IDX_ERR_UNSUPPORTED;
    if (a->p.rows == 0)
        return IDX_OK;
    count_launch();
    if (a->by_rows) {
        AttnParams p = a->rows;
        p.q = static_cast<const uint8_t*>(io->q);
        p.k = static_cast<const uint8_t*>(io->k);
        p.v = static_cast<const uint8_t*>(io->v);
        p.out = static_cast<uint8_t*>(io->out);
        p.k_scale = io->k_scale;
        p.v_scale = io->v_scale;
        p.clen = io->compress_len;
        p.table = io->page_table;
        p.lse = io->lse;
        p.q_row = 2 * io->q_row;
        p.q_head = 2 * io->q_head;
        p.k_slot = kb * io->k_slot;
        p.k_head = kb * io->k_head;
        p.v_slot = kb * io->v_slot;
        p.v_head = kb * io->v_head;
        p.out_row = 2 * io->out_row;
        p.out_head = 2 * io->out_head;
        p.ld_table = io->ld_page_table;
        p.status = static_cast<uint32_t*>(ws);
        p.part_ml = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + 256);
        p.part_o = p.part_ml + a->part_floats / (s.D + 2) * 2;
        return finish(launch_attention_range(p, s.D, s.dtype, fp8, static_cast<cudaStream_t>(stream)));
    }
    CausalParams p = a->p;
    p.q = static_cast<const uint8_t*>(io->q);
    p.k = static_cast<const uint8_t*>(io->k);
    p.v = static_cast<const uint8_t*>(io->v);
    p.out = static_cast<uint8_t*>(io->out);
    p.k_scale = io->k_scale;
    p.v_scale = io->v_scale;
    p.clen = io->compress_len;
    p.table = io->page_table;
    p.lse = io->lse;
    p.q_row = 2 * io->q_row;
    p.q_head = 2 * io->q_head;
    p.k_slot = kb * io->k_slot;
    p.k_head = kb * io->k_head;
    p.v_slot = kb * io->v_slot;
    p.v_head = kb * io->v_head;
    p.out_row = 2 * io->out_row;
    p.out_head = 2 * io->out_head;
    p.out_vec = is_aligned(io->out, 32) && p.out_row % 32 == 0 && p.out_head % 32 == 0;
    p.q_boxes = p.group <= 128 && 128 % p.group == 0 &&
                map_rows(&p.q_map, io->q, s.D, s.Hq, p.rows, p.q_head, p.q_row, p.group,
                         128 / p.group);
    p.ld_table = io->ld_page_table;
    p.status = static_cast<uint32_t*>(ws);
    p.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + 256);
    p.part_lse = p.part_o + a->part_floats / (s.D + 1) * s.D;
    return finish(launch_causal(p, s.D, s.dtype, fp8, static_cast<cudaStream_t>(stream)));
}

int indexer_cache_append(indexer_plan_t plan, indexer_rope_t rope, const indexer_append_io* io,
                         void* stream)
{
    if (!io || !dense_type(io->dtype) || io->rows < 0 || io->heads < 1 ||
        io->heads > IDX_MAX_HEADS || io->D < 1 || io->D > kMaxHeadDim || io->num_slots < 0 ||
        io->page_size < 0 || (rope && rope->D != io->D) ||
        (io->cache_dtype != IDX_BF16 && io->cache_dtype != IDX_FP16 &&
         io->cache_dtype != IDX_CODES) ||
        (io->dtype != IDX_FP32 && io->cache_dtype != IDX_CODES && io->cache_dtype != io->dtype) ||
        (io->cache_dtype == IDX_CODES && io->D % 32 != 0) || io->k_row < 0 || io->k_head < 0 ||
        io->v_row < 0 || io->v_head < 0 || io->kc_slot < 0 || io->kc_head < 0 ||
        io->vc_slot < 0 || io->vc_head < 0 || (!plan && !io->slots))
        return IDX_ERR_INVALID_ARG;
    const bool fp8 = io->cache_dtype == IDX_CODES;
    const size_t eb = type_bytes(io->dtype);
    if (io->rows > 0 &&
        (!io->k || !io->v || ((rope || !io->slots) && !io->positions) || !is_aligned(io->k, eb) ||
         !is_aligned(io->v, eb) || !is_aligned(io->positions, 4) || !is_aligned(io->slots, 4) ||
         !is_aligned(io->page_table, 4) || !is_aligned(io->k_scale, 4) ||
         !is_aligned(io->v_scale, 4)))
        return IDX_ERR_INVALID_ARG;
    if (io->rows > 0 && io->num_slots > 0 &&
        (!io->k_cache || !io->v_cache || !is_aligned(io->k_cache, fp8 ? 8 : 2) ||
         !is_aligned(io->v_cache, fp8 ? 8 : 2) || (fp8 && (!io->k_scale || !io->v_scale)) ||
         (io->heads > 1 && (io->kc_head < io->D || io->vc_head < io->D)) ||
         (io->num_slots > 1 && (io->kc_slot < io->D || io->vc_slot < io->D)) ||
         (fp8 && (io->kc_slot % 8 != 0 || io->kc_head % 8 != 0 || io->vc_slot % 8 != 0 ||
                  io->vc_head % 8 != 0))))
        return IDX_ERR_INVALID_ARG;
    AppendCall c;
    std::memset(&c, 0, sizeof(c));
    if (plan) {
        const PlanView v = plan_view(plan);
        if (io->rows != v.T)
            return IDX_ERR_INVALID_ARG;
        if (!io->slots && io->page_size > 0 && io->rows > 0 &&
            (!io->page_table ||
             io->ld_page_table < (v.max_L + (int64_t)io->page_size - 1) / io->page_size))
            return IDX_ERR_INVALID_ARG;
        c.num_requests = v.R;
        std::copy(v.row_begin, v.row_begin + v.R + 1, c.row_begin);
        std::copy(v.key_begin, v.key_begin + v.R + 1, c.key_begin);
    }
    if (!device_supported())
        return IDX_ERR_UNSUPPORTED;
    if (io->rows == 0 || io->num_slots == 0)
        return IDX_OK;
    RopeParams rp;
    if (rope)
        rp = rope->p;
    else
        std::memset(&rp, 0, sizeof(rp));
    c.k = io->k;
    c.v = io->v;
    c.k_cache = io->k_cache;
    c.v_cache = io->v_cache;
    c.k_scale = io->k_scale;
    c.v_scale = io->v_scale;
    c.positions = io->positions;
    c.slots = io->slots;
    c.table = io->page_table;
    c.k_row = io->k_row;
    c.k_head = io->k_head;
    c.v_row = io->v_row;
    c.v_head = io->v_head;
    c.kc_slot = io->kc_slot;
    c.kc_head = io->kc_head;
    c.vc_slot = io->vc_slot;
    c.vc_head = io->vc_head;
    c.ld_table = io->ld_page_table;
    c.rows = io->rows;
    c.heads = io->heads;
    c.D = io->D;
    c.dtype = io->dtype;
    c.cache_dtype = io->cache_dtype;
    c.num_slots = io->num_slots;
    c.page = io->page_size;
    count_launch();
    return finish(launch_append(rp, c, static_cast<cudaStream_t>(stream)));
}

int indexer_attention_join(const indexer_join_io* io, void* stream)
{
    if (!io || io->parts < 1 || io->parts > IDX_MAX_PARTS || io->rows < 0 || io->heads < 1 ||
        io->heads > IDX_MAX_HEADS || io->D < 1 || io->D > kMaxHeadDim ||
        !dense_type(io->part_dtype) || !dense_type(io->out_dtype) ||
        (io->part_dtype != IDX_FP32 && io->out_dtype != io->part_dtype) || io->out_row < 0 ||
        io->out_head < 0 || (int64_t)io->rows * io->heads > INT32_MAX)
        return IDX_ERR_INVALID_ARG;
    JoinCall c;
    std::memset(&c, 0, sizeof(c));
    for (int p = 0; p < io->parts; ++p) {
        if (io->part_row[p] < 0 || io->part_head[p] < 0 ||
            (io->rows > 0 && (!io->part[p] || !io->part_lse[p] ||
                              !is_aligned(io->part[p], type_bytes(io->part_dtype)) ||
                              !is_aligned(io->part_lse[p], 4))))
            return IDX_ERR_INVALID_ARG;
        // (in place a thread overwrites what it alone has read; with another type or stride, what others
        // are yet to read)
        if (io->rows > 0 && io->part[p] == io->out &&
            (io->part_dtype != io->out_dtype || (io->rows > 1 && io->part_row[p] != io->out_row) ||
             (io->heads > 1 && io->part_head[p] != io->out_head)))
            return IDX_ERR_INVALID_ARG;
        c.part[p] = io->part[p];
        c.part_lse[p] = io->part_lse[p];
        c.part_row[p] = io->part_row[p];
        c.part_head[p] = io->part_head[p];
    }
    if (io->rows > 0 &&
        (!io->out || !is_aligned(io->out, type_bytes(io->out_dtype)) || !is_aligned(io->lse, 4) ||
         !is_aligned(io->sink, 4) || (io->heads > 1 && io->out_head < io->D) ||
         (io->rows > 1 && io->out_row < io->D)))
        return IDX_ERR_INVALID_ARG;
    if (!device_supported())
        return IDX_ERR_UNSUPPORTED;
    if (io->rows == 0)
        return IDX_OK;
    c.out = io->out;
    c.lse = io->lse;
    c.sink = io->sink;
    c.out_row = io->out_row;
    c.out_head = io->out_head;
    c.parts = io->parts;
    c.rows = io->rows;
    c.heads = io->heads;
    c.D = io->D;
    c.part_dtype = io->part_dtype;
    c.out_dtype = io->out_dtype;
    c.by_heads = divisor(c.heads);
    count_launch();
    return finish(launch_join(c, static_cast<cudaStream_t>(stream)));
}

int indexer_rms_norm(const indexer_norm_io* io, void* stream)
{
    if (!io || !dense_type(io->dtype) || io->rows < 0 || io->n < 1 || io->n > kMaxNorm ||
        !(io->eps >= 0.0f) || !std::isfinite(io->eps) ||
        (io->weight && io->weight_dtype != io->dtype && io->weight_dtype != IDX_FP32) ||
        io->x_row < 0 || io->residual_row < 0 || io->total_row < 0 || io->out_row < 0)
        return IDX_ERR_INVALID_ARG;
    if (io->codes && io->group != io->n &&
        ((io->group != 32 && io->group != 64 && io->group != 128 && io->group != 256) ||
         io->n % io->group != 0))
        return IDX_ERR_INVALID_ARG;
    const size_t eb = type_bytes(io->dtype);
    if (io->rows > 0 &&
        (!io->x || (!io->residual && io->total) || (!io->out && !io->codes && !io->total) ||
         !is_aligned(io->x, eb) || !is_aligned(io->residual, eb) ||
         !is_aligned(io->total, eb) || !is_aligned(io->out, eb) ||
         !is_aligned(io->weight, type_bytes(io->weight_dtype)) ||
         (io->codes && (!io->scales || !is_aligned(io->scales, 4))) ||
         (io->rows > 1 && ((io->total && io->total_row < io->n) ||
                           (io->out && io->out_row < io->n)))))
        return IDX_ERR_INVALID_ARG;
    if (!device_supported())
        return IDX_ERR_UNSUPPORTED;
    if (io->rows == 0)
        return IDX_OK;
    const NormCall c{io->x,
                     io->residual,
                     io->weight,
                     io->total,
                     io->out,
                     io->codes,
                     io->scales,
                     io->x_row,
                     io->residual_row,
                     io->total_row,
                     io->out_row,
                     io->rows,
                     io->n,
                     io->group,
                     io->dtype,
                     io->dtype == IDX_FP32 || io->weight_dtype == IDX_FP32,
                     io->eps};
    count_launch();
    return finish(launch_norm(c, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
