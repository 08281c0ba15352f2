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
    // Work items: rows x key/value heads x tiles of query heads, each over the row's key
    // tiles.  Where they do not fill the SMs, the tiles of a row are split.  Two or four splits
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
    const int nh = attention_heads_per_tile(p.group, s->dtype, s->kv_format != IDX_KV_DENSE);
    p.head_tiles = (p.group + nh - 1) / nh;
    const int64_t tiles = (((int64_t)s->num_sel << p.block_shift) + kAttnTile - 1) / kAttnTile;
    const int64_t items = (int64_t)v.T * s->Hkv * p.head_tiles;
    if (items > (1 << 30)) {
        delete a;
        return IDX_ERR_INVALID_ARG;
    }
    double best = INFINITY;
    for (int64_t n = 1; n <= std::min<int64_t>(tiles, kMaxSplits) && items * n <= (1 << 30); ++n) {
        const int64_t per = (tiles + n - 1) / n;
        if ((tiles + per - 1) / per != n)
            continue;
        const double waves = static_cast<double>((items * n + kPlanSms - 1) / kPlanSms);
        const bool cluster = (n == 2 || n == kMaxCluster) && items * n <= kClusterBlocks;
        const double bytes = 4.0 * s->D * nh * (items * n);
        const double join = n == 1 ? 0.0 : cluster ? 1.4 : 1.1 + 0.15 * n + 1e-6 / 4 * bytes;
        const double cost = waves * (0.65 * per + 2.0) + join;
        if (cost < best) {
            best = cost;
            p.cluster = cluster;
            p.splits = static_cast<int32_t>(n);
            p.split_tiles = static_cast<int32_t>(per);
        }
    }
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

}  // extern "C"
