// Internal interfaces between the host library and the kernels.  Nothing in
// here crosses the C ABI.
#pragma once
#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

struct indexer_plan_s;

namespace idx {

// Launch with programmatic stream serialization: the kernel may begin before the
// previous kernel in the stream has finished; it calls pdl_wait_then_release() before
// any global memory access.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl_cluster(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem,
                               cudaStream_t st, int cluster, Args&&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<Args&&>(args)...);
}
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t st, Args&&... args)
{
    return launch_pdl_cluster(kern, grid, block, smem, st, 1, static_cast<Args&&>(args)...);
}

constexpr int kTileKeys = 128;   // MMA M: keys per tile (one TMEM lane each)
constexpr int kTileN = 256;      // MMA N: (row, head) columns per tile
constexpr int kMaxSegments = 48;
constexpr int kMaxRequests = 256;

// Device status word bits (OR-ed by kernels, read by indexer_status).
constexpr uint32_t kStatusTimeout = 1u << 0;
constexpr uint32_t kStatusBadArg = 1u << 1;
constexpr uint32_t kStatusListOverflow = 1u << 2;   // a streamed list lost entries
constexpr uint32_t kStatusFp4Range = 1u << 3;       // an e2m1 key has no exact e4m3 form

// Key formats.

// What the logits kernel does with each (row, key) score.
constexpr int kSinkLogits = 0;   // write fp32 to a [rows, ld] buffer
constexpr int kSinkStream = 1;   // append threshold-passing (score, key) to per-row lists
constexpr int kSinkPool = 2;     // same over cand_block-key block maxima (candidate blocks)
constexpr int kSinkFilter = 3;   // append entries at or above a fixed per-row threshold
constexpr int kSinkPoolFilter = 4;  // the same over cand_block-key block maxima

constexpr int kListsPerSplit = 4;     // one candidate sub-list per epilogue warp quadrant
constexpr int kMaxStreamSlots = 256;  // sub-lists per row (key splits x kListsPerSplit)
constexpr int kMaxMergePieces = 64;   // row pieces per merge launch

// A contiguous piece of work: some rows of one request against a key range
// of that request.  Units (row group x key chunk) are numbered per launch.
struct Segment {
    int32_t row_begin;   // first global row
    int32_t nrows;
    int32_t key_base;    // packed key row of request-local key 0
    int32_t key_count;   // keys of the request; compress_len is clamped to it
    int32_t j_begin;     // request-local first key scored here
    int32_t j_end;       // request-local end (exclusive) of keys written here
    int32_t unit_begin;  // first unit number of this segment in the launch
    int32_t n_row_groups;
    int32_t n_chunks;
    int32_t unit_tiles;  // key tiles per unit
    int32_t tile_stride; // 1: every key tile; s: tiles 0, s, 2s, ... (sampled keys, whose
                         // logits go to consecutive output columns)
    int32_t cap;         // list sinks: entries per sub-list
    int64_t out_offset;  // logits: element offset of (row_begin, j_begin) in the output;
                         // streams: entry offset of row_begin's list for this split
    int64_t out_ld;      // logits: elements between rows; streams: entries between rows
    int64_t cnt_offset;  // streams: counts index of row_begin for this split
    int64_t cnt_ld;      // streams: counts between rows
};

struct LogitsParams {
    CUtensorMap tmap_q;  // [rows*H, D] bytes, box [256 rows, D]; e2m1 queries: [rows*H, D/2]
                         // packed, 64-byte swizzled
    CUtensorMap tmap_k;  // [keys, D] bytes, box [128 rows, D]; e2m1 keys: [keys, D/2]
                         // packed, unpacked by the map into 16-byte groups of 16 codes
    const float* s_q;    // [rows, H]; nullptr for e2m1 queries
    const float* w;      // [rows, H]
    const float* s_k;    // fp8 keys: [keys]
    const int32_t* compress_len;  // [rows]
    const uint8_t* cand_mask;     // nullable [rows, ld_mask] 0/1 per key block
    int64_t ld_mask;
    const int32_t* mask_rows;     // nullable [rows]: row t reads mask row mask_rows[t]
    int64_t mask_row_count;       // rows of cand_mask when mask_rows is set
    int32_t mask_block;
    int32_t num_segments;
    int32_t total_units;
    int32_t pad0_;
    long long timeout_cycles;
    float* out;
    uint32_t* status;
    // streamed top-k
    uint2* lists;         // (score bits, key or block index) entries
    uint32_t* counts;     // entries appended per (row, split), clamped to cap
    uint32_t* gtau;       // [rows] shared lower bound (ord of a score) per row
    int32_t keep;         // k (keys) or cand_topk (blocks)
    int32_t pool;         // keys per block for kSinkPool
    int32_t update_tiles; // tiles between threshold refreshes
    const uint32_t* tau_row;   // kSinkFilter: [rows] fixed threshold (ord of a score)
    const uint32_t* row_fail;  // nullable [rows]: only row groups with a set row run
    const uint32_t* fail_any;  // nullable: the whole launch has no work while it reads 0
    Segment seg[kMaxSegments];
    const uint32_t* k_sf; // e2m1 keys scored natively: [keys] four ue8m0 block scales
                          // (byte b: elements 32b..32b+31); nullptr for e4m3 keys
    const uint32_t* q_sf; // e2m1 queries (with e2m1 keys): [rows * H] four ue8m0 block
                          // scales per query vector; nullptr for e4m3 queries
};

// Host-side launchers (defined in the .cu files).
cudaError_t launch_logits(const LogitsParams& p, int H, int D, int sink, int grid,
                          cudaStream_t stream);
int logits_rows_per_group(int H, bool fp4_keys);   // query rows per MMA tile
bool logits_fp4_native(int H, int D);   // e2m1 keys scored by the block-scaled MMA

// Exact selection over the lists appended by the streaming sinks.  A piece is
// a row range of one request whose lists were filled by the same launch; one
// CTA per row.
struct MergePiece {
    int32_t row_begin;      // first global row
    int32_t nrows;
    int32_t cta_begin;      // first CTA of the piece in the launch
    int32_t slots;          // key splits (lists) per row
    int32_t cap;            // entries per list
    int32_t key_count;      // keys (or blocks) of the piece's request: indices are below it
    int64_t mask_delta;     // mask output: row t of the piece writes mask row t + mask_delta
    int64_t list_offset;    // entry offset of row_begin's first list
    int64_t count_offset;   // counts index of row_begin's first list
};
struct StreamMergeParams {
    const uint2* lists;
    const uint32_t* counts;
    const uint32_t* gtau;   // per-row lower bound on the k-th key: entries below it are skipped
    uint32_t* row_fail;     // [rows] verify: set for rows the lists cannot decide;
                            // only_failed: rows with a clear entry are skipped
    const uint32_t* tau_row;  // verify: the threshold the lists were filled with
    const uint32_t* smax_row; // nullable, verify: the largest sample of each row (ord)
    uint32_t* fail_any;       // verify: set when any row is flagged; only_failed: 0 = no work
    int32_t verify;
    int32_t only_failed;
    int32_t k;
    int32_t num_pieces;
    int32_t total_ctas;
    int32_t bitmap;            // 1: index-order output by bitmap where a row's keys allow
    int32_t* out_idx;
    float* out_val;
    uint8_t* mask;             // blocks: [rows, ld_mask]
    int64_t ld_mask;
    MergePiece piece[kMaxMergePieces];
};
cudaError_t launch_stream_merge(const StreamMergeParams& p, cudaStream_t stream);

// Standalone top-k over user logits [rows, ld].
struct TopkParams {
    const float* logits;
    int64_t ld;
    const int32_t* compress_len;
    int32_t k;
    int32_t total_rows;
    int32_t num_requests;
    int32_t pad_;
    int32_t* out_idx;
    float* out_val;
    const uint32_t* row_fail;    // nullable: only rows with a set flag (none while fail_any is 0)
    const uint32_t* fail_any;
    int32_t req_row_begin[kMaxRequests + 1];
    int32_t req_key_count[kMaxRequests];
};
cudaError_t launch_topk_dense(const TopkParams& p, cudaStream_t stream);

// Sampled path of the top-k over caller logits, one pass of rows [row0, row0 + rows):
// gather every tile_stride-th 128-key tile of each row into samples [rows, sample_cols]
// (keys past the row's length read as -inf), then (after the threshold kernel) append
// every entry at or above the row's threshold to its list.
struct DensePiece {
    int32_t row_begin;      // first global row
    int32_t nrows;
    int32_t request;
    int32_t slots;          // lists per row: key chunk c of the row appends to list c
    int32_t chunk;          // keys per chunk
    int32_t cap;            // entries per list
    int64_t list_offset;    // entry offset of row_begin's first list
    int64_t count_offset;   // counts index of row_begin's first list
};
struct DenseFilterParams {
    const float* logits;
    int64_t ld;
    const int32_t* compress_len;
    float* samples;              // gather: [rows of the pass, sample_cols]
    int32_t sample_cols;
    int32_t num_pieces;
    const uint32_t* tau_row;     // filter: [total rows]
    uint2* lists;
    uint32_t* counts;
    int32_t num_requests;
    int32_t pad_;
    int32_t req_stride[kMaxRequests];   // sampled tile stride (0: not sampled)
    int32_t req_key_count[kMaxRequests];
    DensePiece piece[kMaxMergePieces];
};
cudaError_t launch_dense_gather(const DenseFilterParams& p, int rows, cudaStream_t stream);
cudaError_t launch_dense_filter(const DenseFilterParams& p, int rows, int max_slots,
                                cudaStream_t stream);

// Per-row thresholds from sampled logits [rows, ld] (row t at t - row0): about
// the largest sample of rank mu + 5 sqrt(mu) + 4, mu = k * the row's sampled
// fraction, or 0 (everything passes) for rows of unsampled requests (stride 0),
// rows with at most k valid keys and rows with fewer samples.  With pool > 1 the
// ranked samples are the maxima of aligned pool-key blocks of the sampled keys
// and k counts blocks.
struct SampleParams {
    const float* samples;
    int64_t ld;
    int32_t row0;
    int32_t rows;
    int32_t k;
    int32_t num_requests;
    int32_t pool;                // keys per ranked entry (1: keys; 2, 4, 8: block maxima)
    int32_t pad_;
    const int32_t* compress_len;
    const float* logits;         // nullable: read the samples from caller logits [rows, ld]
                                 // (row t at t, sample e at key (e / 128) stride 128 + e % 128)
                                 // instead of `samples`
    int64_t ld_logits;
    uint32_t* tau_row;           // [total rows], written at row0 .. row0 + rows - 1
    uint32_t* smax_row;          // [total rows]: ord of the row's largest ranked sample where
                                 // tau is nonzero, else 0
    int32_t req_row_begin[kMaxRequests + 1];
    int32_t req_rank[kMaxRequests];    // sampling stride of the request, 0: not sampled
    int32_t req_key_count[kMaxRequests];
    int32_t req_cols[kMaxRequests];    // sample columns a row of the request fills (<= ld)
};
cudaError_t launch_sample_threshold(const SampleParams& p, cudaStream_t stream);

// Top-k over caller logits in one read per row (rows of at most 65,536 keys, k <= 2048):
// every entry at or above the row's sampled threshold is kept in shared memory and the
// exact selection runs there.  Rows it cannot decide (fewer than k entries at or above
// the threshold, more candidates than it holds) are flagged for the direct kernel.
struct RowTopkParams {
    const float* logits;         // [rows, ld], 16-byte aligned rows
    int64_t ld;
    const int32_t* compress_len;
    const uint32_t* tau_row;     // [rows] ord threshold, 0: every finite entry
    const uint32_t* smax_row;    // [rows] ord of the largest sample (bucket range)
    uint32_t* row_fail;
    uint32_t* fail_any;
    uint32_t* row_counter;       // zero at launch: rows are taken in order by the CTAs
    uint32_t* status;
    long long timeout_cycles;
    int32_t* out_idx;
    float* out_val;              // nullable
    int32_t k;
    int32_t total_rows;
    int32_t num_requests;
    int32_t pad_;
    int32_t req_row_begin[kMaxRequests + 1];
    int32_t req_key_count[kMaxRequests];
};
cudaError_t launch_row_topk(const RowTopkParams& p, cudaStream_t st);
int row_topk_max_keys();   // longest row (keys) the kernel takes

// Mask rows of rows with at most cand_topk candidate blocks: row t (of row0 .. row0 +
// rows - 1) writes mask row t + delta, 1 for its blocks below ceil(min(clen[t], keys) /
// block), 0 for the rest of the ld bytes.
cudaError_t launch_fill_mask_rows(uint8_t* mask, int64_t ld, const int32_t* clen, int row0,
                                  int rows, int keys, int block, int64_t delta, cudaStream_t st);
cudaError_t launch_expand_mask(const uint8_t* cand_mask, int64_t ld_mask, const int32_t* clen,
                               uint8_t* key_mask, int64_t ld, int block, int rows,
                               cudaStream_t st);
cudaError_t launch_selftest_timeout(uint32_t* status, long long cycles, cudaStream_t st);

// Page (KV slot) indices of selected raw key indices: out[t, i] =
// table[r, j / page] * page + j % page for 0 <= j < L_r (r the request of row t),
// else -1; -1 also where the table entry is negative or the slot does not fit int32.
struct PageIndexParams {
    const int32_t* raw;          // [rows, k]
    int32_t* out;                // [rows, k] (may be raw itself)
    const int32_t* table;        // [num_requests, ld_table]
    int64_t ld_table;
    int32_t page;
    int32_t k;
    int32_t rows;
    int32_t num_requests;
    int32_t req_row_begin[kMaxRequests + 1];
    int32_t req_key_count[kMaxRequests];
};
cudaError_t launch_page_indices(const PageIndexParams& p, cudaStream_t st);
// e2m1 keys [keys, D/2] (element 2i in the low nibble) with ue8m0 scales
// [keys, D/32] -> e4m3 keys [keys, D] and fp32 s_k [keys] = 2^(largest block
// exponent - 127), exactly; a key whose smaller blocks would need more than
// e4m3's range sets kStatusFp4Range in *status.
cudaError_t launch_fp4_to_fp8(const uint8_t* k4, const uint8_t* sf, int keys, int D, uint8_t* k8,
                              float* s_k, uint32_t* status, cudaStream_t st);
cudaError_t launch_pad_heads(const void* q, const float* s_q, const float* w, void* q_out,
                             float* s_q_out, float* w_out, int rows, int h_in, int h_out, int D,
                             cudaStream_t st);

// ------------------------------------------------- operators around the indexer
// What the operators' entry points read of a plan, and the library's launch counter.
struct PlanView {
    int R, T, Lk, max_L;
    const int32_t* row_begin;    // [R+1]
    const int32_t* key_begin;    // [R+1]
    const int32_t* L;            // [R]
};
PlanView plan_view(const struct ::indexer_plan_s* p);
void count_launch();             // adds one to indexer_launch_count
bool device_supported();         // the current device is one the kernels are built for
int device_sms();                // its SMs

// A kernel's attributes belong to a device: `set` runs in a device's first call, and again in the
// next one if it failed.  `done` has a bit per device (the 65th and later are set every time).
template <typename Set>
cudaError_t once_per_device(std::atomic<uint64_t>& done, int device, Set set)
{
    const uint64_t bit = device >= 0 && device < 64 ? 1ull << device : 0;
    if (done.load(std::memory_order_acquire) & bit)
        return cudaSuccess;
    const cudaError_t e = set();
    if (e == cudaSuccess)
        done.fetch_or(bit, std::memory_order_release);
    return e;
}

// An answer that does not change, kept once there is one (0: none).
template <typename Ask>
int remembered(std::atomic<int>& known, Ask ask)
{
    int v = known.load(std::memory_order_relaxed);
    if (v == 0) {
        v = ask();
        if (v != 0)
            known.store(v, std::memory_order_relaxed);
    }
    return v;
}

constexpr int kMaxRotPairs = 128;
constexpr int kMaxHeadDim = 256;

// Rotation of pairs of a vector's elements.  Pair i turns by position * inc[i] / 2^64
// turns: the product is taken modulo 2^64, so the angle is exact at every position.
struct RopeParams {
    int32_t rot;                 // rotated elements (even); 0: no rotation
    int32_t offset;              // first rotated element
    int32_t interleaved;         // pairs (2i, 2i+1) instead of (i, i + rot/2)
    int32_t inverse;             // turn back
    float amplitude;             // factor of the rotated elements
    uint64_t inc[kMaxRotPairs];
};

// x [rows, heads, D] (element strides, last axis contiguous) rotated into out.
struct RopeCall {
    const void* x;
    void* out;
    const int32_t* positions;    // [rows]
    int64_t x_row, x_head, out_row, out_head;   // strides in elements
    int32_t rows, heads, D, dtype;
};
cudaError_t launch_rope(const RopeParams& rp, const RopeCall& c, cudaStream_t st);

// x [rows, heads, D] rotated (rp.rot > 0) and quantised into rows of a cache
// [num_slots, heads]: row i goes to slot slots[i] (nullptr: i); slots outside
// [0, num_slots) are skipped.
struct CacheWriteCall {
    const void* x;
    const int32_t* positions;
    const int32_t* slots;
    uint8_t* codes;
    void* scales;
    int64_t x_row, x_head;
    int32_t rows, heads, D, dtype, num_slots, fp4;
};
cudaError_t launch_cache_write(const RopeParams& rp, const CacheWriteCall& c, cudaStream_t st);

// k and v [rows, heads, D], k rotated (rp.rot > 0), into slots of their caches: slots[i], or (nullptr)
// that of key positions[i] of row i's request through its page table (page > 0) or among the packed
// keys.  Keys outside the request, unmapped pages and slots outside [0, num_slots) are skipped.
struct AppendCall {
    const void* k;
    const void* v;
    void* k_cache;
    void* v_cache;
    float* k_scale;              // [num_slots, heads] (e4m3)
    float* v_scale;
    const int32_t* positions;
    const int32_t* slots;
    const int32_t* table;
    int64_t k_row, k_head, v_row, v_head;           // strides in elements
    int64_t kc_slot, kc_head, vc_slot, vc_head;
    int64_t ld_table;
    int32_t rows, heads, D, dtype;
    int32_t cache_dtype;         // IDX_BF16, IDX_FP16, or IDX_CODES: e4m3
    int32_t num_slots, page, num_requests;
    int32_t row_begin[kMaxRequests + 1];
    int32_t key_begin[kMaxRequests + 1];
};
cudaError_t launch_append(const RopeParams& rp, const AppendCall& c, cudaStream_t st);

// Cache rows slots[i] (nullptr: i), i < rows: as values of out_dtype, or (out_dtype
// IDX_CODES) as codes and scales.  Rows of slots outside the cache read as zeros.
struct CacheReadCall {
    const uint8_t* codes;
    const void* scales;
    const int32_t* slots;
    void* out;
    void* out_scales;
    int32_t rows, heads, D, num_slots, fp4, out_dtype;
};
cudaError_t launch_cache_read(const CacheReadCall& c, cudaStream_t st);

// Cache slot of every packed key of the batch: key j of request r is at
// table[r, j / page] * page + j % page, -1 where the entry is negative or the slot
// does not fit an int32.
struct PageSlotParams {
    const int32_t* table;
    int64_t ld_table;
    int32_t* slots;              // [total keys]
    int32_t page;
    int32_t num_requests;
    int32_t key_begin[kMaxRequests + 1];
};
cudaError_t launch_page_slots(const PageSlotParams& p, cudaStream_t st);

// Attention over the selected keys.  A work item is (row, key/value head, tile of query
// heads, split of the row's key tiles of kAttnTile keys).
constexpr int kAttnTile = 128;
constexpr int kMaxCluster = 4;      // splits that a cluster joins
constexpr int kMaxSplits = 64;
// Division of numbers below 2^31 by a constant of the call: n / d = (n * mul) >> shift with
// mul = ceil(2^shift / d), shift = 31 + ceil(log2 d).
struct Divisor {
    uint32_t mul;
    int32_t shift;
    int32_t d;
};
inline Divisor divisor(int32_t d)
{
    int l = 0;
    while ((1ll << l) < d)
        ++l;
    return Divisor{static_cast<uint32_t>(((1ull << (31 + l)) + d - 1) / d), 31 + l, d};
}
struct AttnParams {
    const uint8_t* q;            // byte strides
    const uint8_t* k;
    const uint8_t* v;
    uint8_t* out;
    const float* k_scale;
    const float* v_scale;
    const int32_t* sel;
    const int32_t* sel_count;
    const int32_t* clen;
    const int32_t* table;
    float* lse;
    int64_t q_row, q_head, k_slot, k_head, v_slot, v_head, out_row, out_head;
    int64_t ld_sel, ld_table;
    float* part_o;               // [items, heads of a tile, D] of split rows
    float* part_ml;              // [items, heads of a tile, 2]: running maximum (base 2), sum
    uint32_t* status;
    float scale_log2;            // scale * log2(e)
    int32_t rows, Hq, Hkv, group;    // group = Hq / Hkv
    int32_t head_tiles;          // tiles of query heads per key/value head
    int32_t block_shift;         // log2(keys per entry)
    int32_t num_sel;
    int32_t num_slots;
    int32_t page;                // 0: packed keys
    int32_t splits;              // splits per row
    int32_t cluster;             // a row's splits are a cluster's blocks, which join them
    Divisor by_page, by_splits, by_head_tiles, by_hkv;
    int32_t split_tiles;         // key tiles per split
    int32_t window, sinks;       // ranges: as CausalParams has them
    int32_t num_requests;
    int32_t row_begin[kMaxRequests + 1];
    int32_t key_begin[kMaxRequests + 1];
};
// Query heads of one key/value head that a work item takes together.
int attention_heads_per_tile(int group, int dtype, bool fp8);
cudaError_t launch_attention(const AttnParams& p, int D, int dtype, bool fp8, cudaStream_t st);
// The same over the keys below clen (sel and sel_count unused): all of them, or under a window.
cudaError_t launch_attention_range(const AttnParams& p, int D, int dtype, bool fp8, cudaStream_t st);

// Causal attention of a batch's rows over the cached keys of their requests.  A work item is
// (256 (token, query head) rows of a request, key/value head); a block takes a run of items' key
// tiles, which may begin and end inside an item.
constexpr int kCausalRows = 256;
constexpr int kCausalBlocks = 152;
// Tiles of 128 keys that tokens t0..t1 of a request of `tokens` new tokens see where its last token
// sees all its keys (which is what a plan goes by; their lengths are known on the device).
__host__ __device__ inline int causal_tiles(int keys, int tokens, int t0, int t1, int window,
                                            int sinks)
{
    const int before = keys - tokens + 1;
    const int most = before + t1 > 0 ? before + t1 : 0;
    int n = most;
    if (window > 0 && before + t0 - window > sinks)
        n = most - (before + t0 - window) + sinks;
    return n > 128 ? (n + 127) / 128 : 1;
}
struct CausalParams {
    CUtensorMap q_map;           // boxes of 128 rows of queries, 64 elements wide
    int32_t q_boxes;             // whether it holds: the group divides 128
    const uint8_t* q;            // byte strides
    const uint8_t* k;
    const uint8_t* v;
    uint8_t* out;
    const float* k_scale;
    const float* v_scale;
    const int32_t* clen;
    const int32_t* table;
    float* lse;
    int64_t q_row, q_head, k_slot, k_head, v_slot, v_head, out_row, out_head;
    int64_t ld_table;
    float* part_o;               // [2 blocks, kCausalRows, D]: parts of a block's first and last item
    float* part_lse;             // [2 blocks, kCausalRows]
    uint32_t* status;
    float scale_log2;            // scale * log2(e), positive
    int32_t out_vec;             // out takes 32-byte stores
    int32_t rows, Hq, Hkv, group;
    int32_t window, sinks;       // window 0: every key below a row's length
    int32_t num_slots, page;
    int32_t blocks;
    int32_t joined;              // items that are cut,
    int32_t most_rows;           // the most rows that an item has
    Divisor by_page, by_group, by_hkv;
    int32_t cut_item[kCausalBlocks + 1];    // where a block begins: in item, before tile
    int32_t cut_tile[kCausalBlocks + 1];
    int32_t first_cut[kCausalBlocks];       // of each item that is cut: the first block that begins in it
    int32_t num_requests;
    int32_t row_begin[kMaxRequests + 1];
    int32_t key_begin[kMaxRequests + 1];
    int32_t tile_begin[kMaxRequests + 1];   // tiles of kCausalRows rows before a request's
};
// A map of 16-bit rows [rows, heads, D] (byte strides) for boxes of 64 elements; false: none takes them.
bool map_rows(CUtensorMap* m, const void* base, int D, int heads, int rows, int64_t head, int64_t row,
              int box_heads, int box_rows);
cudaError_t launch_causal(const CausalParams& p, int D, int dtype, bool fp8, cudaStream_t st);

// Attention over disjoint sets of keys, joined by their log-sum-exps.
constexpr int kMaxParts = 8;
struct JoinCall {
    const void* part[kMaxParts];
    const float* part_lse[kMaxParts];               // [rows, heads]
    int64_t part_row[kMaxParts], part_head[kMaxParts];   // strides in elements
    void* out;
    float* lse;                  // nullable
    const float* sink;           // [heads], nullable
    int64_t out_row, out_head;
    int32_t parts, rows, heads, D;
    int32_t part_dtype, out_dtype;
    Divisor by_heads;
};
cudaError_t launch_join(const JoinCall& c, cudaStream_t st);

// Rows divided by their root mean square, times a weight.
constexpr int kMaxNorm = 65536;     // elements of a row
struct NormCall {
    const void* x;
    const void* residual;        // nullable
    const void* weight;          // nullable: ones
    void* total;                 // x + residual, nullable
    void* out;                   // nullable
    uint8_t* codes;              // [rows, n] e4m3, nullable
    float* scales;               // [rows, n / group]
    int64_t x_row, residual_row, total_row, out_row;     // strides in elements
    int32_t rows, n, group, dtype, weight_fp32;
    float eps;
};
cudaError_t launch_norm(const NormCall& c, cudaStream_t st);

struct MaskBlocksParams {
    const uint8_t* mask;
    int64_t ld_mask;
    const int32_t* clen;
    int32_t* blocks;
    int32_t* count;              // nullable
    int32_t block, num_sel, rows, num_requests;
    int32_t max_blocks;          // of the longest request: bytes of a mask row that exist
    int32_t row_begin[kMaxRequests + 1];
    int32_t key_count[kMaxRequests];
};
cudaError_t launch_mask_blocks(const MaskBlocksParams& p, cudaStream_t st);

}  // namespace idx
