/*
 * indexer.h -- C ABI of the GB300 (sm_103a) dense prefill indexer.
 *
 * The indexer scores every query row t of a prefill chunk against every
 * compressed prefix key j of the row's request,
 *
 *     logit[t,j] = sum_h w[t,h] * ReLU( s_q[t,h] * s_k[j] * <q[t,h,:], k[j,:]> ),
 *
 * for j < compress_len(t) (the row's causal length), and keeps each row's
 * top-k keys.  Sources, by page and section:
 *   - "chunked-prefill-memory.md", section 1: the low-ratio indexer scores the
 *     chunk's T rows against the whole compressed prefix L and writes
 *     [T, max_seqlen_k] fp32 logits; section 2.3: key blocks with a per-block
 *     top-k and an exact top-k of the union; 8-key block pooling with the
 *     top-2048 blocks as candidates; consumers mask non-candidates.
 *   - SGLang PR #39187 "Bound the dense prefill indexer transient",
 *     Motivation/Modifications: DeepGEMM fp8_fp4_mqa_logits scoring, ragged
 *     requests, a caller-owned `selected` output, masks built straight into
 *     one preallocated buffer, a bounded transient; a block-level mask as the
 *     follow-up format.
 *   - SGLang fork commit log, the ragged-plan commit: per-batch metadata is
 *     built once and reused by every layer; host lengths avoid device syncs.
 * The score formula is the DeepSeek-V4 / NSA indexer's own (ReLU of the
 * scaled per-head dot products, weighted by w over the heads); the pages name
 * its kernels (fp8 / fp8_fp4 MQA logits) but never print it.
 *
 * Conventions shared by every entry point:
 *   - Layout.  Rows of all requests are packed: request r owns global rows
 *     [cu_seqlens_q[r], cu_seqlens_q[r+1]) and packed keys
 *     [cu_seqlens_k[r], cu_seqlens_k[r+1]).  Key indices in outputs are
 *     request-local (0 = first key of the row's request).
 *   - Eligibility.  Key j is eligible for row t iff j < compress_len[t]
 *     (compress_len is clamped to the request's key count) and, when a
 *     candidate mask is given, its block byte is non-zero.
 *   - Ties.  Equal scores are ordered by the lower key index.
 *   - Output order.  Kept indices are listed in ascending key order, then -1
 *     padding; `out_val` (optional) holds each kept key's score, -inf for
 *     padding.  Results are bitwise reproducible run to run and do not
 *     depend on the workspace size or the key-block size.
 *   - Ownership.  The caller owns every buffer (inputs, outputs, workspace).
 *     The plan owns only host metadata; the library allocates no device
 *     memory.  Device pointers are CUDA device addresses on the current
 *     device; `stream` is a cudaStream_t (NULL = legacy default stream).
 *   - Errors.  Return codes only (no exceptions, no exit, no printing).
 *     Argument errors are caught on the host before any launch.  Calls are
 *     asynchronous and never synchronize; a device-side failure (a wait that
 *     timed out) sets a status word in the workspace that indexer_status()
 *     reads.
 *   - Preconditions the library does not check on the device: q/k codes are
 *     finite (no e4m3 NaN codes 0x7F/0xFF, no ue8m0 255), scales s_q, s_k are
 *     positive and finite (so ReLU(s*x) = s*ReLU(x)), w is finite.
 */
#ifndef GB300_PREFILL_INDEXER_H
#define GB300_PREFILL_INDEXER_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes. */
#define IDX_OK 0
#define IDX_ERR_INVALID_ARG (-1)   /* bad size, pointer, alignment or layout */
#define IDX_ERR_UNSUPPORTED (-2)   /* shape/format the library has no kernel for, or not sm_103 */
#define IDX_ERR_WORKSPACE (-3)     /* workspace too small, or budget impossible at plan time */
#define IDX_ERR_CUDA (-4)          /* a CUDA runtime/driver call failed */
#define IDX_ERR_TIMEOUT (-5)       /* a device-side wait ran out (reported by indexer_status) */
#define IDX_ERR_DEVICE_CHECK (-6)  /* a device-side check failed (reported by indexer_status) */

/* Key formats. */
#define IDX_K_FP8_E4M3 0           /* k: e4m3 [keys, D]; k_scale: float s_k[keys] */
#define IDX_K_FP4_E2M1_UE8M0 1     /* k: e2m1 [keys, D/2], element 2i in the low nibble;
                                      k_scale: uint8 ue8m0 [keys, D/32]; s_k is 1.  With 32
                                      heads of 128 the block-scaled MMA applies the block
                                      scales (any block-scale span; k_scale 4-byte
                                      aligned); other head counts score the keys through
                                      their exact e4m3 form (see indexer_convert_fp4) */

/* Query formats. */
#define IDX_Q_FP8_E4M3 0           /* q: e4m3 [T, H, D]; s_q: float [T, H] */
#define IDX_Q_FP4_E2M1_UE8M0 1     /* q: e2m1 [T, H, D/2], element 2i in the low nibble;
                                      the s_q argument carries its block scales instead of
                                      float scales: uint8 ue8m0 [T, H, D/32] (4-byte
                                      aligned, passed as (const float*)); value =
                                      e2m1(code) * 2^(e - 127).  Needs kdtype
                                      IDX_K_FP4_E2M1_UE8M0 and 32 heads of 128: both operands
                                      then stay e2m1 in the block-scaled fp4 MMA
                                      (tcgen05 kind::mxf4, ue8m0 per 32 elements), any
                                      block-scale span on either side */

/* Row selection strategies of indexer_fused_topk (both exact). */
#define IDX_SELECT_AUTO 0          /* sampled row thresholds where rows are long enough,
                                      the running-threshold stream for undecided rows */
#define IDX_SELECT_STREAM 1        /* the running-threshold stream for every row */

/*
 * Problem description, read only by indexer_plan (host memory, copied).
 *   num_requests  R >= 1 (at most 256)
 *   total_rows    T = cu_seqlens_q[R];  total_keys = cu_seqlens_k[R]
 *   H, D          heads and head dim of q; k has D too.  Built shapes:
 *                 (H, D) in {(32,128), (16,128), (64,128), (8,64), (4,64)}; 4 heads run
 *                 as 8 (zero-padded into the workspace, which adds exactly 0)
 *   topk          keys kept per row, 1 <= topk <= 2048
 *   cu_seqlens_q  [R+1] non-decreasing row offsets, starts at 0
 *   cu_seqlens_k  [R+1] non-decreasing key offsets, starts at 0
 *   compress_len  [T] causal length of every row, 0 <= compress_len[t] <= the
 *                 keys of its request (e.g. floor((pos+1)/ratio))
 *   kdtype        IDX_K_FP8_E4M3 or IDX_K_FP4_E2M1_UE8M0
 *   qdtype        IDX_Q_FP8_E4M3 (0) or IDX_Q_FP4_E2M1_UE8M0; other values
 *                 IDX_ERR_INVALID_ARG, an unsupported pairing IDX_ERR_UNSUPPORTED
 *   cand_block    keys per candidate block: 1, 2, 4 or 8 (0 means 8)
 *   cand_topk     candidate blocks kept per row by indexer_candidate_blocks,
 *                 1..4096 (e.g. 2048); 0 = the plan makes no candidate-block
 *                 calls and reserves no workspace for them
 *   key_block     keys per key block of the streamed top-k (0 = planner's
 *                 choice; else a multiple of 128)
 *   transient_budget_bytes  cap on the workspace of the top-k and candidate
 *                 calls (0 means 2 GiB); the planner shrinks key blocks and
 *                 row chunks to fit and fails with IDX_ERR_WORKSPACE if it
 *                 cannot.
 *   select_mode   IDX_SELECT_AUTO or IDX_SELECT_STREAM.  AUTO scores every
 *                 32nd-or-so key tile first and takes, per row, a threshold a
 *                 little below the expected k-th score; the lists then hold every
 *                 key at or above it, and a row whose lists hold fewer than k
 *                 keys (or overflow) is selected again by the stream.  Results
 *                 are identical; only the work differs.
 */
typedef struct indexer_problem {
    int32_t num_requests;
    int32_t total_rows;
    int32_t total_keys;
    int32_t H;
    int32_t D;
    int32_t topk;
    const int32_t* cu_seqlens_q;
    const int32_t* cu_seqlens_k;
    const int32_t* compress_len;
    int32_t kdtype;
    int32_t cand_block;
    int32_t cand_topk;
    int32_t key_block;
    uint64_t transient_budget_bytes;
    int32_t select_mode;
    int32_t qdtype;
} indexer_problem;

typedef struct indexer_plan_s* indexer_plan_t;

/*
 * Validate a problem and build its plan (host metadata only: ragged tables,
 * key-block and row-chunk sizes, workspace layout).  Built once per batch and
 * reused by every layer of that batch (SGLang fork commit log, ragged-plan
 * commit).  *workspace_bytes receives the workspace every call on this plan
 * needs.  Needs no GPU.  Returns IDX_OK, IDX_ERR_INVALID_ARG,
 * IDX_ERR_UNSUPPORTED or IDX_ERR_WORKSPACE (budget impossible).
 */
int indexer_plan(const indexer_problem* problem, indexer_plan_t* out_plan,
                 size_t* workspace_bytes);
void indexer_plan_destroy(indexer_plan_t plan);

/* Key-block size, row-chunk size, key splits per row and key-tile sampling
 * stride (0 = no sampled thresholds) the plan chose (for reporting); any
 * pointer may be NULL. */
int indexer_plan_info(indexer_plan_t plan, int32_t* key_block, int32_t* row_chunk,
                      int32_t* max_splits, int32_t* sample_stride);

/*
 * Dense logits ("chunked-prefill-memory.md" section 1: [T, max_seqlen_k] fp32).
 *   q        e4m3 [T, H, D] (16-byte aligned)
 *   s_q, w   float [T, H]
 *   k        see kdtype (16-byte aligned); k_scale see kdtype
 *   compress_len  int32 [T] on the device, same values as the plan's
 *   logits   float [T, ld], ld >= the largest key count of the batch;
 *            logits[t, j] for j < compress_len[t], -inf for the rest of the row
 * ws/ws_bytes: the plan's workspace (256-byte aligned).
 * Range: every head's score (its fp32 dot product, block scales included) is applied
 * exactly for 2^-62 <= |S| < 2^64 (smaller ones keep an absolute error below 2^-150
 * times the head weight), with |w * s_q| < 2^64.
 */
int indexer_logits(indexer_plan_t plan, const void* q, const float* s_q, const float* w,
                   const void* k, const void* k_scale, const int32_t* compress_len,
                   float* logits, int64_t ld, void* ws, size_t ws_bytes, void* stream);

/*
 * Ragged per-row top-k over given logits [T, ld] (the ragged top-k of
 * "chunked-prefill-memory.md" section 2.3).  Entries j >= compress_len[t] and
 * -inf entries are not eligible.  out_idx int32 [T, topk]; out_val float
 * [T, topk] or NULL.  A row's kept keys are written in ascending key order,
 * then -1 (value -inf) padding.
 * With at least the plan's workspace, rows are sampled for a threshold and read
 * once (for 16-byte aligned rows of at most 65,536 keys the candidates and the
 * exact selection stay in shared memory); rows the sample cannot decide, and
 * every row when ws holds only the status area (256 bytes), get a direct exact
 * selection.  All of these give identical outputs.
 */
int indexer_topk(indexer_plan_t plan, const float* logits, int64_t ld,
                 const int32_t* compress_len, int32_t* out_idx, float* out_val, void* ws,
                 size_t ws_bytes, void* stream);

/*
 * Fused logits + top-k with a bounded transient: keys are scored block by
 * block and only per-block top-k candidates are kept, then merged exactly
 * ("chunked-prefill-memory.md" section 2.3); the [T, L] logits are never
 * materialised.  cand_mask (nullable) uint8 [T, ld_mask]: one byte per
 * cand_block-key block, non-zero = candidate (the consumer layer's mask);
 * ld_mask >= ceil(L/cand_block) for every request.
 */
int indexer_fused_topk(indexer_plan_t plan, const void* q, const float* s_q, const float* w,
                       const void* k, const void* k_scale, const int32_t* compress_len,
                       const uint8_t* cand_mask, int64_t ld_mask, int32_t* out_idx,
                       float* out_val, void* ws, size_t ws_bytes, void* stream);

/*
 * Candidate-source layer: pool each row's logits over cand_block-key blocks
 * (maximum over eligible keys, blocks aligned at key 0), keep the cand_topk
 * blocks with the largest pooled score (ties to the lower block) and write a
 * block-level mask: cand_mask uint8 [T, ld_mask], 1 = kept, 0 otherwise
 * (every byte of every row is written).  ld_mask >= ceil(L/cand_block).
 */
int indexer_candidate_blocks(indexer_plan_t plan, const void* q, const float* s_q,
                             const float* w, const void* k, const void* k_scale,
                             const int32_t* compress_len, uint8_t* cand_mask, int64_t ld_mask,
                             void* ws, size_t ws_bytes, void* stream);

/*
 * Expand a block-level mask to the key-level bool layout the pages' consumer
 * format uses: key_mask uint8 [T, ld], key_mask[t,j] = cand_mask[t, j/cand_block]
 * for j < compress_len[t], 0 otherwise.
 */
int indexer_expand_mask(indexer_plan_t plan, const uint8_t* cand_mask, int64_t ld_mask,
                        const int32_t* compress_len, uint8_t* key_mask, int64_t ld,
                        void* stream);

/*
 * Synchronizes `stream`, then reads the device status word in `ws`: IDX_OK,
 * IDX_ERR_TIMEOUT or IDX_ERR_DEVICE_CHECK.  Every compute call clears the
 * word when it starts.
 */
int indexer_status(indexer_plan_t plan, const void* ws, void* stream);

/*
 * Self-test of the bounded waits: launches one tiny kernel that waits on a
 * barrier nothing arrives on, with a budget of `cycles` SM cycles; it must
 * give up and set the timeout bit in the status word of `ws` (then
 * indexer_status returns IDX_ERR_TIMEOUT).  Never hangs.
 */
int indexer_selftest_timeout(void* ws, long long cycles, void* stream);

/* Budget, in SM clock cycles, of every device-side wait of later calls
   (default about two seconds). */
int indexer_set_wait_budget(indexer_plan_t plan, long long cycles);

/*
 * Fused top-k without a caller-provided workspace (no counterpart on the
 * pages: this entry point exists for callers that cannot allocate device
 * memory).  Some callers have no way to obtain device memory for a workspace:
 * a plugin whose host application owns all device memory through its own pool
 * and exposes no allocator, or a serving loop in which a cudaMalloc would
 * stall every stream on the device.  This variant computes exactly what
 * indexer_fused_topk computes, with the same arguments minus ws/ws_bytes; its
 * workspace is a file-scope device array of IDX_NOALLOC_SCRATCH_BYTES (64 MiB)
 * that every GPU loading this library holds until the process exits.
 *   - Limit: the plan's workspace must fit the array; build the plan with
 *     transient_budget_bytes <= 64 MiB.  A larger plan is rejected with
 *     IDX_ERR_WORKSPACE before anything is launched.
 *   - Allocation: none.  No cudaMalloc, cudaFree or allocating library call.
 *   - Set-up: the first call on a device resolves the array's device address
 *     (cudaGetSymbolAddress) with that device current and caches it; make
 *     that first call before any stream capture.
 *   - Sharing: every call uses the same array and it keeps the previous call's
 *     contents (the call clears what it needs cleared).  Calls whose work
 *     overlaps on the GPU (different streams, or several threads) race on the
 *     array: serialize them.
 *   - Status: device-side failures of a call (a wait that ran out, an e2m1 key
 *     the e4m3 conversion cannot represent, a candidate-mask row out of range) are recorded
 *     in the array's status word, which the call clears when it starts.
 *     indexer_noalloc_status reads it, as indexer_status reads a workspace.
 */
#define IDX_NOALLOC_SCRATCH_BYTES (64ull << 20)
int indexer_fused_topk_noalloc(indexer_plan_t plan, const void* q, const float* s_q,
                               const float* w, const void* k, const void* k_scale,
                               const int32_t* compress_len, const uint8_t* cand_mask,
                               int64_t ld_mask, int32_t* out_idx, float* out_val, void* stream);

/* Status of the last indexer_fused_topk_noalloc call on the current device
 * (no counterpart in the pages either: it is the allocation-free variant's
 * indexer_status).  Synchronizes `stream`, then reads the status word of the
 * library's scratch array: IDX_OK, IDX_ERR_TIMEOUT or IDX_ERR_DEVICE_CHECK
 * exactly as indexer_status; IDX_ERR_CUDA if a CUDA call fails,
 * IDX_ERR_UNSUPPORTED on a device other than sm_103.  Allocates nothing. */
int indexer_noalloc_status(void* stream);

/* Diagnostic: synchronizes `stream` and returns how many rows the last
   indexer_fused_topk / indexer_candidate_blocks / indexer_topk call on this
   workspace sent to the exact path (rows its sampled threshold could not
   decide), or a negative status.  The result is right only while the
   workspace has not been used by another call since. */
long long indexer_fallback_rows(indexer_plan_t plan, const void* ws, void* stream);

/* Number of kernels this library has launched in this process (a
   diagnostic counter for benchmarks; never reset). */
long long indexer_launch_count(void);

/* Benchmark diagnostic: while set, every indexer_fused_topk /
   indexer_candidate_blocks call records start_event (a cudaEvent_t) on its
   stream just before the first list-filling logits launch of its first pass
   and stop_event just after it, so the caller can time the dominant kernel
   inside a step.  NULL, NULL turns it off.  Process-wide, not thread-safe;
   the events are owned by the caller. */
void indexer_profile_main_kernel(void* start_event, void* stop_event);

/* ------------------------------------------- tail-only candidates, row maps
 * Under a decoder sliding-window bounded replay only each request's tail rows
 * are consumed by the later layers ("[SGLang PR 39187]", the third change:
 * publish only each request's tail rows, since the consumer slices every mask
 * down to them anyway).
 *
 * indexer_candidate_blocks_tail: indexer_candidate_blocks for request r's last
 *   publish_rows[r] rows only (host array [num_requests], 0 <= publish_rows[r]
 *   <= rows of r), packed: cand_mask is [sum_r publish_rows[r], ld_mask], request
 *   order, each request's rows in order.  Only those rows are scored.  A row's
 *   mask is byte-identical to the one indexer_candidate_blocks gives it.
 *   IDX_ERR_INVALID_ARG for a count out of range or a NULL array.
 *
 * indexer_fused_topk_mapped: indexer_fused_topk with a candidate mask whose rows
 *   are addressed through a row map: row t of the batch uses mask row
 *   mask_rows[t] (device int32 [total_rows]) of cand_mask [mask_row_count,
 *   ld_mask].  A map entry outside [0, mask_row_count) is reported by
 *   indexer_status as IDX_ERR_DEVICE_CHECK (that row then reads mask row 0).
 *   cand_mask and mask_rows are required (IDX_ERR_INVALID_ARG otherwise).
 */
int indexer_candidate_blocks_tail(indexer_plan_t plan, const void* q, const float* s_q,
                                  const float* w, const void* k, const void* k_scale,
                                  const int32_t* compress_len, const int32_t* publish_rows,
                                  uint8_t* cand_mask, int64_t ld_mask, void* ws,
                                  size_t ws_bytes, void* stream);
int indexer_fused_topk_mapped(indexer_plan_t plan, const void* q, const float* s_q,
                              const float* w, const void* k, const void* k_scale,
                              const int32_t* compress_len, const uint8_t* cand_mask,
                              int64_t ld_mask, const int32_t* mask_rows, int64_t mask_row_count,
                              int32_t* out_idx, float* out_val, void* ws, size_t ws_bytes,
                              void* stream);

/* ------------------------------------------------------------ fp4 operands
 * Exact conversion of e2m1 codes with one ue8m0 exponent per 32 elements
 * (OCP MX fp4: value = e2m1(code) * 2^(e - 127)) into e4m3 codes and one fp32
 * scale per row, value = e4m3(out) * out_scale[row] exactly, out_scale =
 * 2^(largest block exponent of the row - 127).  This is how the library runs
 * e2m1 keys for head counts without a block-scaled kernel (inside the calls, kdtype
 * IDX_K_FP4_E2M1_UE8M0; 32 heads of 128 use the block-scaled MMA instead), and how a
 * caller runs e2m1 queries with those head counts: convert q as T*H rows of D and pass
 * the e4m3 codes as q and the row scales as s_q (qdtype IDX_Q_FP8_E4M3).  With 32 heads
 * of 128, qdtype IDX_Q_FP4_E2M1_UE8M0 scores e2m1 queries natively instead.
 *   codes: device [rows, D/2] bytes, element 2i in the low nibble;
 *   block_scales: device [rows, D/32]; D a multiple of 32 (64 or 128 here);
 *   out_e4m3: device [rows, D]; out_scale: device fp32 [rows];
 *   ws: at least 256 bytes of device memory, 256-byte aligned: its status word is
 *   cleared, and a row whose smaller blocks fall below e4m3's range sets a bit
 *   that indexer_status(NULL, ws) reports as IDX_ERR_DEVICE_CHECK (read it before
 *   the workspace is used by another call, which clears it).
 * Async on `stream`, no allocation.
 */
int indexer_convert_fp4(const uint8_t* codes, const uint8_t* block_scales, int64_t rows,
                        int32_t D, uint8_t* out_e4m3, float* out_scale, void* ws,
                        size_t ws_bytes, void* stream);

/* ------------------------------------------------------ page-index transform
 * The indexer's selected keys as KV-cache slots ("[SGLang PR 39187]",
 * Accuracy / equivalence: the indexer's outputs are page_indices and
 * raw_indices; the pages name the top-k-then-transform step without printing
 * it, so this is the usual paged addressing):
 *     page_idx[t, i] = page_table[r, j / page_size] * page_size + j % page_size
 * for j = raw_idx[t, i] with 0 <= j < L_r, r the request of row t (the plan's
 * cu_seqlens_q) and L_r its key count (cu_seqlens_k); -1 where j is -1 or out
 * of [0, L_r), where the table entry is negative (an unmapped page), or where
 * the slot does not fit an int32.
 *   raw_idx, page_idx: device int32 [total_rows, topk] (the plan's topk), row-major;
 *     page_idx may equal raw_idx (in place).
 *   page_table: device int32 [num_requests, ld_page_table], row r holds request
 *     r's physical page of each logical page; ld_page_table must be at least
 *     ceil(max L_r / page_size), else IDX_ERR_INVALID_ARG.
 *   page_size >= 1 (a power of two takes a shift path).
 * Async on `stream`, no allocation, no workspace, no device-side errors.
 */
int indexer_page_indices(indexer_plan_t plan, const int32_t* raw_idx, const int32_t* page_table,
                         int64_t ld_page_table, int32_t page_size, int32_t* page_idx,
                         void* stream);

/* ------------------------------------------------------------ chunk planner
 * Adaptive prefill chunk ("chunked-prefill-memory.md", section 2.1, for callers
 * that still materialise [T, L] fp32 logits and must keep T x L under a budget):
 * for a prefix of prefix_len compressed keys
 *     chunk(L) = clamp( round_down( budget_token2 / L ), chunk_min, chunk_max )
 * where round_down goes to a multiple of `page` (pow2 == 0: the section's
 * formula) or to a power of two (pow2 != 0: this reproduces the schedule the
 * section prints -- 2048 up to ~98k keys, 1024 to ~195k, 512 to ~390k, 256
 * beyond).  The section's values: budget_token2 = 2.0e8, chunk_min = 256,
 * chunk_max = 2048, page = 256.  prefix_len <= 0 gives chunk_max.
 * Returns the chunk (>= chunk_min > 0), or IDX_ERR_INVALID_ARG when
 * budget_token2 <= 0 (or not finite), chunk_min < 1, chunk_max < chunk_min or
 * page < 1.  Host only: no device, no allocation, thread-safe.
 */
int indexer_chunk_rows(int64_t prefix_len, double budget_token2, int32_t chunk_min,
                       int32_t chunk_max, int32_t page, int32_t pow2);

/* ---------------------------------------------------------- rotary positions
 * The operators below are what a layer needs around the indexer: its bf16
 * projections turned into the indexer's operands, a quantised cache of them, and
 * attention over the keys the indexer selected.
 *
 * A rotation turns pairs of a head vector's elements: pair i of row t becomes
 *     a' = m (a cos u - b sin u),   b' = m (a sin u + b cos u),   u = position[t] * f_i
 * in fp32 with one rounding; the other elements are copied.
 *   D            elements of a head vector, 2..256
 *   rot_dim      rotated elements, even, 2..D; rot_offset the first of them
 *   layout       IDX_ROPE_HALF: pairs (i, i + rot_dim/2) of the rotated part;
 *                IDX_ROPE_INTERLEAVED: pairs (2i, 2i+1)
 *   base         f_i = base^(-2i/rot_dim)
 *   factor       context scaling, >= 1 (1: none).  With original_len <= 0 every f_i is
 *                divided by it.  With original_len > 0 pairs that make at most beta_slow
 *                turns over original_len positions are divided by it, those that make at
 *                least beta_fast are kept, and those between are mixed linearly in i
 *                (bounds rounded outwards to whole pairs)
 *   amplitude    m (1: none), applied to the rotated elements only
 * The angle is reduced exactly for every int32 position (a 64-bit phase per position), so
 * its error is below 3e-7 rad at any context length.
 */
#define IDX_BF16 0
#define IDX_FP16 1
#define IDX_FP32 2
#define IDX_CODES 3                /* indexer_cache_read: codes and scales as stored */
#define IDX_ROPE_HALF 0
#define IDX_ROPE_INTERLEAVED 1
#define IDX_MAX_HEADS 1024         /* heads of one call of the operators below */

typedef struct indexer_rope_spec {
    int32_t D;
    int32_t rot_dim;
    int32_t rot_offset;
    int32_t layout;
    double base;
    double factor;
    double original_len;
    double beta_fast;
    double beta_slow;
    double amplitude;
} indexer_rope_spec;

typedef struct indexer_rope_s* indexer_rope_t;

/* Validate a rotation and keep its frequencies (host only, needs no GPU; built once per
 * model and used by every call). */
int indexer_rope_create(const indexer_rope_spec* spec, indexer_rope_t* out_rope);
void indexer_rope_destroy(indexer_rope_t rope);

/* Rotate x [rows, heads, D] of dtype IDX_BF16, IDX_FP16 or IDX_FP32 into out (same type).
 * Strides are in elements (last axis contiguous, none negative; output rows and heads at
 * least D apart).  out may be x itself with the same strides, else the two must not
 * overlap.  positions: device int32 [rows], any value.  inverse = 1 turns back (the
 * rotation's transpose: also its gradient).  16-byte aligned rows, rot_dim a multiple of 16 and
 * rot_offset of 8 take the vector kernel. */
int indexer_rope(indexer_rope_t rope, const void* x, int32_t dtype, int32_t rows, int32_t heads,
                 int64_t row_stride, int64_t head_stride, const int32_t* positions,
                 int32_t inverse, void* out, int64_t out_row_stride, int64_t out_head_stride,
                 void* stream);

/* ------------------------------------------------- quantised operands and caches
 * A cache holds num_slots x heads vectors of D elements (D a multiple of 32, 32..256) in
 * one of the key formats:
 *   IDX_K_FP8_E4M3         codes e4m3 [num_slots, heads, D], scales float [num_slots, heads]:
 *                          scale = largest magnitude / 448 (at least 2^-126; 1 for a zero
 *                          vector), code = e4m3(x / scale), both quotients in fp32, ties
 *                          to even, saturating
 *   IDX_K_FP4_E2M1_UE8M0   codes [num_slots, heads, D/2] (element 2i in the low nibble),
 *                          scales ue8m0 [num_slots, heads, D/32]: 2^e with e =
 *                          floor(log2(largest magnitude)) - 2 of the 32 elements (1 for a
 *                          zero block), code = e2m1(x / 2^e), ties to even, saturating
 * With heads = 1 these are the indexer's keys, with slots = NULL its queries (T rows of H
 * heads: codes [T, H, D], s_q [T, H]).
 *
 * indexer_cache_write: x [rows, heads, D] (dtype and strides as above) is rotated (rope not
 *   NULL: positions int32 [rows], rope's D = D; the rotated values stay in fp32) and
 *   quantised into slot slots[i] (int32 [rows]; NULL: slot i).  Rows whose slot is negative
 *   or not below num_slots are skipped.  No two rows of a call may name the same slot.  NaN
 *   is stored as 0 and an infinity as the largest code of the largest scale, so codes and
 *   scales are always finite, as the indexer needs them.
 * indexer_cache_read: rows slots[i] (NULL: row i) of the cache into out [rows, heads, D] of
 *   out_dtype IDX_BF16, IDX_FP16 or IDX_FP32 as code * scale in fp32, rounded to the type; or with
 *   out_dtype IDX_CODES as codes (out) and scales (out_scales) packed in the cache's own
 *   format, which is how a paged cache becomes the packed keys of the indexer's calls.  A
 *   slot outside the cache reads as zeros (scale 1).
 * codes and out are 16-byte aligned, scales 4-byte aligned.
 */
int indexer_cache_write(indexer_rope_t rope, const void* x, int32_t dtype, int32_t rows,
                        int32_t heads, int32_t D, int64_t row_stride, int64_t head_stride,
                        const int32_t* positions, const int32_t* slots, int32_t num_slots,
                        int32_t format, void* codes, void* scales, void* stream);
int indexer_cache_read(const void* codes, const void* scales, int32_t format, int32_t num_slots,
                       int32_t heads, int32_t D, const int32_t* slots, int32_t rows,
                       int32_t out_dtype, void* out, void* out_scales, void* stream);

/* Cache slots of the batch's packed keys: slots [total_keys] = page_table[r, j / page_size] *
 * page_size + j % page_size for key j of request r, -1 where the entry is negative or the slot
 * does not fit an int32.  page_table as in indexer_page_indices.  Built once per batch, for
 * indexer_cache_read of whole prefixes. */
int indexer_page_slots(indexer_plan_t plan, const int32_t* page_table, int64_t ld_page_table,
                       int32_t page_size, int32_t* slots, void* stream);

/* ------------------------------------------- attention over the selected keys
 * For row t of request r, query head h and its key/value head g = h / (Hq / Hkv):
 *     a_j = scale * <q[t,h,:], k[slot(j),g,:]>,   lse[t,h] = log sum_j exp(a_j),
 *     out[t,h,:] = sum_j exp(a_j - lse[t,h]) v[slot(j),g,:]
 * over the row's selected keys j.  Entry sel[t,i] selects the keys
 * [sel * block, sel * block + block) of the row's request (block = 1: the indexer's key
 * indices); those below compress_len[t] and the request's key count take part.  Negative
 * entries, entries past the row's keys and entries at or past sel_count[t] select nothing, in any
 * place of the row; a key selected twice counts twice.  A row that selects nothing gives out = 0 and
 * lse = -inf.
 *   slot(j) = page_table[r, j / page_size] * page_size + j % page_size with page_size > 0,
 *   else the packed key cu_seqlens_k[r] + j.  Keys on negative table entries, or whose
 *   slot is not below num_slots, are left out.
 * Formats: q and out are dtype (IDX_BF16, IDX_FP16); k and v are of that type
 * (IDX_KV_DENSE) or caches of format IDX_K_FP8_E4M3 with their scales [num_slots, Hkv]
 * (IDX_KV_FP8_E4M3).  Scores, softmax and sums are fp32; the softmax weights (times v's scale) enter
 * the product with v with 8 significant bits, 11 where q is fp16 (over fp16 keys those below 2^-21 of
 * the row's largest with fewer, down to 2^-31 of it).  Under bf16 queries values from 2^-84 to 2^80
 * in size keep those bits in every list.
 *
 * indexer_attention_spec:
 *   Hq, Hkv      query and key/value heads, Hkv divides Hq, Hq <= IDX_MAX_HEADS
 *   D            64 or 128 (others IDX_ERR_UNSUPPORTED)
 *   block        keys per entry: 1, 2, 4, ... 128
 *   num_sel      entries per row, 1..65,536
 *   num_slots    rows of k and v
 *   scale        magnitude at most 1e38
 * indexer_attention_create: host only, needs no GPU, once per batch (plan: its requests, rows
 *   and key counts); *workspace_bytes receives what a call needs: 256 bytes for its status, and
 *   partial results where the rows alone do not fill the GPU and their keys are split over many
 *   blocks.  The plan may be destroyed afterwards.
 */
#define IDX_KV_DENSE 0
#define IDX_KV_FP8_E4M3 1

typedef struct indexer_attention_spec {
    int32_t Hq;
    int32_t Hkv;
    int32_t D;
    int32_t block;
    int32_t num_sel;
    int32_t dtype;
    int32_t kv_format;
    int32_t num_slots;
    int32_t page_size;
    float scale;
} indexer_attention_spec;

typedef struct indexer_attention_s* indexer_attention_t;

int indexer_attention_create(indexer_plan_t plan, const indexer_attention_spec* spec,
                             indexer_attention_t* out_attention, size_t* workspace_bytes);
void indexer_attention_destroy(indexer_attention_t attention);

/* Operands of one call.  Strides in elements, none negative; rows and heads of q, k and v
 * are 16-byte aligned (base and strides), the last axis contiguous, rows of k and v less than
 * 4 GiB apart; out's rows and heads are at least D apart.
 *   q [rows, Hq, D], k and v [num_slots, Hkv, D], out [rows, Hq, D]
 *   k_scale, v_scale  float [num_slots, Hkv] packed (IDX_KV_FP8_E4M3), positive and finite (as
 *                     indexer_cache_write leaves them) on slots that are selected; else NULL
 *   sel               int32 [rows, num_sel], rows ld_sel apart
 *   sel_count         int32 [rows] or NULL (num_sel for every row)
 *   compress_len      int32 [rows]
 *   page_table        int32 [requests, ld_page_table] (page_size > 0), else NULL
 *   lse               float [rows, Hq] packed, or NULL
 */
typedef struct indexer_attention_io {
    const void* q;
    const void* k;
    const void* v;
    void* out;
    const float* k_scale;
    const float* v_scale;
    const int32_t* sel;
    const int32_t* sel_count;
    const int32_t* compress_len;
    const int32_t* page_table;
    float* lse;
    int64_t q_row, q_head;
    int64_t k_slot, k_head;
    int64_t v_slot, v_head;
    int64_t out_row, out_head;
    int64_t ld_sel;
    int64_t ld_page_table;
} indexer_attention_io;

/* ws: 256-byte aligned, at least what indexer_attention_create asked for (NULL only where the
 * batch has no rows); its contents need no initialisation.  Two calls that overlap on the GPU
 * need a workspace each.  A wait that gave up sets the call's status, which
 * indexer_status(NULL, ws, stream) reads. */
int indexer_sparse_attention(indexer_attention_t attention, const indexer_attention_io* io,
                             void* ws, size_t ws_bytes, void* stream);

/* Block lists of a candidate mask (indexer_candidate_blocks' output, or any mask of
 * `block` keys per byte): blocks int32 [rows, num_sel] = the row's first num_sel non-zero
 * blocks below ceil(min(compress_len[t], L_r) / block) in ascending order, then -1; count
 * int32 [rows] (or NULL) how many those are.  ld_mask >= ceil(max L_r / block). */
int indexer_mask_blocks(indexer_plan_t plan, const uint8_t* cand_mask, int64_t ld_mask,
                        const int32_t* compress_len, int32_t block, int32_t* blocks,
                        int32_t num_sel, int32_t* count, void* stream);

/* ------------------------------------------------------------ causal attention
 * Attention of a batch's new tokens over the cached keys of their requests.  For row t of request r,
 * query head h and its key/value head g = h / (Hq / Hkv), with n = compress_len[t] (at most the
 * request's key count):
 *     a_j = scale * <q[t,h,:], k[slot(j),g,:]>,   lse[t,h] = log sum_j exp(a_j),
 *     out[t,h,:] = sum_j exp(a_j - lse[t,h]) v[slot(j),g,:]
 * over the keys j < n, with window > 0 only those with j >= n - window or j < sinks (a key that is
 * both counts once).  Lengths may be any in any order: a row of length 0 (padding) sees nothing.  A
 * row that sees no key gives out = 0 and lse = -inf.
 *   slot(j), formats, strides, rounding of weights: as indexer_sparse_attention has them (weights of
 *   8 significant bits, 11 under fp16 queries, those below 2^-21 of the row's largest with fewer over
 *   fp16 keys).  Keys on negative table entries, or whose slot is not below num_slots, are left out.
 *   Keys that no row of the call sees are not read, or have no effect, whatever they hold.
 *   A value that is not finite makes its column of the rows that see its key infinite or NaN (where the
 *   key's weight is above 0 in fp32), and changes neither other columns nor other rows.  A score that is
 *   NaN or +inf leaves its row no number.
 *
 * indexer_causal_spec:
 *   Hq, Hkv      query and key/value heads, Hkv divides Hq, Hq <= IDX_MAX_HEADS
 *   D            64 or 128 (others IDX_ERR_UNSUPPORTED)
 *   window       keys a row sees up to its own, 0: all of them
 *   sinks        first keys that stay visible under a window
 *   num_slots    rows of k and v
 *   page_size    0: packed keys
 *   scale        magnitude at most 1e38
 * indexer_causal_attention_create: host only, needs no GPU, once per batch (plan: its requests, rows
 *   and key counts); *workspace_bytes receives what a call needs: 256 bytes for its status, and
 *   partial results where work is cut so that all SMs get an equal share: up to 40 MB at D = 128, 20 at
 *   64, in tiles.  The plan may be destroyed afterwards.
 */
typedef struct indexer_causal_spec {
    int32_t Hq;
    int32_t Hkv;
    int32_t D;
    int32_t window;
    int32_t sinks;
    int32_t dtype;
    int32_t kv_format;
    int32_t num_slots;
    int32_t page_size;
    float scale;
} indexer_causal_spec;

typedef struct indexer_causal_s* indexer_causal_t;

int indexer_causal_attention_create(indexer_plan_t plan, const indexer_causal_spec* spec,
                                    indexer_causal_t* out_attention, size_t* workspace_bytes);
void indexer_causal_attention_destroy(indexer_causal_t attention);

/* What was chosen: *tiles 1 for tiles of rows, 0 for rows one by one; of the tiles, the blocks that share
 * them and how many (row tile, key/value head) items are cut between blocks and joined (else 0). */
int indexer_causal_attention_info(indexer_causal_t attention, int32_t* tiles, int32_t* blocks,
                                  int32_t* joined);

/* Operands of one call, as those of indexer_sparse_attention (rows and heads of q, and rows of k and v,
 * less than 4 GiB apart). */
typedef struct indexer_causal_io {
    const void* q;
    const void* k;
    const void* v;
    void* out;
    const float* k_scale;
    const float* v_scale;
    const int32_t* compress_len;
    const int32_t* page_table;
    float* lse;
    int64_t q_row, q_head;
    int64_t k_slot, k_head;
    int64_t v_slot, v_head;
    int64_t out_row, out_head;
    int64_t ld_page_table;
} indexer_causal_io;

/* ws and status: as indexer_sparse_attention's. */
int indexer_causal_attention(indexer_causal_t attention, const indexer_causal_io* io, void* ws,
                             size_t ws_bytes, void* stream);

/* --------------------------------------------------------------- cache append
 * New keys and values of a batch into their caches, the keys rotated on the way, in one launch:
 * for row t with position p = positions[t]
 *     k_cache[slot] = k[t] turned by rope to position p (rope NULL: as it is),  v_cache[slot] = v[t]
 * rounded once to the cache's type, or (cache_dtype IDX_CODES) as codes and scales of format
 * IDX_K_FP8_E4M3, exactly as indexer_cache_write stores them.
 *   slot = slots[t] where slots is given (the plan may then be NULL, positions too without rope);
 *   else that of key p of the row's request: page_table[r, p / page_size] * page_size +
 *   p % page_size with page_size > 0, the packed key cu_seqlens_k[r] + p without.
 * Rows whose position is not a key of the request (0 <= p < its key count), whose page is unmapped
 * (a negative entry) or whose slot is not in [0, num_slots) are skipped: the caches stay as they
 * are.  No two rows of a call may name the same slot.
 *   k, v              [rows, heads, D] of dtype IDX_BF16, IDX_FP16 or IDX_FP32, strides in elements
 *                     (last axis contiguous, none negative); rows: the plan's, where there is one
 *   k_cache, v_cache  [num_slots, heads, D] of cache_dtype: dtype itself (any of the two 16-bit types
 *                     for IDX_FP32), or IDX_CODES: e4m3 codes (D a multiple of 32, 8-byte aligned
 *                     rows and heads) with k_scale, v_scale float [num_slots, heads] packed.  Strides
 *                     in elements, slots and heads at least D apart: two halves of one tensor will do
 *   D                 1..256 (with rope: rope's)
 */
typedef struct indexer_append_io {
    const void* k;
    const void* v;
    void* k_cache;
    void* v_cache;
    float* k_scale;
    float* v_scale;
    const int32_t* positions;
    const int32_t* slots;
    const int32_t* page_table;
    int64_t k_row, k_head;
    int64_t v_row, v_head;
    int64_t kc_slot, kc_head;
    int64_t vc_slot, vc_head;
    int64_t ld_page_table;
    int32_t rows;
    int32_t heads;
    int32_t D;
    int32_t dtype;
    int32_t cache_dtype;
    int32_t num_slots;
    int32_t page_size;
} indexer_append_io;

int indexer_cache_append(indexer_plan_t plan, indexer_rope_t rope, const indexer_append_io* io,
                         void* stream);

/* ------------------------------------------------------ attention parts joined
 * Attention over disjoint sets of keys as one: of `parts` outputs and log-sum-exps of the same rows
 * (indexer_sparse_attention's and indexer_causal_attention's, say)
 *     lse[t,h] = log(sum_p exp(lse_p[t,h]) + exp(sink[h])),
 *     out[t,h,:] = sum_p exp(lse_p[t,h] - lse[t,h]) out_p[t,h,:]
 * in fp32 with one rounding.  sink float [heads]: a learned logit of attending to nothing (NULL: none).
 * A part whose lse is -inf, or whose weight is 0 in fp32, takes no part, whatever its output holds; where
 * all are -inf, and there is no sink, out = 0 and lse = -inf.
 *   part[p]      [rows, heads, D] of part_dtype, strides in elements (last axis contiguous);
 *   part_lse[p]  float [rows, heads] packed
 *   out          [rows, heads, D] of out_dtype: part_dtype, or any type over IDX_FP32 parts; may be
 *                one of the parts with its type and strides (others at its address are refused), else it
 *                overlaps none
 *   lse          float [rows, heads] packed, or NULL; may be one of the parts'
 *   D            1..256; rows * heads below 2^31
 */
#define IDX_MAX_PARTS 8

typedef struct indexer_join_io {
    const void* part[IDX_MAX_PARTS];
    const float* part_lse[IDX_MAX_PARTS];
    int64_t part_row[IDX_MAX_PARTS];
    int64_t part_head[IDX_MAX_PARTS];
    void* out;
    float* lse;
    const float* sink;
    int64_t out_row, out_head;
    int32_t parts;
    int32_t rows;
    int32_t heads;
    int32_t D;
    int32_t part_dtype;
    int32_t out_dtype;
} indexer_join_io;

int indexer_attention_join(const indexer_join_io* io, void* stream);

/* ------------------------------------------------------------------- RMS norm
 *     h = x + residual,   y = h / sqrt(mean(h^2) + eps) * weight
 * per row of n elements (1..65,536), in fp32 (so the squares of a row have to be within its range);
 * h is rounded where it is stored (total), y where it is (out), and its codes are those of the
 * unrounded y: e4m3, a scale for every `group` elements, as format IDX_K_FP8_E4M3 has them (largest
 * magnitude / 448; NaN as 0, an infinity as the largest code).
 *   x, residual, total, out  [rows, n] of dtype IDX_BF16, IDX_FP16 or IDX_FP32, rows `_row` elements
 *                 apart (outputs at least n); residual may be NULL (h = x), total and out too.  total
 *                 may be residual or x, out may be x (with the same strides); no other overlap
 *   weight        [n] of weight_dtype: dtype or IDX_FP32 (NULL: ones)
 *   codes         [rows, n] packed, or NULL; scales float [rows, n / group] packed
 *   group         32, 64, 128 or 256, a divisor of n, or n itself (one scale a row)
 *   eps           >= 0
 */
typedef struct indexer_norm_io {
    const void* x;
    const void* residual;
    const void* weight;
    void* total;
    void* out;
    uint8_t* codes;
    float* scales;
    int64_t x_row, residual_row, total_row, out_row;
    int32_t rows;
    int32_t n;
    int32_t group;
    int32_t dtype;
    int32_t weight_dtype;
    float eps;
} indexer_norm_io;

int indexer_rms_norm(const indexer_norm_io* io, void* stream);

const char* indexer_error_string(int status);
int indexer_version(void);

#ifdef __cplusplus
}
#endif
#endif
