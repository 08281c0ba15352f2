// Attention over the selected keys, and the block lists of candidate masks.
#include "attention_tc.cuh"

namespace idx {
namespace {

// The bits of a word's non-zero bytes.
__device__ __forceinline__ uint32_t nonzero_bytes(uint32_t w)
{
    const uint32_t m = __vsetgtu4(w, 0u);        // 1 in every non-zero byte
    return (m | m >> 7 | m >> 14 | m >> 21) & 15u;
}

// One warp per row.  A lane reads 16 mask bytes of each of four runs of 512 at once and counts
// them; its first set byte's place is the row's count so far plus the lanes' before it.  (A byte
// a lane with a ballot per 32 bytes waited for memory at every step.)  16,384 rows of 18,750 blocks:
// 3.5 TB/s, the walk over set bits between the reads.
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
    const uint8_t* all_end = p.mask + (p.rows - 1) * p.ld_mask + p.max_blocks;
    int32_t* out = p.blocks + t * p.num_sel;
    // from the 16-byte boundary at or below the row (whole vectors only inside the mask)
    const int skew = static_cast<int>(reinterpret_cast<uintptr_t>(m) & 15);
    int n = 0;
    for (int b0 = -skew; b0 < nb && n < p.num_sel; b0 += 2048) {
        uint32_t bits[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int b = b0 + 512 * k + 16 * lane;
            bits[k] = 0;
            if (b < nb) {
                if (m + b >= p.mask && m + b + 16 <= all_end) {
                    const uint4 w = *reinterpret_cast<const uint4*>(m + b);
                    bits[k] = nonzero_bytes(w.x) | nonzero_bytes(w.y) << 4 |
                              nonzero_bytes(w.z) << 8 | nonzero_bytes(w.w) << 12;
                } else {
                    for (int i = max(0, -b); i < 16 && b + i < nb; ++i)
                        bits[k] |= (m[b + i] != 0 ? 1u : 0u) << i;
                }
                if (b < 0)
                    bits[k] &= 0xFFFFu << -b;            // bytes of the row before
                if (b + 16 > nb)
                    bits[k] &= (1u << (nb - b)) - 1u;    // past the row's blocks
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int mine = __popc(bits[k]);
            int before = mine;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, before, d);
                before += lane >= d ? v : 0;
            }
            const int total = __shfl_sync(0xFFFFFFFFu, before, 31);
            int at = n + before - mine;
            for (uint32_t left = bits[k]; left != 0 && at < p.num_sel; left &= left - 1)
                out[at++] = b0 + 512 * k + 16 * lane + __ffs(left) - 1;
            n += total;
        }
    }
    n = min(n, p.num_sel);
    for (int i = n + lane; i < p.num_sel; i += 32)
        out[i] = -1;
    if (p.count && lane == 0)
        p.count[t] = n;
}

}  // namespace

int attention_heads_per_tile(int group, int dtype, bool fp8)
{
    // The smallest tile that holds the group: a wider one computes heads that are none (16 heads in
    // tiles of 16 153 us, of 32 168; 32 heads of 32 176, of 64 226: 2,048 rows, 2,048 keys of
    // 128 bf16; e4m3 190, 217, 219, 298), a narrower one gathers the keys again for each (32 heads in two
    // of 16 298 us, 64 in two of 32 337 against 236; e4m3 361 and 419 against 302).  fp16 queries over
    // e4m3 caches: two of 32, the terms of 64 leave room for two tiles and too few registers (541
    // us against 476).
    if (fp8 && dtype == IDX_FP16)
        return group <= 16 ? 16 : 32;
    return group <= 16 ? 16 : group <= 32 ? 32 : 64;
}

cudaError_t launch_attention(const AttnParams& p, int D, int dtype, bool fp8, cudaStream_t st)
{
    return attention_any<false>(p, D, dtype, fp8, st);
}

cudaError_t launch_mask_blocks(const MaskBlocksParams& p, cudaStream_t st)
{
    return launch_pdl(mask_blocks_kernel, dim3(static_cast<unsigned>((p.rows + 3) / 4)), dim3(128),
                      0, st, p);
}

}  // namespace idx
