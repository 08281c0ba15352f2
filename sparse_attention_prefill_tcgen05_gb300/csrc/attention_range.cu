// Causal attention of single tokens: each row over the keys of its own range, with the selected keys'
// kernel.  There keys are the MMA's rows, so a token's few heads waste none of them, and a row's keys
// come to it alone, as a list's do.  64 rows over 16,384 paged keys, 4 x 8 heads of 128: 322 us, 2.15 GB at
// 6.7 TB/s, 98 % of the copy rate (in the tiles of the other form, of whose 128 rows 8 are used, 444 us).  64 rows
// under a window of 1,024 e4m3 keys, 8 x 8 heads of 64: 33 us against 73; 512 items of nine tiles on 152 SMs,
// 0.65 us a tile and 2 an item, bound by the tiles' chain of gather, scores, softmax and product.
#include "attention_tc.cuh"

namespace idx {

cudaError_t launch_attention_range(const AttnParams& p, int D, int dtype, bool fp8, cudaStream_t st)
{
    return attention_any<true>(p, D, dtype, fp8, st);
}

}  // namespace idx
