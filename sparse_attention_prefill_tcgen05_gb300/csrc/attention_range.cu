// Causal attention of single tokens: each row over the keys of its own range.
#include "attention_tc.cuh"

namespace idx {

cudaError_t launch_attention_range(const AttnParams& p, int D, int dtype, bool fp8, cudaStream_t st)
{
    return attention_any<true>(p, D, dtype, fp8, st);
}

}  // namespace idx
