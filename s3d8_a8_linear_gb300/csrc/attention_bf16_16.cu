// Paged attention over a bf16 cache, 9 to 16 query rows a block.
#include "paged_attention.cuh"

namespace s3d8 {

namespace attn {

cudaError_t launch_bf16_16(const AttnArgs &a, const AttnPlan &p, int ctas, cudaStream_t stream)
{
    return launch_pages<false, 2>(a, p, ctas, stream);
}

}  // namespace attn

}  // namespace s3d8
