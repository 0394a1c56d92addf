// attn_bf16.cu -- the decode attention's kernels for a cache in BF16.
#include "attn_kernel.cuh"

namespace qmm {

cudaError_t launch_attn_bf16(AttnParams &p, int sm_count, cudaStream_t s)
{
    return launch_kind<kBF16>(p, sm_count, s);
}

AttnSpace attn_space_bf16(int D) { return space_kind<kBF16>(D); }

} // namespace qmm
