// attn_q8.cu -- the decode attention's kernels for a cache in Q8_0.
#include "attn_kernel.cuh"

namespace qmm {

cudaError_t launch_attn_q8(AttnParams &p, int sm_count, cudaStream_t s)
{
    return launch_kind<kQ8>(p, sm_count, s);
}

AttnSpace attn_space_q8(int D) { return space_kind<kQ8>(D); }

} // namespace qmm
