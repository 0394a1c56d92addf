// attn_f16.cu -- the decode attention's kernels for a cache in F16.
#include "attn_kernel.cuh"

namespace qmm {

cudaError_t launch_attn_f16(AttnParams &p, int sm_count, cudaStream_t s)
{
    return launch_kind<kF16>(p, sm_count, s);
}

AttnSpace attn_space_f16(int D) { return space_kind<kF16>(D); }

} // namespace qmm
