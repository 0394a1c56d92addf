// attn_decode.cu -- which of the decode attention's kernels (attn_kernel.cuh) runs.
#include <cstring>

#include "qmm_internal.h"

namespace qmm {

bool attn_takes_head_dim(int D)
{
    return D == 64 || D == 96 || D == 128 || D == 192 || D == 256;
}

AttnSpace attn_space(int type, int D)
{
    return type == QMM_F16 ? attn_space_f16(D)
           : type == QMM_BF16 ? attn_space_bf16(D)
                              : attn_space_q8(D);
}

cudaError_t launch_attn_decode(const AttnArgs &a, int sm_count, cudaStream_t s)
{
    AttnParams p;
    memset(static_cast<void *>(&p), 0, sizeof(p));
    p.a = a;
    p.group = a.n_q / a.c.n_heads;
    switch (a.type) {
    case QMM_F16: return launch_attn_f16(p, sm_count, s);
    case QMM_BF16: return launch_attn_bf16(p, sm_count, s);
    default: return launch_attn_q8(p, sm_count, s);
    }
}

} // namespace qmm
