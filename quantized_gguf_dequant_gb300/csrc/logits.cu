// logits.cu -- a model's logits adjusted before sampling: penalties for
// repeated tokens, biases, and a mask of what a grammar allows, in one pass.
//
//   c = times v occurs in the row's history
//   z = logits[v];  c > 0:  z = z > 0 ? z / r : z * r;  z -= presence + frequency * c
//   z += the row's biases for v, added in list order
//   bit v of the row's mask clear:  z = -inf
// all in fp32, rounded once to the logits' type.
//
// Bytes bound it: each logit is read and written once.  A block owns a chunk
// of one row: it takes the chunk's logits into registers, counts the history
// tokens that fall into the chunk in shared memory (whole-number atomics: no
// order to matter) while those loads are under way, and applies everything on
// the way out.  The history is scanned by every chunk of its row, out of L2.
// A bias list may name a token twice: the entry with the lowest index owns
// the token and adds the others in list order, so the sum is repeatable.
// Groups of four logits are taken at their 16-byte boundaries whatever the
// row's own alignment, so an odd vocabulary costs nothing but its ragged ends.
#include <algorithm>

#include "kv_cache.cuh"
#include "qmm_device.cuh"
#include "qmm_internal.h"

namespace qmm {

namespace {

constexpr int kThreads = 256;
constexpr uint32_t kNoOwner = 0xffffffffu;
constexpr int WIDE = 4;   // groups of four logits of a thread where rows are many
constexpr int AHEAD = 4;  // history tokens of a thread under way at once

__device__ __forceinline__ int64_t clamp64(int64_t v, int64_t hi)
{
    return v < 0 ? 0 : (v > hi ? hi : v);
}

// VEC: input and output rows are equally misaligned, groups of four go as one.
template <typename IO, int GROUPS, bool VEC>
__global__ void __launch_bounds__(kThreads) adjust_kernel(const __grid_constant__ LogitsArgs P)
{
    constexpr int CHUNK = GROUPS * kThreads * 4;
    extern __shared__ __align__(16) uint32_t shared[];
    uint32_t *counts = shared;
    uint32_t *bias = shared + (P.n_history > 0 ? CHUNK : 0);  // owner's index, then the sum's bits
    pdl_wait();
    pdl_launch_dependents();
    const int64_t b = blockIdx.x;
    const IO *in = static_cast<const IO *>(P.in) + b * P.ld_in;
    IO *out = static_cast<IO *>(P.out) + b * P.ld_out;
    // logits before the row's first group boundary
    const int shift = VEC ? int((reinterpret_cast<uintptr_t>(in) / sizeof(IO)) & 3) : 0;
    const int v0 = int(blockIdx.y) * CHUNK - shift;  // (n_vocab <= 2^26)
    const int V = int(P.V), tid = threadIdx.x;

    // Everything whose place is known is asked for at once: the logits, the
    // mask's words, the lists' ends and the penalties.
    float4 x[GROUPS];
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) {
        const int e = v0 + (i * kThreads + tid) * 4;
        x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (VEC && e >= 0 && e + 4 <= V) {
            x[i] = load4(in + e);
        } else {
            float *f = reinterpret_cast<float *>(&x[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (e + j >= 0 && e + j < V)
                    f[j] = load1(in + e + j);
        }
    }
    uint32_t word[GROUPS];
    const uint32_t *mask = P.mask ? P.mask + b * P.ld_mask : nullptr;
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) {
        const int e = v0 + (i * kThreads + tid) * 4;
        word[i] = mask && e < V ? __ldg(mask + (e < 0 ? 0 : e >> 5)) : 0u;
    }
    int64_t h0 = 0, h1 = 0, b0 = 0, b1 = 0;
    if (P.n_history > 0) {
        h0 = clamp64(__ldg(P.history_offsets + b), P.n_history);
        h1 = clamp64(__ldg(P.history_offsets + b + 1), P.n_history);
    }
    if (P.n_biases > 0) {
        b0 = clamp64(__ldg(P.bias_offsets + b), P.n_biases);
        b1 = clamp64(__ldg(P.bias_offsets + b + 1), P.n_biases);
    }
    const float r = P.repeat ? __ldg(P.repeat + b) : 1.f;
    const float presence = P.presence ? __ldg(P.presence + b) : 0.f;
    const float frequency = P.frequency ? __ldg(P.frequency + b) : 0.f;
    const bool counted = h1 > h0, biased = b1 > b0;
    if (counted || biased) {
        // a token's place in this chunk, or -1
        auto place = [&](int id) {
            const unsigned at = unsigned(id) - unsigned(v0);
            return unsigned(id) < unsigned(V) && at < unsigned(CHUNK) ? int(at) : -1;
        };
        // the first of the lists are on their way while the arrays are cleared
        int id[AHEAD], bid = -1;
        float bval = 0.f;
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            const int64_t i = h0 + tid + j * kThreads;
            id[j] = i < h1 ? __ldg(P.history + i) : -1;
        }
        if (b0 + tid < b1) {
            bid = __ldg(P.bias_ids + b0 + tid);
            bval = __ldg(P.bias_values + b0 + tid);
        }
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) {
            const int at = (i * kThreads + tid) * 4;
            if (counted)
                *reinterpret_cast<uint4 *>(counts + at) = make_uint4(0, 0, 0, 0);
            if (biased)
                *reinterpret_cast<uint4 *>(bias + at) =
                    make_uint4(kNoOwner, kNoOwner, kNoOwner, kNoOwner);
        }
        __syncthreads();
        for (int64_t i = h0 + tid; i < h1; i += AHEAD * kThreads) {
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                const int at = place(id[j]);
                if (at >= 0)
                    atomicAdd(counts + at, 1u);
                const int64_t next = i + (AHEAD + j) * kThreads;
                id[j] = next < h1 ? __ldg(P.history + next) : -1;
            }
        }
        if (biased) {
            int at = place(bid);
            if (at >= 0)
                atomicMin(bias + at, uint32_t(tid));
            for (int64_t i = b0 + tid + kThreads; i < b1; i += kThreads) {
                const int a2 = place(__ldg(P.bias_ids + i));
                if (a2 >= 0)
                    atomicMin(bias + a2, uint32_t(i - b0));
            }
            __syncthreads();
            bool twice = at >= 0 && bias[at] != uint32_t(tid);  // a token of this chunk named twice
            for (int64_t i = b0 + tid + kThreads; i < b1; i += kThreads) {
                const int a2 = place(__ldg(P.bias_ids + i));
                twice |= a2 >= 0 && bias[a2] != uint32_t(i - b0);
            }
            twice = __syncthreads_or(twice);
            for (int64_t i = b0 + tid; i < b1; i += kThreads) {
                if (i >= b0 + kThreads) {
                    bid = __ldg(P.bias_ids + i);
                    bval = __ldg(P.bias_values + i);
                    at = place(bid);
                }
                if (at < 0)
                    continue;
                float sum = bval;
                if (twice) {
                    // (the owners' indices are being overwritten: look at the list)
                    int64_t k = b0;
                    while (k < i && __ldg(P.bias_ids + k) != bid)
                        ++k;
                    if (k < i)
                        continue;
                    for (k = i + 1; k < b1; ++k)
                        if (__ldg(P.bias_ids + k) == bid)
                            sum = __fadd_rn(sum, __ldg(P.bias_values + k));
                }
                const uint32_t bits = __float_as_uint(sum);
                bias[at] = bits == kNoOwner ? 0x7fffffffu : bits;
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) {
        const int at = (i * kThreads + tid) * 4;
        const int e = v0 + at;
        if (e + 4 <= 0 || e >= V)
            continue;
        float *f = reinterpret_cast<float *>(&x[i]);
        if (counted) {
            const uint4 c4 = *reinterpret_cast<const uint4 *>(counts + at);
            if (c4.x | c4.y | c4.z | c4.w) {
                const uint32_t c[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (c[j]) {
                        const float z = f[j] > 0.f ? __fdiv_rn(f[j], r) : __fmul_rn(f[j], r);
                        f[j] =
                            __fsub_rn(z, __fadd_rn(presence, __fmul_rn(frequency, float(c[j]))));
                    }
            }
        }
        if (biased) {
            const uint4 s4 = *reinterpret_cast<const uint4 *>(bias + at);
            if ((s4.x & s4.y & s4.z & s4.w) != kNoOwner) {
                const uint32_t s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (s[j] != kNoOwner)
                        f[j] = __fadd_rn(f[j], __uint_as_float(s[j]));
            }
        }
        if (mask) {
            const int first = e < 0 ? 0 : e, w = first >> 5;
            // (groups at odd places may reach into the next word)
            const uint32_t hi = (first & 31) > 28 && (w + 1) * 32 < V ? __ldg(mask + w + 1) : 0u;
            const uint32_t bits = __funnelshift_r(word[i], hi, first & 31);
            const uint32_t four = e < 0 ? bits << -e : bits;  // bit j: logit e + j
#pragma unroll
            for (int j = 0; j < 4; ++j)
                f[j] = four & (1u << j) ? f[j] : -INFINITY;
        }
        if (VEC && e >= 0 && e + 4 <= V) {
            store4(out + e, x[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (e + j >= 0 && e + j < V)
                    store1(out + e + j, f[j]);
        }
    }
}

template <typename IO, int GROUPS, bool VEC>
cudaError_t launch(const LogitsArgs &a, cudaStream_t s)
{
    constexpr int CHUNK = GROUPS * kThreads * 4;
    const auto kern = adjust_kernel<IO, GROUPS, VEC>;
    const size_t smem = size_t(CHUNK) * 4 * ((a.n_history > 0) + (a.n_biases > 0));
    cudaError_t e = func_smem(reinterpret_cast<const void *>(kern), smem);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(a.B), unsigned((a.V + 3 + CHUNK - 1) / CHUNK));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
    return counted(cudaLaunchKernelEx(&cfg, kern, a));
}

template <typename IO>
cudaError_t launch_io(const LogitsArgs &a, int sm_count, cudaStream_t s)
{
    const size_t unit = 4 * sizeof(IO);
    const bool vec =
        (reinterpret_cast<uintptr_t>(a.in) - reinterpret_cast<uintptr_t>(a.out)) % unit == 0 &&
        (a.B == 1 || size_t(a.ld_in - a.ld_out) * sizeof(IO) % unit == 0);
    // Long chunks share a row's history scan; short ones spread a small batch
    // over the SMs.
    const bool wide = a.B * a.V >= int64_t(sm_count) * 4 * 8192;
    if (wide)
        return vec ? launch<IO, WIDE, true>(a, s) : launch<IO, WIDE, false>(a, s);
    return vec ? launch<IO, 2, true>(a, s) : launch<IO, 2, false>(a, s);
}

} // namespace

cudaError_t launch_logits_adjust(const LogitsArgs &a, int sm_count, cudaStream_t s)
{
    switch (a.dtype) {
    case QMM_F32: return launch_io<float>(a, sm_count, s);
    case QMM_F16: return launch_io<__half>(a, sm_count, s);
    default: return launch_io<__nv_bfloat16>(a, sm_count, s);
    }
}

} // namespace qmm
