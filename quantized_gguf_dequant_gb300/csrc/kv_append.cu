// kv_append.cu -- new tokens into the paged key-value cache: rotary positions
// for q and k, the rotated k and the v rounded into the cache's type, one
// launch; and the way back out (qmm_kv_read).
//
// Pair i of a head's first n_rot dims, (a, b) = (i, i + n_rot/2) or
// (2i, 2i+1), turns by angle_i = fl32(pos[axis(i)] * inv_freq[i]):
//   a' = a cos - b sin,  b' = b cos + a sin
// each product and difference rounded to fp32 on its own, so that the stored
// bits do not depend on how a compiler contracts them.
//
// Bytes bound it: q, k and v are read once, q_out and the cache rows written
// once.  A block takes one token (or, when there are few tokens, one part of
// its heads, so that a decode step spreads over the SMs): the token's cosines
// and sines are computed once into shared memory and serve all its heads.  A
// warp owns whole rows of D values, four to a lane; it holds a row and the
// row's partners in registers before it stores anything, so q_out may be q.
// A Q8_0 block of 32 values is eight lanes.
#include <algorithm>
#include <cstring>

#include "kv_cache.cuh"
#include "qmm_device.cuh"
#include "qmm_internal.h"

namespace qmm {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

enum Kind { kF16, kBF16, kQ8 };

// Four rounded values of a Q8_0 block held by eight lanes (scale = amax/127,
// code = rint(x / scale), the scale kept in fp16).
__device__ __forceinline__ uint32_t quantize4(float4 x, float &d)
{
    float amax = fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w)));
    // a NaN must reach the stored scale: fmaxf would drop it
    const bool nan = x.x != x.x || x.y != x.y || x.z != x.z || x.w != x.w;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const unsigned lanes = __ballot_sync(0xffffffffu, nan);
    if ((lanes >> (threadIdx.x & 24)) & 0xffu)
        amax = __int_as_float(0x7fc00000);
    d = __fdiv_rn(amax, 127.f);
    const float inv = d > 0.f ? __fdiv_rn(1.f, d) : 0.f;
    auto code = [&](float v) {
        return uint32_t(__float2int_rn(__fmul_rn(v, inv))) & 0xffu;
    };
    return code(x.x) | (code(x.y) << 8) | (code(x.z) << 16) | (code(x.w) << 24);
}

template <Kind KIND, typename IO, int D>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendArgs P)
{
    constexpr int LPR = D / 4 < 32 ? D / 4 : 32;         // lanes per row
    constexpr int RPW = D <= 64 ? 32 / LPR : 1;          // rows per warp and pass
    constexpr int PASSES = (D + 127) / 128;
    constexpr int SP = kv_scales_per_row(D);
    __shared__ float2 turn[128];  // (cos, sin) of each pair
    pdl_wait();
    pdl_launch_dependents();
    const int64_t tok = blockIdx.x;
    const int half = P.n_rot >> 1;
    for (int i = threadIdx.x; i < half; i += kThreads) {
        int ax = 0;
        while (i >= P.axis_end[ax])
            ++ax;
        const float angle =
            __fmul_rn(float(P.pos[int64_t(ax) * P.T + tok]), __ldg(P.inv_freq + i));
        float sn, cn;
        sincosf(angle, &sn, &cn);
        turn[i] = make_float2(cn, sn);
    }
    __syncthreads();
    const int64_t slot = __ldg(P.slots + tok);
    const KvView &c = P.c;
    const bool stored = slot >= 0 && slot < int64_t(c.n_pages) * c.page_size;
    if (slot >= 0 && !stored && threadIdx.x == 0 && blockIdx.y == 0)
        atomicOr(P.status, kStatusBadSlotBit);
    int64_t row0 = 0;
    if (stored) {
        const int64_t page = slot / c.page_size;
        row0 = page * c.n_heads * c.page_size + (slot - page * c.page_size);
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = lane / LPR, li = lane % LPR;
    const int rows = P.n_q + 2 * c.n_heads;
    const bool vec = (P.n_rot & 7) == 0;
    for (int base = (int(blockIdx.y) * kWarps + warp) * RPW; base < rows;
         base += int(gridDim.y) * kWarps * RPW) {
        const int r = base + sub;
        const bool isq = r < P.n_q, isk = !isq && r < P.n_q + c.n_heads;
        const bool active = sub < RPW && r < rows && (isq || stored);
        const int head = isq ? r : (isk ? r - P.n_q : r - P.n_q - c.n_heads);
        const IO *src = static_cast<const IO *>(isq ? P.q : (isk ? P.k : P.v)) +
                        tok * (isq ? P.ldq : (isk ? P.ldk : P.ldv)) + int64_t(head) * D;
        const bool rot = isq || isk;
        float4 own[PASSES], par[PASSES];
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const int e = p * 128 + 4 * li;
            own[p] = par[p] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (!active || e >= D)
                continue;
            own[p] = load4(src + e);
            if (rot && !P.adjacent && e < P.n_rot) {
                if (vec) {
                    par[p] = load4(src + (e < half ? e + half : e - half));
                } else {
                    float *f = reinterpret_cast<float *>(&par[p]);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (e + j < P.n_rot)
                            f[j] = load1(src + (e + j < half ? e + j + half : e + j - half));
                }
            }
        }
        __syncwarp();  // q_out may be q: every load of the row is done before its first store
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const int e = p * 128 + 4 * li;
            const bool here = active && e < D;
            float4 y = own[p];
            if (here && rot && e < P.n_rot) {
                const float *x = reinterpret_cast<const float *>(&own[p]);
                const float *o = reinterpret_cast<const float *>(&par[p]);
                float *f = reinterpret_cast<float *>(&y);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (e + j >= P.n_rot)
                        continue;
                    const bool second = P.adjacent ? (j & 1) : e + j >= half;
                    const int pair = P.adjacent ? (e + j) >> 1 : (second ? e + j - half : e + j);
                    const float other = P.adjacent ? x[j ^ 1] : o[j];
                    const float2 cs = turn[pair];
                    const float a = __fmul_rn(x[j], cs.x), b = __fmul_rn(other, cs.y);
                    f[j] = second ? __fadd_rn(a, b) : __fsub_rn(a, b);
                }
            }
            if (here && isq)
                store4(static_cast<IO *>(P.q_out) + tok * P.ldqo + int64_t(head) * D + e, y);
            const int64_t row = row0 + int64_t(head) * c.page_size;
            uint8_t *dst = (isk ? c.k : c.v);
            if constexpr (KIND == kQ8) {
                float d;
                const uint32_t codes = quantize4(y, d);  // (every lane: it shuffles)
                if (here && !isq) {
                    *reinterpret_cast<uint32_t *>(dst + row * D + e) = codes;
                    if ((lane & 7) == 0)
                        static_cast<__half *>(isk ? c.ks : c.vs)[row * SP + e / 32] =
                            __float2half_rn(d);
                }
            } else if (here && !isq) {
                if constexpr (KIND == kF16)
                    store4(reinterpret_cast<__half *>(dst) + row * D + e, y);
                else
                    store4(reinterpret_cast<__nv_bfloat16 *>(dst) + row * D + e, y);
            }
        }
    }
}

// Rows of the cache as values: a thread takes four values of k and of v.
template <Kind KIND, typename IO>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ KvReadArgs P)
{
    pdl_wait();
    pdl_launch_dependents();
    const KvView &c = P.c;
    const int D = c.D, quads = D / 4, SP = kv_scales_per_row(D);
    const int per_token = c.n_heads * quads;
    const int64_t n = P.T * per_token;
    for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < n;
         i += int64_t(gridDim.x) * kThreads) {
        const int64_t tok = i / per_token;
        const int in = int(i - tok * per_token);
        const int head = in / quads, e = (in - head * quads) * 4;
        const int64_t slot = __ldg(P.slots + tok);
        const bool held = slot >= 0 && slot < int64_t(c.n_pages) * c.page_size;
        if (slot >= 0 && !held && in == 0)
            atomicOr(P.status, kStatusBadSlotBit);
        float4 kv[2] = {};
        if (held) {
            const int64_t page = slot / c.page_size;
            const int64_t row =
                (page * c.n_heads + head) * c.page_size + (slot - page * c.page_size);
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                if (!(w ? P.v : P.k))
                    continue;
                const uint8_t *src = w ? c.v : c.k;
                if constexpr (KIND == kF16) {
                    kv[w] = load4(reinterpret_cast<const __half *>(src) + row * D + e);
                } else if constexpr (KIND == kBF16) {
                    kv[w] = load4(reinterpret_cast<const __nv_bfloat16 *>(src) + row * D + e);
                } else {
                    const char4 q = *reinterpret_cast<const char4 *>(src + row * D + e);
                    const float d = __half2float(
                        static_cast<const __half *>(w ? c.vs : c.ks)[row * SP + e / 32]);
                    kv[w] = make_float4(q.x * d, q.y * d, q.z * d, q.w * d);
                }
            }
        }
        if (P.k)
            store4(static_cast<IO *>(P.k) + tok * P.ldk + int64_t(head) * D + e, kv[0]);
        if (P.v)
            store4(static_cast<IO *>(P.v) + tok * P.ldv + int64_t(head) * D + e, kv[1]);
    }
}

template <typename Args>
cudaError_t launch(void (*k)(Args), dim3 grid, cudaStream_t s, const Args &a)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
    return counted(cudaLaunchKernelEx(&cfg, k, a));
}

template <Kind KIND, typename IO>
cudaError_t append_for_dim(const AppendArgs &a, dim3 grid, cudaStream_t s)
{
    switch (a.c.D) {
    case 64: return launch(append_kernel<KIND, IO, 64>, grid, s, a);
    case 96: return launch(append_kernel<KIND, IO, 96>, grid, s, a);
    case 128: return launch(append_kernel<KIND, IO, 128>, grid, s, a);
    case 192: return launch(append_kernel<KIND, IO, 192>, grid, s, a);
    case 256: return launch(append_kernel<KIND, IO, 256>, grid, s, a);
    }
    return cudaErrorInvalidValue;
}

template <Kind KIND>
cudaError_t append_for_io(const AppendArgs &a, dim3 grid, cudaStream_t s)
{
    switch (a.dtype) {
    case QMM_F32: return append_for_dim<KIND, float>(a, grid, s);
    case QMM_F16: return append_for_dim<KIND, __half>(a, grid, s);
    case QMM_BF16: return append_for_dim<KIND, __nv_bfloat16>(a, grid, s);
    }
    return cudaErrorInvalidValue;
}

template <Kind KIND>
cudaError_t read_for_io(const KvReadArgs &a, dim3 grid, cudaStream_t s)
{
    switch (a.dtype) {
    case QMM_F32: return launch(read_kernel<KIND, float>, grid, s, a);
    case QMM_F16: return launch(read_kernel<KIND, __half>, grid, s, a);
    case QMM_BF16: return launch(read_kernel<KIND, __nv_bfloat16>, grid, s, a);
    }
    return cudaErrorInvalidValue;
}

} // namespace

cudaError_t launch_kv_append(const AppendArgs &a, int sm_count, cudaStream_t s)
{
    // Few tokens: a block takes as few heads as keep about four blocks on
    // every SM; from there on a block takes the whole token.
    const int rpw = a.c.D <= 64 ? 2 : 1;
    const int passes = (a.n_q + 2 * a.c.n_heads + kWarps * rpw - 1) / (kWarps * rpw);
    const int64_t parts = std::max<int64_t>(1, std::min<int64_t>(passes, 4 * sm_count / a.T));
    const dim3 grid(unsigned(a.T), unsigned(parts));
    switch (a.type) {
    case QMM_F16: return append_for_io<kF16>(a, grid, s);
    case QMM_BF16: return append_for_io<kBF16>(a, grid, s);
    default: return append_for_io<kQ8>(a, grid, s);
    }
}

cudaError_t launch_kv_read(const KvReadArgs &a, int sm_count, cudaStream_t s)
{
    const int64_t n = a.T * a.c.n_heads * (a.c.D / 4);
    const int64_t want = (n + kThreads - 1) / kThreads;
    const dim3 grid(unsigned(std::min<int64_t>(want, int64_t(sm_count) * 16)));
    switch (a.type) {
    case QMM_F16: return read_for_io<kF16>(a, grid, s);
    case QMM_BF16: return read_for_io<kBF16>(a, grid, s);
    default: return read_for_io<kQ8>(a, grid, s);
    }
}

} // namespace qmm
