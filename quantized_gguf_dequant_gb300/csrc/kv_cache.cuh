// kv_cache.cuh -- the paged key-value cache as the device sees it, and the
// small conversions its kernels (kv_append.cu, attn_decode.cu) share.
//
// One buffer holds keys, another of the same layout values:
//   F16, BF16: [page][kv head][slot of the page][head_dim]
//   Q8_0: int8 codes [page][kv head][slot][head_dim], followed (after the
//         last page's codes) by fp16 scales [page][kv head][slot][SP],
//         SP = head_dim/32 rounded up to even; element d of a row stands for
//         code[d] * scale[d/32].  GGUF's Q8_0 block (one scale, 32 codes) with
//         the scales in a plane of their own, so that every row of codes
//         starts on a 16-byte boundary.
// One head's rows of a page are contiguous: what one attention block streams.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qmm_internal.h"

namespace qmm {

// n / d for 0 <= n < 2^31 by one high product, after Granlund and Montgomery,
// "Division by Invariant Integers using Multiplication" (1994):
// q = (umulhi(mul, n) + n) >> shift.
__device__ __forceinline__ uint32_t fast_div(const FastDiv &f, uint32_t n)
{
    return (__umulhi(f.mul, n) + n) >> f.shift;
}

__host__ __device__ constexpr int kv_scales_per_row(int D) { return (D / 32 + 1) / 2 * 2; }

// ------------------------------------------------------------------ 4 values
__device__ __forceinline__ float4 load4(const float *p)
{
    return *reinterpret_cast<const float4 *>(p);
}
__device__ __forceinline__ float4 load4(const __half *p)
{
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&u.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&u.y));
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p)
{
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                       __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ float load1(const __half *p) { return __half2float(*p); }
__device__ __forceinline__ float load1(const __nv_bfloat16 *p) { return __bfloat162float(*p); }

__device__ __forceinline__ uint32_t pack2(float a, float b, __half)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 unpack2(uint32_t u, __half)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&u));
}
__device__ __forceinline__ float2 unpack2(uint32_t u, __nv_bfloat16)
{
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ void store4(float *p, float4 v)
{
    *reinterpret_cast<float4 *>(p) = v;
}
template <typename H>
__device__ __forceinline__ void store4(H *p, float4 v)
{
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack2(v.x, v.y, H()), pack2(v.z, v.w, H()));
}
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void store1(__half *p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void store1(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

} // namespace qmm
