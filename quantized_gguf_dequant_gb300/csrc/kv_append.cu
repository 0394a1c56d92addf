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
// and sines are computed once into shared memory and serve all its heads,
// while the first rows' loads are already under way.  A lane holds its part of
// a row in registers before it stores any of it, so q_out may be q.  A Q8_0
// block of 32 values is eight lanes of fp32 or four of 16-bit values.
// Small blocks, many to an SM: a block lives for about 2 us, most of it waiting
// for its rows (256 threads instead of 64 took 24.5 us where these take 18.7).
// Measured on one GB300: 4096 tokens of 32 + 8 + 8 heads of 128, bf16, three axes,
// into f16: 18.6 us, 5.4 TB/s; 2011 tokens of fp32 into Q8_0 and back out: 20.9 us;
// 16 tokens: 2.4 us; reading 16384 tokens of 8 heads out of Q8_0 in bf16: 18.4 us,
// 5.6 TB/s; 301 tokens: 1.9 us.
#include <algorithm>
#include <cstring>
#include <type_traits>

#include "kv_cache.cuh"
#include "qmm_device.cuh"
#include "qmm_internal.h"

namespace qmm {

namespace {

constexpr int kThreads = 64, kWarps = kThreads / 32;  // of an append block
constexpr int kAppendBlocks = 14;  // resident blocks of an SM, at least (for the registers)
constexpr int kReadThreads = 256;

enum Kind { kF16, kBF16, kQ8 };

// 16 bytes of values.
template <typename IO>
struct Chunk {
    static constexpr int N = 16 / sizeof(IO);
    uint4 raw;
    __device__ __forceinline__ void load(const IO *p) { raw = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void values(float (&v)[N]) const
    {
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(IO) == 4) {
                v[i] = __uint_as_float(w[i]);
            } else {
                const float2 f = unpack2(w[i], IO());
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
    }
};

// N (4 or 8) values to consecutive places of a type.
template <int N, typename T>
__device__ __forceinline__ void store_values(T *p, const float (&v)[N])
{
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            *reinterpret_cast<float4 *>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    } else if constexpr (N == 8) {
        *reinterpret_cast<uint4 *>(p) =
            make_uint4(pack2(v[0], v[1], T()), pack2(v[2], v[3], T()), pack2(v[4], v[5], T()),
                       pack2(v[6], v[7], T()));
    } else {
        *reinterpret_cast<uint2 *>(p) =
            make_uint2(pack2(v[0], v[1], T()), pack2(v[2], v[3], T()));
    }
}

// A Q8_0 block of 32 values, N to a lane: scale = amax/127, code =
// rint(x / scale) in fp32.  Every lane of the warp calls it.
template <int N>
__device__ __forceinline__ void quantize(const float (&x)[N], uint32_t (&codes)[N / 4], float &d)
{
    constexpr int LANES = 32 / N;
    // The bits of |x| are in its order, a NaN's above infinity's.
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
        top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1)
        top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float amax = __uint_as_float(top);
    d = __fdiv_rn(amax, 127.f);
    const float inv = d > 0.f ? __fdiv_rn(1.f, d) : 0.f;
    // At 1.5 * 2^23 a float's spacing is 1: the sum rounds to the code, in its
    // low byte.  A block without a finite scale has codes of zero.
    const uint32_t keep = inv > 0.f ? 0xffffffffu : 0u;
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = __float_as_uint(__fadd_rn(__fmul_rn(x[i + j], inv), 12582912.f));
        codes[i / 4] = __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040),
                                   0x5410) & keep;
    }
}

// The token's cosines and sines, and where its rows go: slot's row of head 0,
// or -1 for a token that is not stored.
__device__ __forceinline__ void turns_of(const AppendArgs &P, int64_t tok, float2 *turn)
{
    for (int i = threadIdx.x; i < P.n_rot >> 1; i += kThreads) {
        int ax = 0;
        while (i >= P.axis_end[ax])
            ++ax;
        const float angle =
            __fmul_rn(float(P.pos[int64_t(ax) * P.T + tok]), __ldg(P.inv_freq + i));
        float sn, cn;
        sincosf(angle, &sn, &cn);
        turn[i] = make_float2(cn, sn);
    }
}
__device__ __forceinline__ int64_t row_of_slot(const AppendArgs &P, int64_t slot)
{
    const KvView &c = P.c;
    const bool stored = slot >= 0 && slot < int64_t(c.n_pages) * c.page_size;
    if (slot >= 0 && !stored && threadIdx.x == 0 && blockIdx.y == 0)
        atomicOr(P.status, kStatusBadSlotBit);
    if (!stored)
        return -1;
    const uint32_t page = uint32_t(uint64_t(slot) / uint32_t(c.page_size));
    return int64_t(page) * c.n_heads * c.page_size +
           (slot - int64_t(page) * c.page_size);
}

// N values of a k or v row, at element e, into the cache.  Every lane of the
// warp calls it (Q8_0 shuffles within each block's lanes).
template <Kind KIND, int N>
__device__ __forceinline__ void put(const KvView &c, bool isk, int64_t row, int D, int e,
                                    const float (&y)[N], bool write)
{
    uint8_t *dst = isk ? c.k : c.v;
    if constexpr (KIND == kQ8) {
        uint32_t codes[N / 4];
        float d;
        quantize<N>(y, codes, d);
        if (write) {
            if constexpr (N == 8)
                *reinterpret_cast<uint2 *>(dst + row * D + e) = make_uint2(codes[0], codes[1]);
            else
                *reinterpret_cast<uint32_t *>(dst + row * D + e) = codes[0];
            if (e % 32 == 0)
                static_cast<__half *>(isk ? c.ks : c.vs)[row * kv_scales_per_row(D) + e / 32] =
                    __float2half_rn(d);
        }
    } else if (write) {
        if constexpr (KIND == kF16)
            store_values<N>(reinterpret_cast<__half *>(dst) + row * D + e, y);
        else
            store_values<N>(reinterpret_cast<__nv_bfloat16 *>(dst) + row * D + e, y);
    }
}

// The usual shapes: a lane takes two chunks of a row that hold whole pairs
// between them, so that nothing is loaded twice and no element asks what it
// is: (u, u + half the rotated chunks) for halves, then consecutive chunks of
// what passes through; (u, u + half the row's chunks) for adjacent pairs.
template <Kind KIND, typename IO, int D>
__global__ void __launch_bounds__(kThreads, kAppendBlocks) append_kernel(const __grid_constant__ AppendArgs P)
{
    constexpr int N = Chunk<IO>::N;
    constexpr int LPR = D / N / 2;      // lanes per row
    constexpr int RPW = 32 / LPR;       // rows per warp
    constexpr int BATCH = 2;            // row groups under way at once
    __shared__ __align__(16) float2 turn[128];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t tok = blockIdx.x;
    const KvView &c = P.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = lane / LPR, u = lane % LPR;
    const int rows = P.n_q + 2 * c.n_heads;
    const int stride = int(gridDim.y) * kWarps * RPW;
    const int64_t slot = __ldg(P.slots + tok);
    const IO *const qs = static_cast<const IO *>(P.q) + tok * P.ldq;
    const IO *const ks = static_cast<const IO *>(P.k) + tok * P.ldk;
    const IO *const vs = static_cast<const IO *>(P.v) + tok * P.ldv;
    IO *const qd = static_cast<IO *>(P.q_out) + tok * P.ldqo;
    // the lane's two chunks (first elements), and whether they turn
    int ea, eb;
    bool turn_a, turn_b;
    const int hc = P.n_rot / 2 / N;  // chunks of half the rotated dims
    if (P.adjacent || hc == 0) {
        ea = u * N;
        eb = (u + LPR) * N;
        turn_a = ea < P.n_rot;
        turn_b = eb < P.n_rot;
    } else {
        const int rest = u - hc;
        ea = (rest < 0 ? u : 2 * hc + 2 * rest) * N;
        eb = (rest < 0 ? u + hc : 2 * hc + 2 * rest + 1) * N;
        turn_a = turn_b = rest < 0;
    }
    Chunk<IO> xa[BATCH], xb[BATCH];
    auto load = [&](int base) {
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int r = base + i * stride + sub;
            const IO *src = r < P.n_q ? qs + r * D
                            : r < P.n_q + c.n_heads ? ks + (r - P.n_q) * D
                                                    : vs + (r - P.n_q - c.n_heads) * D;
            if (sub < RPW && r < rows) {
                xa[i].load(src + ea);
                xb[i].load(src + eb);
            } else {
                xa[i].raw = xb[i].raw = make_uint4(0, 0, 0, 0);
            }
        }
    };
    int base = (int(blockIdx.y) * kWarps + warp) * RPW;
    load(base);
    turns_of(P, tok, turn);
    const int64_t row0 = row_of_slot(P, slot);
    __syncthreads();
    while (base < rows) {
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int r = base + i * stride + sub;
            const bool isq = r < P.n_q, isk = !isq && r < P.n_q + c.n_heads;
            const bool active = sub < RPW && r < rows;
            float a[N], b[N];
            xa[i].values(a);
            xb[i].values(b);
            if (isq || isk) {
                if (P.adjacent) {
                    auto pairs = [&](float (&x)[N], int e) {
                        const float4 *cs = reinterpret_cast<const float4 *>(turn + e / 2);
#pragma unroll
                        for (int j = 0; j < N; j += 4) {
                            const float4 w = cs[j / 4];
                            const float x0 = x[j], x1 = x[j + 1], x2 = x[j + 2], x3 = x[j + 3];
                            x[j] = __fsub_rn(__fmul_rn(x0, w.x), __fmul_rn(x1, w.y));
                            x[j + 1] = __fadd_rn(__fmul_rn(x1, w.x), __fmul_rn(x0, w.y));
                            x[j + 2] = __fsub_rn(__fmul_rn(x2, w.z), __fmul_rn(x3, w.w));
                            x[j + 3] = __fadd_rn(__fmul_rn(x3, w.z), __fmul_rn(x2, w.w));
                        }
                    };
                    if (turn_a)
                        pairs(a, ea);
                    if (turn_b)
                        pairs(b, eb);
                } else if (turn_a) {
                    const float4 *cs = reinterpret_cast<const float4 *>(turn + ea);
#pragma unroll
                    for (int j = 0; j < N; j += 2) {
                        const float4 w = cs[j / 2];
                        const float a0 = a[j], a1 = a[j + 1], b0 = b[j], b1 = b[j + 1];
                        a[j] = __fsub_rn(__fmul_rn(a0, w.x), __fmul_rn(b0, w.y));
                        b[j] = __fadd_rn(__fmul_rn(b0, w.x), __fmul_rn(a0, w.y));
                        a[j + 1] = __fsub_rn(__fmul_rn(a1, w.z), __fmul_rn(b1, w.w));
                        b[j + 1] = __fadd_rn(__fmul_rn(b1, w.z), __fmul_rn(a1, w.w));
                    }
                }
            }
            if (isq) {  // (a row's loads are in registers: q_out may be q)
                if (active) {
                    store_values<N>(qd + r * D + ea, a);
                    store_values<N>(qd + r * D + eb, b);
                }
            }
            // (Q8_0's blocks of 32 are neighbouring lanes' first, or second, chunks:
            // all lanes shuffle where any of the warp's rows is not q's)
            if (KIND == kQ8 ? base + i * stride + RPW > P.n_q : !isq) {
                const int head = isk ? r - P.n_q : r - P.n_q - c.n_heads;
                const int64_t row = row0 + int64_t(head) * c.page_size;
                const bool write = active && !isq && row0 >= 0;
                put<KIND, N>(c, isk, row, D, ea, a, write);
                put<KIND, N>(c, isk, row, D, eb, b, write);
            }
        }
        base += BATCH * stride;
        if (base < rows)
            load(base);
    }
}

// Any even number of rotated dims and any head size: a lane takes consecutive
// chunks of a row, which the warp passes through shared memory, where every
// chunk finds its partners.  A chunk is loaded and stored by the same lane, so
// q_out may be q.  4096 tokens of 32 + 8 + 8 heads of 128 in bf16, half of each
// rotated, into Q8_0 and back out: 31 us (append_kernel, all of each: 25); when
// every element looked up its partner in global memory: 81.
template <Kind KIND, typename IO, int PASSES>  // chunks of a lane in a row
__global__ void __launch_bounds__(kThreads, kAppendBlocks) append_any_kernel(const __grid_constant__ AppendArgs P)
{
    constexpr int N = Chunk<IO>::N;
    constexpr int BATCH = 4 / PASSES;  // row groups under way at once
    __shared__ __align__(16) float2 turn[128];
    __shared__ uint4 staged[kWarps][BATCH][PASSES * 32];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t tok = blockIdx.x;
    const KvView &c = P.c;
    const int D = c.D, half = P.n_rot >> 1, chunks = D / N;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rpw = max(1, 32 / chunks);  // rows of a warp
    const int sub = chunks < 32 ? lane / chunks : 0, u = lane - sub * chunks;
    const int rows = P.n_q + 2 * c.n_heads;
    const int stride = int(gridDim.y) * kWarps * rpw;
    const bool aligned = half % N == 0;  // a chunk's partners are a chunk
    const int64_t slot = __ldg(P.slots + tok);
    Chunk<IO> x[BATCH][PASSES];
    auto turned = [&](int r, int e) { return r < P.n_q + c.n_heads && e < P.n_rot; };
    auto load = [&](int base) {
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int r = base + i * stride + sub;
            const bool isq = r < P.n_q, isk = !isq && r < P.n_q + c.n_heads;
            const int head = isq ? r : (isk ? r - P.n_q : r - P.n_q - c.n_heads);
            const IO *src = static_cast<const IO *>(isq ? P.q : (isk ? P.k : P.v)) +
                            tok * (isq ? P.ldq : (isk ? P.ldk : P.ldv)) + head * D;
#pragma unroll
            for (int p = 0; p < PASSES; ++p) {
                const int e = (p * 32 + u) * N;
                x[i][p].raw = make_uint4(0, 0, 0, 0);
                if (sub < rpw && r < rows && e < D)
                    x[i][p].load(src + e);
            }
        }
    };
    int base = (int(blockIdx.y) * kWarps + warp) * rpw;
    load(base);
    turns_of(P, tok, turn);
    const int64_t row0 = row_of_slot(P, slot);
    __syncthreads();
    while (base < rows) {
        if (!P.adjacent && half > 0) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < BATCH; ++i)
#pragma unroll
                for (int p = 0; p < PASSES; ++p)
                    staged[warp][i][p * 32 + lane] = x[i][p].raw;
            __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int r = base + i * stride + sub;
            const bool isq = r < P.n_q, isk = !isq && r < P.n_q + c.n_heads;
            const IO *row = reinterpret_cast<const IO *>(staged[warp][i] + (lane - u));
            const int head = isq ? r : (isk ? r - P.n_q : r - P.n_q - c.n_heads);
#pragma unroll
            for (int p = 0; p < PASSES; ++p) {
                const int e = (p * 32 + u) * N;
                const bool active = sub < rpw && r < rows && e < D;
                float y[N];
                x[i][p].values(y);
                if (active && turned(r, e)) {
                    float o[N];  // the partners
                    if (P.adjacent) {
#pragma unroll
                        for (int j = 0; j < N; ++j)
                            o[j] = y[j ^ 1];
                    } else if (aligned) {
                        Chunk<IO> other;
                        other.load(row + (e < half ? e + half : e - half));
                        other.values(o);
                    } else {
#pragma unroll
                        for (int j = 0; j < N; ++j) {
                            const int d = e + j;
                            o[j] = load1(row + (d < half ? d + half : max(d - half, 0)));
                        }
                    }
                    if (!P.adjacent && aligned) {
                        const bool second = e >= half;
                        const float sign = second ? 1.f : -1.f;
                        const float4 *cs =
                            reinterpret_cast<const float4 *>(turn + (second ? e - half : e));
#pragma unroll
                        for (int j = 0; j < N; j += 2) {
                            const float4 w = cs[j / 2];
                            y[j] = __fadd_rn(__fmul_rn(y[j], w.x), __fmul_rn(o[j], sign * w.y));
                            y[j + 1] =
                                __fadd_rn(__fmul_rn(y[j + 1], w.z), __fmul_rn(o[j + 1], sign * w.w));
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < N; ++j) {
                            if (e + j >= P.n_rot)
                                continue;
                            const bool second = P.adjacent ? (j & 1) : e + j >= half;
                            const float2 w =
                                turn[P.adjacent ? (e + j) >> 1 : (second ? e + j - half : e + j)];
                            const float b = __fmul_rn(o[j], w.y);
                            const float a = __fmul_rn(y[j], w.x);
                            y[j] = second ? __fadd_rn(a, b) : __fsub_rn(a, b);
                        }
                    }
                }
                if (isq && active)
                    store_values<N>(static_cast<IO *>(P.q_out) + tok * P.ldqo + head * D + e, y);
                // (Q8_0: all lanes shuffle where any of the warp's rows is not q's)
                if (KIND == kQ8 ? base + i * stride + rpw > P.n_q : !isq)
                    put<KIND, N>(c, isk, row0 + int64_t(head) * c.page_size, D, e, y,
                                 active && !isq && row0 >= 0);
            }
        }
        base += BATCH * stride;
        if (base < rows)
            load(base);
    }
}

// Rows of the cache as values.  A block takes a few consecutive tokens: it
// finds their rows once, then every thread asks for all its chunks of k and of
// v before it converts the first.  A chunk is what 16 bytes of output hold.
constexpr int kReadTokens = 64;  // of a block, at most
constexpr int kReadUnits = 4;    // chunks of a thread under way at once

template <Kind KIND, typename IO>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const __grid_constant__ KvReadArgs P)
{
    constexpr int N = Chunk<IO>::N;
    using H = typename std::conditional<KIND == kBF16, __nv_bfloat16, __half>::type;
    __shared__ uint32_t row_of[kReadTokens];  // row of head 0; ~0 for none
    pdl_wait();
    pdl_launch_dependents();
    const KvView &c = P.c;
    const int D = c.D, SP = kv_scales_per_row(D);
    const int64_t tok0 = int64_t(blockIdx.x) * P.tokens;
    const int n = int(min(int64_t(P.tokens), P.T - tok0));
    if (int(threadIdx.x) < n) {
        const int64_t slot = __ldg(P.slots + tok0 + threadIdx.x);
        const bool held = slot >= 0 && slot < int64_t(c.n_pages) * c.page_size;
        if (slot >= 0 && !held)
            atomicOr(P.status, kStatusBadSlotBit);
        uint32_t row = ~0u;
        if (held) {
            const uint32_t page = slot < 0x7fffffff
                                      ? fast_div(c.page, uint32_t(slot))
                                      : uint32_t(uint64_t(slot) / uint32_t(c.page_size));
            row = page * uint32_t(c.n_heads) * uint32_t(c.page_size) +
                  uint32_t(slot - int64_t(page) * c.page_size);
        }
        row_of[threadIdx.x] = row;
    }
    __syncthreads();
    const int units = n * int(P.unit.d);
    for (int i0 = threadIdx.x; i0 < units; i0 += kReadUnits * kReadThreads) {
        uint2 raw[2][kReadUnits] = {};  // 4 or 8 codes, or 4 values of 16 bits
        uint2 more[2][kReadUnits] = {}; // 8 values of 16 bits: the second half
        __half scale[2][kReadUnits];
        int64_t at[kReadUnits];         // token
        int off[kReadUnits];            // element within the token
        bool held[kReadUnits];
#pragma unroll
        for (int u = 0; u < kReadUnits; ++u) {
            const int i = min(i0 + u * kReadThreads, units - 1);
            const int t = int(fast_div(P.unit, unsigned(i)));
            const int in = i - t * int(P.unit.d);
            const int head = int(fast_div(P.chunk, unsigned(in)));
            const int e = (in - head * int(P.chunk.d)) * N;
            const uint32_t row0 = row_of[t];
            held[u] = row0 != ~0u;
            at[u] = tok0 + t;
            off[u] = head * D + e;
            const uint64_t row =
                held[u] ? uint64_t(row0) + unsigned(head) * unsigned(c.page_size) : 0;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                if (!(w ? P.v : P.k))
                    continue;
                const uint8_t *src = w ? c.v : c.k;
                if constexpr (KIND == kQ8) {
                    if constexpr (N == 8)
                        raw[w][u] = __ldg(reinterpret_cast<const uint2 *>(src + row * D + e));
                    else
                        raw[w][u].x = __ldg(reinterpret_cast<const uint32_t *>(src + row * D + e));
                    scale[w][u] =
                        __ldg(static_cast<const __half *>(w ? c.vs : c.ks) + row * SP + e / 32);
                } else {
                    const H *p = reinterpret_cast<const H *>(src) + row * D + e;
                    if constexpr (N == 8) {
                        const uint4 q = __ldg(reinterpret_cast<const uint4 *>(p));
                        raw[w][u] = make_uint2(q.x, q.y);
                        more[w][u] = make_uint2(q.z, q.w);
                    } else {
                        raw[w][u] = __ldg(reinterpret_cast<const uint2 *>(p));
                    }
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kReadUnits; ++u) {
            if (i0 + u * kReadThreads >= units)
                continue;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                IO *out = static_cast<IO *>(w ? P.v : P.k);
                if (!out)
                    continue;
                float v[N];
                const uint32_t q[4] = {raw[w][u].x, raw[w][u].y, more[w][u].x, more[w][u].y};
                if constexpr (KIND == kQ8) {
                    const float d = __half2float(scale[w][u]);
#pragma unroll
                    for (int j = 0; j < N; ++j)
                        v[j] = float(int(int8_t(q[j / 4] >> (8 * (j & 3))))) * d;
                } else {
#pragma unroll
                    for (int j = 0; j < N; j += 2) {
                        const float2 f = unpack2(q[j / 2], H());
                        v[j] = f.x;
                        v[j + 1] = f.y;
                    }
                }
                if (!held[u]) {
#pragma unroll
                    for (int j = 0; j < N; ++j)
                        v[j] = 0.f;
                }
                store_values<N>(out + at[u] * (w ? P.ldv : P.ldk) + off[u], v);
            }
        }
    }
}

template <typename Args>
cudaError_t launch(void (*k)(Args), dim3 grid, int threads, cudaStream_t s, const Args &a)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(unsigned(threads));
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
    return counted(cudaLaunchKernelEx(&cfg, k, a));
}

// Whether append_kernel's lanes hold whole pairs, and whole Q8_0 blocks are
// neighbouring lanes.
template <Kind KIND, int N>
bool append_regular(const AppendArgs &a)
{
    const int D = a.c.D;
    if (a.adjacent ? a.n_rot % N != 0 : a.n_rot % (2 * N) != 0)
        return false;
    if (KIND != kQ8)
        return true;
    return D % 64 == 0 && (a.adjacent || a.n_rot == 0 || a.n_rot == D);
}

template <Kind KIND, typename IO>
cudaError_t append_for_dim(const AppendArgs &a, int sm_count, cudaStream_t s)
{
    constexpr int N = Chunk<IO>::N;
    const bool regular = append_regular<KIND, N>(a);
    // Few tokens: a block takes as few heads as keep about four blocks on
    // every SM; from there on a block takes the whole token.
    // rows of a block at a time
    const int rows = kWarps * (regular ? 32 / (a.c.D / N / 2) : std::max(1, 32 / (a.c.D / N)));
    const int passes = (a.n_q + 2 * a.c.n_heads + rows - 1) / rows;
    const int64_t parts = std::max<int64_t>(1, std::min<int64_t>(passes, 4 * sm_count / a.T));
    const dim3 grid(unsigned(a.T), unsigned(parts));
    if (!regular)
        return launch(N == 4 && a.c.D > 128 ? append_any_kernel<KIND, IO, N == 4 ? 2 : 1>
                                            : append_any_kernel<KIND, IO, 1>,
                      grid, kThreads, s, a);
    switch (a.c.D) {
    case 64: return launch(append_kernel<KIND, IO, 64>, grid, kThreads, s, a);
    case 96:
        if constexpr (KIND != kQ8)  // (there append_regular says no)
            return launch(append_kernel<KIND, IO, 96>, grid, kThreads, s, a);
        break;
    case 128: return launch(append_kernel<KIND, IO, 128>, grid, kThreads, s, a);
    case 192: return launch(append_kernel<KIND, IO, 192>, grid, kThreads, s, a);
    case 256: return launch(append_kernel<KIND, IO, 256>, grid, kThreads, s, a);
    }
    return cudaErrorInvalidValue;
}

template <Kind KIND>
cudaError_t append_for_io(const AppendArgs &a, int sm_count, cudaStream_t s)
{
    switch (a.dtype) {
    case QMM_F32: return append_for_dim<KIND, float>(a, sm_count, s);
    case QMM_F16: return append_for_dim<KIND, __half>(a, sm_count, s);
    case QMM_BF16: return append_for_dim<KIND, __nv_bfloat16>(a, sm_count, s);
    }
    return cudaErrorInvalidValue;
}

template <Kind KIND>
cudaError_t read_for_io(const KvReadArgs &a, dim3 grid, cudaStream_t s)
{
    switch (a.dtype) {
    case QMM_F32: return launch(read_kernel<KIND, float>, grid, kReadThreads, s, a);
    case QMM_F16: return launch(read_kernel<KIND, __half>, grid, kReadThreads, s, a);
    case QMM_BF16: return launch(read_kernel<KIND, __nv_bfloat16>, grid, kReadThreads, s, a);
    }
    return cudaErrorInvalidValue;
}

} // namespace

cudaError_t launch_kv_append(const AppendArgs &a, int sm_count, cudaStream_t s)
{
    switch (a.type) {
    case QMM_F16: return append_for_io<kF16>(a, sm_count, s);
    case QMM_BF16: return append_for_io<kBF16>(a, sm_count, s);
    default: return append_for_io<kQ8>(a, sm_count, s);
    }
}

cudaError_t launch_kv_read(const KvReadArgs &args, int sm_count, cudaStream_t s)
{
    KvReadArgs a = args;
    const int n = a.dtype == QMM_F32 ? 4 : 8;                    // values of a chunk
    const int64_t units = int64_t(a.c.n_heads) * (a.c.D / n);    // of a token
    a.unit = make_fast_div(uint32_t(units));
    a.chunk = make_fast_div(uint32_t(a.c.D / n));
    // tokens of a block: what its threads ask for at once, fewer while there
    // are SMs without a block
    a.tokens = int(std::max<int64_t>(
        1, std::min({int64_t(kReadUnits * kReadThreads) / units, (a.T + 4 * sm_count - 1) / (4 * sm_count),
                     int64_t(kReadTokens)})));
    const dim3 grid(unsigned((a.T + a.tokens - 1) / a.tokens));
    switch (a.type) {
    case QMM_F16: return read_for_io<kF16>(a, grid, s);
    case QMM_BF16: return read_for_io<kBF16>(a, grid, s);
    default: return read_for_io<kQ8>(a, grid, s);
    }
}

} // namespace qmm
