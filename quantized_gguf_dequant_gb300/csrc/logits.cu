// logits.cu -- a model's logits adjusted before sampling: penalties for
// repeated tokens, biases, and a mask of what a grammar allows, in one launch.
//
//   c = times v occurs in the row's history
//   z = logits[v];  c > 0:  z = z > 0 ? z / r : z * r;  z -= presence + frequency * c
//   z += the row's biases for v, added in list order
//   bit v of the row's mask clear:  z = -inf
// all in fp32, rounded once to the logits' type.
//
// Bytes bound it: each logit is read and written once.  A block takes a part
// of a row.  First it streams the part from input to output, 16 bytes a lane,
// under the mask alone; a call in place without a mask skips this, and its
// time no longer depends on the vocabulary's size.  Few logits are named by
// the history or a bias (a thousand or two of a hundred thousand), so these are
// done on their own: a bitmap of the part's named tokens, counts by their rank
// in it (whole-number atomics: no order to matter), then one thread a token,
// which computes from the input.  Testing every logit against dense counts
// instead takes three times the instructions of the stream itself and was
// bound by issuing them (256 rows of 128256 logits: 67 us).
// Measured on one GB300: those rows with 1000-2000 tokens of history, 100 biases
// and a mask each: 56 us, 4.8 TB/s (41.5 us, 6.3 TB/s, without lists); one row: 3.8 us.
// A bias list may name a token twice: then one warp walks the list and adds in
// its order, so the sum is repeatable and the time follows the list's length (4
// rows of 128256, 30000 entries each that name 15000 tokens: 0.23 ms, without
// repetitions 0.06; when each token's owner searched the rest of the list: 10).
// Groups are taken at their 16-byte boundaries whatever the row's own
// alignment, so an odd vocabulary costs nothing but its ragged ends.
#include <algorithm>
#include <type_traits>

#include "kv_cache.cuh"
#include "qmm_device.cuh"
#include "qmm_internal.h"

namespace qmm {

namespace {

constexpr int kThreads = 256;
constexpr int kResident = 5;       // blocks of an SM
constexpr int kLongest = 16384;    // logits of a part, at most
// History tokens that a thread keeps in registers from before the stream on; longer
// lists are read again in each phase.  256 rows of 128256 with up to 500, 1000, 2000
// and 4000 tokens: 52.5, 53.7, 56.9 and 72 us; with four 50.5, 51.7, 59.0 and 74;
// with two 54, 57, 63 and 79; with twelve 56, 57, 60 and 73.
constexpr int kAhead = 8;
constexpr int kPlaces = 1024;      // named tokens counted at once
constexpr uint32_t kNoOwner = 0xffffffffu;

__device__ __forceinline__ int64_t clamp64(int64_t v, int64_t hi)
{
    return v < 0 ? 0 : (v > hi ? hi : v);
}

// 32 mask bits from bit v on (those past the vocabulary are of no matter).
__device__ __forceinline__ uint32_t mask_bits(const uint32_t *mask, int v, int V)
{
    const int w = v >> 5, s = v & 31;
    const uint32_t lo = __ldg(mask + w);
    const uint32_t hi = s && (w + 1) * 32 < V ? __ldg(mask + w + 1) : 0u;
    return __funnelshift_r(lo, hi, s);
}

// The block's part [lo, hi) of a row from `in` to `out` under the mask.  VEC:
// both rows are equally misaligned and lo is 0 or at a 16-byte boundary.
template <typename IO, bool VEC>
__device__ __forceinline__ void stream_part(const IO *in, IO *out, const uint32_t *mask, int lo,
                                            int hi, int V)
{
    constexpr int N = 16 / sizeof(IO), DEEP = 4;
    const int tid = threadIdx.x;
    auto one = [&](int v) {
        float z = load1(in + v);
        if (mask && !(mask_bits(mask, v, V) & 1u))
            z = -INFINITY;
        store1(out + v, z);
    };
    if (!VEC) {
        for (int v = lo + tid; v < hi; v += kThreads)
            one(v);
        return;
    }
    const int head = min(hi, lo + int((-(reinterpret_cast<uintptr_t>(in + lo) / sizeof(IO))) & (N - 1)));
    const int groups = (hi - head) / N;
    if (lo + tid < head)
        one(lo + tid);
    if (head + groups * N + tid < hi)
        one(head + groups * N + tid);
    const uint4 *src = reinterpret_cast<const uint4 *>(in + head);
    uint4 *dst = reinterpret_cast<uint4 *>(out + head);
    const bool odd = head % N != 0;  // groups may reach into a second mask word
    for (int g0 = tid; g0 < groups; g0 += DEEP * kThreads) {
        uint4 x[DEEP];
        uint32_t word[DEEP], next[DEEP];
#pragma unroll
        for (int i = 0; i < DEEP; ++i)
            x[i] = __ldcs(src + min(g0 + i * kThreads, groups - 1));
        if (mask) {
#pragma unroll
            for (int i = 0; i < DEEP; ++i)
                word[i] = __ldg(mask + ((head + min(g0 + i * kThreads, groups - 1) * N) >> 5));
            if (odd) {
#pragma unroll
                for (int i = 0; i < DEEP; ++i)
                    next[i] = __ldg(
                        mask + ((head + min(g0 + i * kThreads, groups - 1) * N + N - 1) >> 5));
            }
        }
#pragma unroll
        for (int i = 0; i < DEEP; ++i) {
            if (g0 + i * kThreads >= groups)
                break;
            if (mask) {
                const int s = (head + (g0 + i * kThreads) * N) & 31;
                const uint32_t bits = odd ? __funnelshift_r(word[i], next[i], s) : word[i] >> s;
                uint32_t *w = reinterpret_cast<uint32_t *>(&x[i]);
                if constexpr (N == 4) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        w[j] = bits & (1u << j) ? w[j] : 0xff800000u;
                } else {
                    constexpr uint32_t inf = std::is_same<IO, __half>::value ? 0xfc00u : 0xff80u;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t keep = (bits & (1u << (2 * j)) ? 0xffffu : 0u) |
                                              (bits & (2u << (2 * j)) ? 0xffff0000u : 0u);
                        w[j] = (w[j] & keep) | ((inf | inf << 16) & ~keep);
                    }
                }
            }
            dst[g0 + i * kThreads] = x[i];
        }
    }
}

// One warp adds up the biases [b0, b1) of every place in list order: 32 entries
// at a time, of which the first of each place takes the others' values in turn.
// owner: each place's first entry.
template <typename Place>
__device__ __forceinline__ void add_in_order(const LogitsArgs &P, int64_t b0, int64_t b1,
                                             const uint32_t *owner, float *sums, Place place)
{
    constexpr int DEEP = 4;
    const int lane = threadIdx.x & 31;
    for (int64_t i0 = b0; i0 < b1; i0 += 32 * DEEP) {
        int token[DEEP];
#pragma unroll
        for (int j = 0; j < DEEP; ++j) {
            const int64_t i = i0 + j * 32 + lane;
            token[j] = i < b1 ? __ldg(P.bias_ids + i) : -1;
        }
#pragma unroll
        for (int j = 0; j < DEEP; ++j) {
            const int64_t i = i0 + j * 32 + lane;
            const uint32_t p = place(token[j]);
            const bool in = p < uint32_t(kPlaces);
            if (!__any_sync(0xffffffffu, in))
                continue;
            const float value = in ? __ldg(P.bias_values + i) : 0.f;
            const unsigned same = __match_any_sync(0xffffffffu, in ? p : uint32_t(kPlaces) + lane);
            const bool first = in && lane == __ffs(same) - 1;
            float sum = value;
            if (first && owner[p] != uint32_t(i - b0))
                sum = __fadd_rn(sums[p], value);
            unsigned rest = first ? same & (same - 1) : 0u;
            while (__any_sync(0xffffffffu, rest)) {
                const float v = __shfl_sync(0xffffffffu, value, rest ? __ffs(rest) - 1 : lane);
                sum = rest ? __fadd_rn(sum, v) : sum;
                rest &= rest - 1;
            }
            if (first)
                sums[p] = sum;
            __syncwarp();
        }
    }
}

template <typename IO, bool VEC>
__global__ void __launch_bounds__(kThreads, kResident) adjust_kernel(const __grid_constant__ LogitsArgs P)
{
    constexpr int N = 16 / sizeof(IO);
    extern __shared__ __align__(16) uint32_t shared[];
    __shared__ uint32_t warp_sum_[kThreads / 32];
    __shared__ int twice;  // the bias list names a token twice
    uint32_t *bitmap = shared, *before = shared + P.words;   // named tokens; those of earlier words
    uint32_t *counts = before + P.words, *owner = counts + kPlaces, *ids = owner + kPlaces;
    float *sums = reinterpret_cast<float *>(ids + kPlaces);  // of the places' biases
    const int tid = threadIdx.x, lane = tid & 31, V = int(P.V);  // (n_vocab <= 2^26)
    pdl_wait();
    pdl_launch_dependents();
    const int64_t b = blockIdx.x / unsigned(P.parts);
    const int rank = int(blockIdx.x % unsigned(P.parts));
    const IO *in = static_cast<const IO *>(P.in) + b * P.ld_in;
    IO *out = static_cast<IO *>(P.out) + b * P.ld_out;
    const uint32_t *mask = P.mask ? P.mask + b * P.ld_mask : nullptr;
    // parts end at 16-byte boundaries
    const int shift = VEC ? int((reinterpret_cast<uintptr_t>(in) / sizeof(IO)) & (N - 1)) : 0;
    const int lo = min(V, max(0, rank * P.part - shift));
    const int hi = rank + 1 == P.parts ? V : min(V, max(0, (rank + 1) * P.part - shift));

    int64_t h0 = 0, h1 = 0, b0 = 0, b1 = 0;
    if (P.n_history > 0) {
        h0 = clamp64(__ldg(P.history_offsets + b), P.n_history);
        h1 = clamp64(__ldg(P.history_offsets + b + 1), P.n_history);
    }
    if (P.n_biases > 0) {
        b0 = clamp64(__ldg(P.bias_offsets + b), P.n_biases);
        b1 = clamp64(__ldg(P.bias_offsets + b + 1), P.n_biases);
    }
    // the lists' first tokens are on their way while the part is streamed
    int held[kAhead], held_bias = -1;
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
        held[j] = h0 + tid + j * kThreads < h1 ? __ldg(P.history + h0 + tid + j * kThreads) : -1;
    if (b0 + tid < b1)
        held_bias = __ldg(P.bias_ids + b0 + tid);
    const bool in_place = P.in == P.out;
    if (!in_place || mask)
        stream_part<IO, VEC>(in, out, mask, lo, hi, V);
    if (h0 >= h1 && b0 >= b1)
        return;  // (the row's other blocks do the same)
    const float r = P.repeat ? __ldg(P.repeat + b) : 1.f;
    const float presence = P.presence ? __ldg(P.presence + b) : 0.f;
    const float frequency = P.frequency ? __ldg(P.frequency + b) : 0.f;

    // f(token) for the history, f(token, entry) for the biases
    auto each_said = [&](auto f) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            f(held[j]);
#pragma unroll 4
        for (int64_t i = h0 + tid + kAhead * kThreads; i < h1; i += kThreads)
            f(__ldg(P.history + i));
    };
    auto each_bias = [&](auto f) {
        f(held_bias, uint32_t(tid));
        for (int64_t i = b0 + tid + kThreads; i < b1; i += kThreads)
            f(__ldg(P.bias_ids + i), uint32_t(i - b0));
    };
    const int span = hi - lo, words = (span + 31) / 32;  // (the bitmap holds a part)
    // A short part counts at the tokens' own places instead of their ranks.
    const bool direct = span <= kPlaces;
    uint32_t total = uint32_t(span);
    if (tid == 0)
        twice = 0;
    if (!direct) {
        for (int i = tid; i < words; i += kThreads)
            bitmap[i] = 0u;
        __syncthreads();
        auto note = [&](int token) {
            const unsigned at = unsigned(token) - unsigned(lo);
            if (token >= 0 && at < unsigned(span))
                atomicOr(bitmap + (at >> 5), 1u << (at & 31));
        };
        each_said(note);
        each_bias([&](int token, uint32_t) { note(token); });
        __syncthreads();
        // ranks: a thread takes `run` consecutive words
        const int run = (words + kThreads - 1) / kThreads;
        uint32_t mine = 0;
        for (int k = 0; k < run; ++k) {
            const int i = tid * run + k;
            if (i < words) {
                before[i] = mine;
                mine += __popc(bitmap[i]);
            }
        }
        uint32_t upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
            upto += lane >= o ? v : 0u;
        }
        if (lane == 31)
            warp_sum_[tid >> 5] = upto;
        __syncthreads();
        total = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            upto += w < (tid >> 5) ? warp_sum_[w] : 0u;
            total += warp_sum_[w];
        }
        for (int k = 0; k < run; ++k)
            if (tid * run + k < words)
                before[tid * run + k] += upto - mine;
    }
    // named tokens by rank, kPlaces at a time
    for (uint32_t first = 0; first < total; first += kPlaces) {
        const uint32_t n = min(uint32_t(kPlaces), total - first);
        for (uint32_t i = tid; i < n; i += kThreads) {
            counts[i] = 0u;
            owner[i] = kNoOwner;
        }
        __syncthreads();
        auto place = [&](int token) {  // its place, or kPlaces and more
            const unsigned at = unsigned(token) - unsigned(lo);
            if (token < 0 || at >= unsigned(span))
                return uint32_t(kPlaces);
            if (direct)
                return at;
            return before[at >> 5] + __popc(bitmap[at >> 5] & ((1u << (at & 31)) - 1u)) - first;
        };
        each_said([&](int token) {
            const uint32_t p = place(token);
            if (p < kPlaces) {
                atomicAdd(counts + p, 1u);
                ids[p] = token;
            }
        });
        each_bias([&](int token, uint32_t i) {
            const uint32_t p = place(token);
            if (p < kPlaces) {
                ids[p] = token;
                if (atomicMin(owner + p, i) != kNoOwner)
                    twice = 1;
            }
        });
        __syncthreads();
        const bool again = twice;
        if (again) {  // in list order by the first warp
            if (tid < 32)
                add_in_order(P, b0, b1, owner, sums, place);
            __syncthreads();
        }
        for (uint32_t p = tid; p < n; p += kThreads) {
            const uint32_t c = counts[p], first_bias = owner[p];
            if (direct && c == 0 && first_bias == kNoOwner)
                continue;
            const int token = direct ? lo + int(p) : int(ids[p]);
            float z = load1(in + token);
            const bool banned = mask && !(mask_bits(mask, token, V) & 1u);
            if (c) {
                z = z > 0.f ? __fdiv_rn(z, r) : __fmul_rn(z, r);
                z = __fsub_rn(z, __fadd_rn(presence, __fmul_rn(frequency, float(c))));
            }
            if (first_bias != kNoOwner)
                z = __fadd_rn(z, again ? sums[p] : __ldg(P.bias_values + b0 + first_bias));
            store1(out + token, banned ? -INFINITY : z);
        }
        __syncthreads();
    }
}

template <typename IO, bool VEC>
cudaError_t launch(LogitsArgs a, int sm_count, cudaStream_t s)
{
    constexpr int N = 16 / sizeof(IO);
    const auto kern = adjust_kernel<IO, VEC>;
    const LogitsPlan plan = plan_logits(a.B, a.V, int(sizeof(IO)), sm_count);
    a.parts = plan.parts;
    a.part = plan.part;
    a.words = (a.part + N + 31) / 32 + 1;
    const bool named = a.n_history > 0 || a.n_biases > 0;
    const size_t smem =
        named ? (size_t(a.words) * 2 + kPlaces * (a.n_biases > 0 ? 4 : 3)) * 4 : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(a.B * a.parts));
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
    const bool vec =
        (reinterpret_cast<uintptr_t>(a.in) - reinterpret_cast<uintptr_t>(a.out)) % 16 == 0 &&
        (a.B == 1 || uint64_t(a.ld_in - a.ld_out) * sizeof(IO) % 16 == 0);
    return vec ? launch<IO, true>(a, sm_count, s) : launch<IO, false>(a, sm_count, s);
}

} // namespace

// Every block of a row scans its lists: as few parts as hold kLongest logits
// at most, then what fills the last wave of resident blocks (30 rows of 128256
// in bf16 with 2000 tokens: 9.9 us, with halved parts until each SM had four
// blocks 12.3; 8 rows in fp32 with 500: 7.0 and 8.1).
LogitsPlan plan_logits(int64_t B, int64_t V, int bytes, int sm_count)
{
    const int n = 16 / bytes;
    const int64_t fewest = (V + kLongest - 1) / kLongest, slots = int64_t(kResident) * sm_count;
    const int64_t waves = (B * fewest + slots - 1) / slots;
    LogitsPlan p;
    p.parts = int(std::max(fewest, std::min(waves * slots / B, (V + 1023) / 1024)));
    p.part = int((V + n + p.parts - 1) / p.parts + n - 1) / n * n;
    p.at_once = kPlaces;
    return p;
}

cudaError_t launch_logits_adjust(const LogitsArgs &a, int sm_count, cudaStream_t s)
{
    switch (a.dtype) {
    case QMM_F32: return launch_io<float>(a, sm_count, s);
    case QMM_F16: return launch_io<__half>(a, sm_count, s);
    default: return launch_io<__nv_bfloat16>(a, sm_count, s);
    }
}

} // namespace qmm
