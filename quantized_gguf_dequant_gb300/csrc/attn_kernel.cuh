// attn_kernel.cuh -- attention of one new token per sequence over the paged
// key-value cache, split over the cache's length and joined.
//
//   s_j = scale q.k_j;  capped: cap tanh(s/cap);  + slope_h (j - (len-1))
//   out = sum_j softmax(s)_j v_j,  lse = ln sum_j exp(s_j),
//   j over the keys in [max(0, len - window), len)
//
// One pass over the cache with a running maximum m and sum l (base 2): a tile
// of 16 or 32 keys rescales what was gathered by 2^(m_old - m_new).
//
// What bounds it: the cache bytes, and around them the latency of a call's
// start and end.  Every key and value is read once for the query heads that
// share it and used for 4 flops a head, far below what the tensor cores take,
// so the design is about keeping enough loads in flight.  Each warp streams
// its own tiles through its own ring of shared-memory stages with cp.async (no
// block-wide barrier inside a segment; masked keys are not read but filled
// with zeros, so that stale NaNs cannot meet a zero probability).  A tile's
// work is a chain of dependent steps of about a microsecond: eight to sixteen
// warps an SM cover it.
//
// Measured on one GB300 (bytes of keys, values, q and out; the card copies
// 6.77 TB/s): 16 sequences of 2000-4001 keys, 32 heads on 8 of 128, bf16: 32.7 us,
// 5.0 TB/s; 64 sequences of 8192-16384 keys in Q8_0: 287 us, 5.7 TB/s (bound by
// issuing instructions: about 500 a 16 keys); one of 131071 keys, 32 heads on 4, f16,
// capped: 50 us, 5.3 TB/s; 24 with windows of 1024, 12 heads of 64: 16.3 us,
// 4.3 TB/s; one of 337 keys: 6.8 us.  Of the 32.7 us the loads take about 22, at the
// card's rate; 2.3 go by until the first tile is asked for (lengths, page ids,
// addresses: three dependent loads), 5 in the joins, the rest in the launch.
//
// Split: the tiles of all (sequence, kv head, tile of query heads) items form
// one list, cut into equal contiguous ranges, one per resident block, whatever
// the lengths (in whole shares an item while blocks outnumber items); the
// lengths are read on the device, so a captured graph serves every step.  An
// item that spans blocks leaves one partial (m, l, sum) per block in the
// workspace; the block that finishes last (a ticket per item, and per group of
// 16 blocks where many share one) joins them in block order, so results are
// bitwise repeatable.
//
// Products run on mma.sync m16n8k16 (two operands of 16 bits, fp32 sums): at
// one new token the tensor work is a fraction of the load time, and eight
// heads fill its n (values) or half its m (keys).  q is split into 16-bit pieces,
// and so are the probabilities: two after a power-of-two normalisation for f16
// operands, which hold 22 bits of each number, three for bf16, which hold 24.  A
// third f16 piece would be half as many products again, against errors that the
// sums make anyway: root mean squares against 64 bits are 0.15 to 0.25 units of
// 2^-24 sum |q k| for a score (f16 keys, whose products are longer, 0.5 to 0.9) and
// 1 to 1.3 of 2^-24 sum p |v| for an output of four keys (f16 1.9 to 2.4);
// exponentials are ex2.approx, 2 units.  The first two q pieces share one
// instruction: piece 0 in rows 0-7, piece 1 in rows 8-15; with four heads an
// instruction takes up to four pieces.
//   QK:  S[16 = (piece, head)][8 keys] += Q[16][16 d] K[8 keys][16 d]^T
//   PV:  O^T[16 d][8 heads] = V[16 keys][16 d]^T P[16 keys][8 heads]
// The score registers of a tile are the value product's B operand as they
// stand.  The value product of a tile starts from zero and is added to the
// running sum with a rounding FMA: sums kept inside the tensor cores lose
// low bits over thousands of tiles.
// Q8_0: codes enter as f16 integers; key scales multiply the scores of their
// 32-value block, value scales the probabilities, which are first brought to
// f16's range by the power of two that the largest finite value scale so far
// asks for.  (Codes + 128 as f16 subnormals are a byte permute cheaper a pair,
// but then the sums carry 128 times the sum of q: with one large code a block
// and small ones beside it scores were off by 12 units of 2^-24 sum |q k| instead
// of 0.2.  That and the look for infinite scales cost the 64 sequences 277 -> 287 us.)
#pragma once

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cstring>
#include <type_traits>

#include "kv_cache.cuh"
#include "qmm_device.cuh"
#include "qmm_internal.h"

namespace qmm {

namespace {

constexpr int kGroup = 16;  // keys of an instruction group (the instruction's k and two n)
constexpr int kLens = 512;  // lengths kept in shared memory
// The fixed part of an item's time in a block (its first loads, its joins), in
// the time of 16-key groups; blocks get equal shares of groups and these.
constexpr int kItemCost = 12;
// A block takes at least so much: splitting an item costs a join, which is
// worth it from about twenty saved groups on.
constexpr int kMinUnits = 36;
// Keys of a sequence, at most: the units of 32 sequences fit 32 bits, and keys
// past the last tile 31.
constexpr int64_t kMostKeys = 0x7fff0000;
constexpr int kLaneSeqs = 4;  // sequences of a lane in the plan of some sequences
constexpr int kStatic = 3072;  // the kernel's static shared memory, at most
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

enum Kind { kF16, kBF16, kQ8 };

// Groups of a tile, the keys a warp takes in one step.  Two share the step's
// fixed instructions and its latency where shared memory still holds enough
// warps' stages.
constexpr int attn_groups(Kind k, int D) { return k == kQ8 && D <= 128 ? 2 : 1; }

template <Kind KIND, int D, int HEADS, int WARPS>
struct Shape {
    static constexpr int W = WARPS, THREADS = 32 * W;
    // heads of an operand, and operands of the block's heads
    static constexpr int NH = HEADS < 8 ? HEADS : 8, HT = HEADS / NH;
    static constexpr int KT = attn_groups(KIND, D), TILE = KT * kGroup;
    static constexpr unsigned ALL = KT == 2 ? 0xffffffffu : 0xffffu;  // every key valid
    static constexpr int COST = kItemCost / KT, MIN_UNITS = kMinUnits / KT;  // in tiles
    static constexpr int ROWB = KIND == kQ8 ? D : 2 * D;           // bytes of a row
    // Rows in shared memory.  16-bit values: 16-byte chunk c of row r sits at
    // c ^ (r & 7), so that the eight rows of an ldmatrix lie in different banks.
    // Q8_0: 32-byte block c sits at c ^ swz8(r), which spreads both the eight
    // rows of its key loads and the four even or odd ones of its value loads.
    // Rows that are not whole 128 bytes are padded instead.
    static constexpr bool SWZ = ROWB % 128 == 0;
    static constexpr int RS = SWZ ? ROWB : KIND == kQ8 ? ROWB + (D % 64 == 0 ? 32 : 0) : ROWB + 16;
    static __host__ __device__ constexpr int swz8(int r) { return ((r & 7) ^ ((r & 7) >> 2)) & 3; }
    // Byte of chunk ch of row r of a tile.
    static __host__ __device__ constexpr uint32_t chunk_place(int r, int ch)
    {
        return r * RS + (!SWZ ? ch : KIND == kQ8 ? ch ^ (swz8(r) * 2) : ch ^ (r & 7)) * 16;
    }
    static constexpr int SP = kv_scales_per_row(D);
    static constexpr int SCB = KIND == kQ8 ? SP * 2 : 0;           // bytes of a row's scales
    static constexpr int STAGE = 2 * TILE * (RS + SCB);
    static constexpr int CHUNKS = ROWB / 16;                       // 16-byte chunks of a row
    static constexpr int KSTEPS = D / 16;
    // q's operand registers in shared memory: four a lane (two pieces of eight
    // heads, or up to four of four), and two for a third piece of eight heads
    static constexpr bool THIRD = KIND == kBF16 && NH == 8;
    static constexpr int QF1 = KSTEPS * (THIRD ? 768 : 512), QFRAG = HT * QF1;
    static constexpr int OSTRIDE = D + 4;
    static constexpr int JOIN = W * HEADS * (OSTRIDE + 2) * 4;
    // Resident blocks an SM: as many as leave two stages a warp (and, for the
    // registers, four): a warp's work on a tile is a chain of dependent
    // steps that other warps have to cover.
    static constexpr int LEAST = QFRAG + 2 * W * STAGE + kStatic + 1024;
    static constexpr int BLOCKS = 228 * 1024 / LEAST < 16 / W ? 228 * 1024 / LEAST : 16 / W;
    static constexpr int FIT =
        (228 * 1024 / BLOCKS - QFRAG - kStatic - 1024) / (W * STAGE);
    static constexpr int STAGES = FIT < 6 ? FIT : 6;
    static constexpr int RING = W * STAGES * STAGE;
    static constexpr int SMEM = QFRAG + (RING > JOIN ? RING : JOIN);
    static_assert(STAGES >= 2, "ring");
    // Where the 16-byte chunk it * 32 + lane of a tile's contiguous rows goes;
    // copy_base is the lane's part of it where rows are powers of two.
    static constexpr bool POW2 = 32 % CHUNKS == 0;
    static __device__ __forceinline__ uint32_t copy_base(int lane)
    {
        return chunk_place(lane / CHUNKS, lane % CHUNKS);
    }
    static __device__ __forceinline__ uint32_t copy_at(uint32_t base, int it, int lane)
    {
        if constexpr (POW2) {  // (the swizzles are linear in the row's bits)
            constexpr int R = 32 / CHUNKS;  // rows of an instruction
            return (base ^ (chunk_place(it * R, 0) - it * R * RS)) + it * R * RS;
        } else {
            const int idx = it * 32 + lane;
            return chunk_place(idx / CHUNKS, idx % CHUNKS);
        }
    }
    // Address of 32-byte column c of a row, from that of column 0.
    static __device__ __forceinline__ uint32_t column(uint32_t row, int c)
    {
        return SWZ ? (row ^ ((c & 3) * 32)) + (c >> 2) * 128 : row + c * 32;
    }
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, unsigned bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void *src, unsigned bytes)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
    return v;
}
// N words from a 4-byte boundary (one load where N is 1, 2 or 4 and the
// address a multiple of their size).
template <int N>
__device__ __forceinline__ void lds_words(uint32_t (&v)[N], uint32_t addr)
{
    if constexpr (N == 2) {
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];"
                     : "=r"(v[0]), "=r"(v[1])
                     : "r"(addr)
                     : "memory");
    } else if constexpr (N == 4) {
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                     : "r"(addr)
                     : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = lds32(addr + 4 * i);
    }
}
__device__ __forceinline__ uint2 lds64(uint32_t addr)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}

template <Kind KIND>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1)
{
    if constexpr (KIND == kBF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <Kind KIND>
using Half = typename std::conditional<KIND == kBF16, __nv_bfloat16, __half>::type;

// Four int8 codes, as bytes code + 128, to two pairs of f16: 1024 + byte by
// the exponent byte 0x64, minus 1152.
__device__ __forceinline__ uint32_t codes_f16(uint32_t biased, unsigned sel)
{
    const uint32_t w = __byte_perm(biased, 0x64646464u, sel);
    const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&w),
                              __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Codes 0 and 2 of four int8 codes as two f16: 1024 + (code + 128) in one logical
// operation, minus 1152; and codes 1 and 3.
__device__ __forceinline__ uint32_t even_codes(uint32_t w)
{
    const uint32_t x = (w & 0x00ff00ffu) ^ 0x64806480u;
    const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&x),
                              __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t odd_codes(uint32_t w) { return even_codes(w >> 8); }

// The tile list of one sequence: keys [lo, hi), tiles t0 .. t0 + n - 1 (tiles
// counted from key 0).
struct Span {
    int lo, hi, t0, n;
};
template <int TILE>
__device__ __forceinline__ Span tiles_of(const AttnArgs &a, int len)
{
    Span s;
    s.hi = max(0, min(len, int(min(a.ld_table * a.c.page_size, kMostKeys))));
    s.lo = a.window > 0 ? max(0, s.hi - a.window) : 0;
    s.t0 = s.lo / TILE;
    s.n = s.hi > s.lo ? (s.hi + TILE - 1) / TILE - s.t0 : 0;
    return s;
}

template <typename IO>
__device__ __forceinline__ float load_io(const void *p, int64_t i)
{
    return load1(static_cast<const IO *>(p) + i);
}
__device__ __forceinline__ float load_any(const void *p, int64_t i, int dtype)
{
    return dtype == QMM_F32   ? load_io<float>(p, i)
           : dtype == QMM_F16 ? load_io<__half>(p, i)
                              : load_io<__nv_bfloat16>(p, i);
}
__device__ __forceinline__ void store4_any(void *p, int64_t i, float4 v, int dtype)
{
    if (dtype == QMM_F32)
        store4(static_cast<float *>(p) + i, v);
    else if (dtype == QMM_F16)
        store4(static_cast<__half *>(p) + i, v);
    else
        store4(static_cast<__nv_bfloat16 *>(p) + i, v);
}
__device__ __forceinline__ void add4(float4 &s, float f, float4 v)
{
    s.x += f * v.x;
    s.y += f * v.y;
    s.z += f * v.z;
    s.w += f * v.w;
}

// The dim of a head that lane group g's accumulator pair x of value tile ds holds.
template <Kind KIND>
__device__ __forceinline__ int dim_of(int ds, int g, int x)
{
    return KIND == kQ8 ? (ds / 2) * 32 + 4 * g + 2 * (ds & 1) + x : ds * 16 + g + x * 8;
}

// One value of a buffer (data, and the scales of Q8_0): the slow paths' access.
template <Kind KIND, int D>
__device__ __forceinline__ float value_at(const uint8_t *data, const void *scales, uint64_t row,
                                          int d)
{
    if constexpr (KIND == kQ8)
        return float(reinterpret_cast<const int8_t *>(data)[row * D + d]) *
               __half2float(static_cast<const __half *>(scales)[row * kv_scales_per_row(D) + d / 32]);
    else
        return load1(reinterpret_cast<const Half<KIND> *>(data) + row * D + d);
}

template <Kind KIND, int D, int HEADS, int WARPS>
__global__ void __launch_bounds__(Shape<KIND, D, HEADS, WARPS>::THREADS,
                                  Shape<KIND, D, HEADS, WARPS>::BLOCKS)
    attn_kernel(const __grid_constant__ AttnParams P)
{
    using S = Shape<KIND, D, HEADS, WARPS>;
    constexpr int NH = S::NH, HT = S::HT;
    constexpr int kWarps = S::W, kThreads = S::THREADS, KT = S::KT, TILE = S::TILE;
    using H = Half<KIND>;
    constexpr int STAGES = S::STAGES;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t warp_units[kWarps];
    __shared__ int warp_longest[kWarps];
    __shared__ int64_t found_at;   // first tile of the sequence that the block starts in
    __shared__ int found_seq;
    __shared__ int lens[kLens];
    __shared__ unsigned strides[32 * kLaneSeqs];
    __shared__ unsigned valid_ring[kWarps][STAGES];
    __shared__ int qexp[HEADS];
    __shared__ bool settles[HEADS];  // a score of the head that is NaN may not be (below)
    __shared__ bool last_block;

    const AttnArgs &A = P.a;
    const KvView &C = A.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    pdl_wait();
    pdl_launch_dependents();

    // ---- the plan: prefix sums of the sequences' units
    // An item's units (and, for few sequences, what rounds them up to whole shares).
    int round = 0;
    auto stride_of = [&](int n) { return n ? unsigned(n + S::COST) : 0u; };
    auto units_of = [&](int n) { return int64_t(stride_of(n)) * P.items; };
    auto len_of = [&](int b) { return b < kLens ? lens[b] : __ldg(A.lens + b); };
    // Sequences without keys are no one's item: their outputs are zero.
    auto fill_empty = [&]() {
        for (int b = blockIdx.x; b < A.n_seqs; b += gridDim.x) {
            if (tiles_of<TILE>(A, __ldg(A.lens + b)).n > 0)
                continue;
            for (int i = tid; i < A.n_q * D / 4; i += kThreads)
                store4_any(A.out, b * A.ldo + 4 * i, make_float4(0.f, 0.f, 0.f, 0.f), A.dtype);
            if (A.lse)
                for (int i = tid; i < A.n_q; i += kThreads)
                    A.lse[int64_t(b) * A.n_q + i] = -INFINITY;
        }
    };
    // Block c takes units [c * per, (c + 1) * per): unit x is block x / per's.
    // Equal shares for all resident blocks, but no smaller ones than pay for
    // a join; those small ones divide the longest item evenly.
    auto share = [&](int64_t total, int longest) {
        const unsigned item = unsigned(longest + S::COST);
        const unsigned parts = max(1u, item / unsigned(S::MIN_UNITS));
        const int64_t even = total <= 0xffffffffll
                                 ? int64_t((unsigned(total) - 1) / gridDim.x + 1)
                                 : (total - 1) / int64_t(gridDim.x) + 1;
        return max(int64_t((item + parts - 1) / parts), even);
    };
    int64_t total = 0, per, r0, seq_at;
    int seq, seq_len;
    unsigned seq_stride;  // units of an item of the sequence
    if (A.n_seqs <= 32) {
        // every warp by itself, a sequence a lane
        const int len = lane < A.n_seqs ? __ldg(A.lens + lane) : 0;
        const Span sp = tiles_of<TILE>(A, len);
        if (blockIdx.x == 0 && warp == 0 && (len < 0 || len > sp.hi))
            atomicOr(A.status, kStatusBadLengthBit);
        if (warp == 0)
            lens[lane] = len;  // (read after later barriers)
        const unsigned own = stride_of(sp.n);
        // (kMostKeys: sums of 32 fit 32 bits)
        total = int64_t(__reduce_add_sync(0xffffffffu, own)) * P.items;
        if (total == 0) {
            fill_empty();
            return;
        }
        per = share(total, __reduce_max_sync(0xffffffffu, sp.n));
        // With fewer items than blocks, shares a little larger may let every
        // block keep to one item: a second one costs it another start and join.
        // (Sixteenths: Q8_0's wide rows take too long for their bytes to wait for
        // a larger share; 16 sequences of 4096 keys: 32 us, with larger ones 34,
        // head_dim 256: 54 and 60.)
        constexpr unsigned MORE = KIND == kQ8 && D >= 128 && WARPS == 4 ? 0 : 4;
        unsigned stride = own;
        if (per < (1 << 23) && __reduce_max_sync(0xffffffffu, own) < (1u << 23)) {
            const unsigned p0 = unsigned(per);
            for (unsigned more = 0; more <= MORE; more += 2) {
                const unsigned p = p0 + p0 * more / 16u;
                unsigned parts = unsigned(__fdividef(float(own), float(p)));
                parts += parts * p < own;  // (rounded down or exact: up)
                if (uint64_t(__reduce_add_sync(0xffffffffu, parts)) * unsigned(P.items) <=
                    gridDim.x) {
                    round = int(p);
                    stride = parts * p;
                    break;
                }
            }
            if (round)
                per = round;
        }
        if (warp == 0)
            strides[lane] = stride;  // (read after later barriers)
        unsigned sum = stride;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned v = __shfl_up_sync(0xffffffffu, sum, o);
            sum += lane >= o ? v : 0u;
        }
        const int64_t upto = int64_t(sum) * P.items, mine = int64_t(stride) * P.items;
        total = __shfl_sync(0xffffffffu, upto, 31);
        r0 = per * blockIdx.x;
        const unsigned past = __ballot_sync(0xffffffffu, upto > r0);
        if (!past) {
            fill_empty();
            return;
        }
        seq = __ffs(past) - 1;
        seq_at = __shfl_sync(0xffffffffu, upto - mine, seq);
        seq_len = __shfl_sync(0xffffffffu, len, seq);
        seq_stride = __shfl_sync(0xffffffffu, stride, seq);
    }
    // Some more, none of astronomical length (sums fit 32 bits): the same with
    // up to four neighbouring sequences a lane, where the general plan's barriers
    // and loops cost more (128 sequences of 100 keys, 2 heads of 64: 11.4 -> 6.0 us;
    // 48 of 1000, one head of 128: 14.9 -> 12.8).  Not for Q8_0: its kernel lost
    // registers of the main loop to this (64 sequences 294 us, without it 276 then).
    bool some = KIND != kQ8 && A.n_seqs > 32 && A.n_seqs <= 32 * kLaneSeqs;
    if (some) {
        const int each = (A.n_seqs + 31) / 32;  // sequences of a lane
        int len[kLaneSeqs];
        unsigned stride[kLaneSeqs], own = 0;
        int most = 0;
#pragma unroll
        for (int i = 0; i < kLaneSeqs; ++i) {
            const int b = lane * each + i;
            len[i] = i < each && b < A.n_seqs ? __ldg(A.lens + b) : 0;
        }
#pragma unroll
        for (int i = 0; i < kLaneSeqs; ++i) {
            const Span sp = tiles_of<TILE>(A, len[i]);
            if (blockIdx.x == 0 && warp == 0 && (len[i] < 0 || len[i] > sp.hi))
                atomicOr(A.status, kStatusBadLengthBit);
            if (warp == 0 && i < each)
                lens[lane * each + i] = len[i];  // (read after later barriers)
            stride[i] = stride_of(sp.n);
            own += min(stride[i], 1u << 24);
            most = max(most, sp.n);
        }
        most = __reduce_max_sync(0xffffffffu, most);
        some = most < (1 << 23);
        total = int64_t(__reduce_add_sync(0xffffffffu, own)) * P.items;
        if (total == 0) {
            fill_empty();
            return;
        }
        if (some) {
            per = share(total, most);
            // With fewer items than blocks, shares a little larger may let every
            // block keep to one item: a second one costs it another start and join.
            if (per < (1 << 23)) {
                const unsigned p0 = unsigned(per);
                unsigned parts[kLaneSeqs];
                for (unsigned more = 0; more <= 4 && !round; more += 2) {
                    const unsigned p = p0 + p0 * more / 16u;
                    unsigned sum = 0;
#pragma unroll
                    for (int i = 0; i < kLaneSeqs; ++i) {
                        parts[i] = unsigned(__fdividef(float(stride[i]), float(p)));
                        parts[i] += parts[i] * p < stride[i];  // (rounded down or exact: up)
                        sum += parts[i];
                    }
                    if (uint64_t(__reduce_add_sync(0xffffffffu, sum)) * unsigned(P.items) <=
                        gridDim.x)
                        round = int(p);
                }
                if (round) {
                    per = round;
                    own = 0;
#pragma unroll
                    for (int i = 0; i < kLaneSeqs; ++i) {
                        stride[i] = parts[i] * unsigned(round);
                        own += stride[i];
                    }
                }
            }
            unsigned sum = own;  // of this lane's sequences and those before
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned v = __shfl_up_sync(0xffffffffu, sum, o);
                sum += lane >= o ? v : 0u;
            }
            total = int64_t(__shfl_sync(0xffffffffu, sum, 31)) * P.items;
            r0 = per * blockIdx.x;
            const unsigned past = __ballot_sync(0xffffffffu, int64_t(sum) * P.items > r0);
            if (!past) {
                fill_empty();
                return;
            }
            // the first of the lane's sequences that reaches past r0
            unsigned at = sum - own;
            int mine = 0;
            bool found = false;
#pragma unroll
            for (int i = 0; i < kLaneSeqs; ++i) {
                if (warp == 0 && i < each)
                    strides[lane * each + i] = stride[i];  // (read after later barriers)
                found |= int64_t(at + stride[i]) * P.items > r0;
                if (!found) {
                    at += stride[i];
                    ++mine;
                }
            }
            const int from = __ffs(past) - 1;
            int my_len = len[0];
            unsigned my_stride = stride[0];
#pragma unroll
            for (int i = 1; i < kLaneSeqs; ++i) {
                my_len = mine == i ? len[i] : my_len;
                my_stride = mine == i ? stride[i] : my_stride;
            }
            seq = from * each + __shfl_sync(0xffffffffu, mine, from);
            seq_at = int64_t(__shfl_sync(0xffffffffu, at, from)) * P.items;
            seq_len = __shfl_sync(0xffffffffu, my_len, from);
            seq_stride = __shfl_sync(0xffffffffu, my_stride, from);
        }
    }
    if (A.n_seqs > 32 && !some) {
        total = 0;
        for (int b = tid; b < min(A.n_seqs, kLens); b += kThreads)
            lens[b] = __ldg(A.lens + b);
        __syncthreads();
        const int per_thread = (A.n_seqs + kThreads - 1) / kThreads;
        const int sb0 = min(A.n_seqs, tid * per_thread), sb1 = min(A.n_seqs, sb0 + per_thread);
        int64_t mine = 0;
        int most = 0;
        for (int b = sb0; b < sb1; ++b) {
            const int len = len_of(b);
            const Span sp = tiles_of<TILE>(A, len);
            mine += units_of(sp.n);
            most = max(most, sp.n);
            if (blockIdx.x == 0 && (len < 0 || len > sp.hi))
                atomicOr(A.status, kStatusBadLengthBit);
        }
        int64_t upto = mine;  // units of the sequences up to this thread's
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
            upto += lane >= o ? v : 0;
        }
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 31) {
            warp_units[warp] = upto;
            warp_longest[warp] = most;
        }
        __syncthreads();
        int longest = 0;  // tiles of the longest item
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            upto += w < warp ? warp_units[w] : 0;
            total += warp_units[w];
            longest = max(longest, warp_longest[w]);
        }
        if (total == 0) {
            fill_empty();
            return;
        }
        per = share(total, longest);
        r0 = per * blockIdx.x;
        if (r0 >= total) {
            fill_empty();
            return;
        }
        if (r0 < upto && r0 >= upto - mine) {
            int64_t at = upto - mine;
            for (int b = sb0; b < sb1; ++b) {
                const int64_t n = units_of(tiles_of<TILE>(A, len_of(b)).n);
                if (r0 < at + n) {
                    found_seq = b;
                    found_at = at;
                    break;
                }
                at += n;
            }
        }
        __syncthreads();
        seq = found_seq;
        seq_at = found_at;
        seq_len = len_of(seq);
        seq_stride = stride_of(tiles_of<TILE>(A, seq_len).n);
    }
    const int64_t blk = blockIdx.x, r1 = min(total, r0 + per);
    Span sp = tiles_of<TILE>(A, seq_len);

    const uint32_t smem_base = smem_u32(smem);
    // this lane's row and half-chunk of an ldmatrix over 16 keys x 16 values
    const uint32_t frag_row =
        S::chunk_place((lane >> 4) * 8 + (lane & 7), (lane >> 3) & 1);
    // Q8_0: this lane's key row g and value rows 2t, 2t + 1 in a group
    const uint32_t key_row = g * S::RS + (S::SWZ ? S::swz8(g) * 32 : 0) + t * 8;
    uint32_t val_row[2];
#pragma unroll
    for (int x = 0; x < 2; ++x)
        val_row[x] = (2 * t + x) * S::RS + (S::SWZ ? S::swz8(2 * t + x) * 32 : 0) + 4 * g;
    const uint32_t copy_row = S::copy_base(lane);
    const bool whole_groups = C.page.d % kGroup == 0;  // a group lies in one page
    const uint32_t ring = smem_base + S::QFRAG + warp * STAGES * S::STAGE;
    float *join = reinterpret_cast<float *>(smem + S::QFRAG);
    float *join_ml = join + kWarps * HEADS * S::OSTRIDE;

    for (int64_t at = r0; at < r1;) {
        while (at >= seq_at + int64_t(seq_stride) * P.items) {
            seq_at += int64_t(seq_stride) * P.items;
            ++seq;
            sp = tiles_of<TILE>(A, len_of(seq));
            seq_stride = round ? strides[seq] : stride_of(sp.n);
        }
        // the item and this block's tiles [ta, tb) of it
        const int item = int(uint64_t(at - seq_at) / seq_stride);
        const int64_t item_at = seq_at + int64_t(item) * seq_stride, tiles_at = item_at + S::COST;
        const int ta = int(max(int64_t(0), at - tiles_at));
        const int tb = int(max(int64_t(0), min(r1 - tiles_at, int64_t(sp.n))));
        at = item_at + seq_stride;
        if (tb <= ta)
            break;  // the range ends in the item's overhead: the next block starts the item
        const int kvh = item / P.head_tiles, h0 = (item % P.head_tiles) * HEADS;
        const int nh = min(HEADS, P.group - h0);
        const int head0 = kvh * P.group + h0;  // first query head
        const int nw = max(0, (tb - ta - warp + kWarps - 1) / kWarps);  // this warp's tiles
        const int32_t *table = A.table + int64_t(seq) * A.ld_table;

        // ---- loading
        auto key_of = [&](int i) { return (sp.t0 + ta + warp + i * kWarps) * TILE + (lane & (TILE - 1)); };
        // the page of this lane's key of tile i (a guarded load and no branch,
        // so that several are under way at once)
        auto page_id = [&](int i) -> int {
            const int j = key_of(i);
            const bool in = i < nw && j >= sp.lo && j < sp.hi;
            const int id = __ldg(table + (in ? fast_div(C.page, unsigned(j)) : 0u));
            return in ? id : -1;
        };
        auto row_of = [&](int j, uint32_t &row) {  // (the slow paths')
            if (j < sp.lo || j >= sp.hi)
                return false;
            const unsigned pg = fast_div(C.page, unsigned(j));
            const int id = __ldg(table + pg);
            row = (uint32_t(id) * unsigned(C.n_heads) + unsigned(kvh)) * C.page.d + unsigned(j) -
                  pg * C.page.d;
            return unsigned(id) < C.n_pages;
        };
        auto slow_dot = [&](int h, uint32_t row) {  // q of head h times a key
            const int64_t q0 = int64_t(seq) * A.ldq + int64_t(head0 + h) * D;
            float dot = 0.f;
#pragma unroll 1
            for (int d = 0; d < D; ++d)
                dot += load_any(A.q, q0 + d, A.dtype) * value_at<KIND, D>(C.k, C.ks, row, d);
            return dot;
        };
        auto issue = [&](int i, int id) {
            const int first = (sp.t0 + ta + warp + i * kWarps) * TILE;
            const int st = i % STAGES;
            const uint32_t kdst = ring + st * S::STAGE, vdst = kdst + TILE * S::RS;
            if (i < nw && whole_groups && first >= sp.lo && first + TILE <= sp.hi &&
                __all_sync(0xffffffffu, unsigned(id) < C.n_pages)) {
                // sixteen keys of one page at a time: contiguous rows
                if (lane == 0)
                    valid_ring[warp][st] = S::ALL;
#pragma unroll
                for (int u = 0; u < KT; ++u) {
                    const unsigned key = unsigned(first + u * kGroup);
                    const unsigned pg = unsigned(KT == 1 ? id : __shfl_sync(0xffffffffu, id, u * 16));
                    const uint32_t row = (pg * unsigned(C.n_heads) + unsigned(kvh)) * C.page.d + key -
                                         fast_div(C.page, key) * C.page.d;
                    const uint64_t o = uint64_t(row) * S::ROWB + lane * 16;
                    const uint8_t *ksrc = C.k + o, *vsrc = C.v + o;
#pragma unroll
                    for (int it = 0; it < kGroup * S::CHUNKS / 32; ++it) {
                        const uint32_t at = S::copy_at(copy_row, it, lane) + u * kGroup * S::RS;
                        cp16(kdst + at, ksrc + it * 512);
                        cp16(vdst + at, vsrc + it * 512);
                    }
                    if constexpr (KIND == kQ8) {
                        // SCB chunks of scales, lanes 0.. the keys', 16.. the values'
                        const uint8_t *ssrc = static_cast<const uint8_t *>(lane < 16 ? C.ks : C.vs);
                        if ((lane & 15) < S::SCB)
                            cp16(kdst + 2 * TILE * S::RS +
                                     ((lane >> 4) * TILE + u * kGroup) * S::SCB + (lane & 15) * 16,
                                 ssrc + uint64_t(row) * S::SCB + (lane & 15) * 16);
                    }
                }
            } else if (i < nw) {
                const int j = key_of(i);
                const bool ok = unsigned(id) < C.n_pages;
                if (!ok && j >= sp.lo && j < sp.hi)
                    atomicOr(A.status, kStatusBadPageBit);
                uint32_t row = 0;
                if (ok) {
                    const uint32_t off = unsigned(j) - fast_div(C.page, unsigned(j)) * C.page.d;
                    row = (uint32_t(id) * unsigned(C.n_heads) + unsigned(kvh)) * C.page.d + off;
                }
                const unsigned valid = __ballot_sync(0xffffffffu, ok) & S::ALL;
                if (lane == 0)
                    valid_ring[warp][st] = valid;
#pragma unroll
                for (int it = 0; it < TILE * S::CHUNKS / 32; ++it) {
                    const int idx = it * 32 + lane;
                    const int r = idx / S::CHUNKS, ch = idx % S::CHUNKS;
                    const uint64_t o =
                        uint64_t(__shfl_sync(0xffffffffu, row, r)) * S::ROWB + ch * 16;
                    const unsigned bytes = (valid >> r) & 1u ? 16u : 0u;
                    const uint32_t at = S::chunk_place(r, ch);
                    cp16(kdst + at, C.k + o, bytes);
                    cp16(vdst + at, C.v + o, bytes);
                }
                if constexpr (KIND == kQ8) {
                    constexpr int W = S::SCB / 4;  // words of a row's scales
                    const uint32_t sdst = kdst + 2 * TILE * S::RS;
#pragma unroll
                    for (int it = 0; it < (TILE * W + 31) / 32; ++it) {
                        const int idx = it * 32 + lane;
                        const int r = (idx / W) & (TILE - 1), w = idx % W;
                        const uint64_t o =
                            uint64_t(__shfl_sync(0xffffffffu, row, r)) * S::SCB + w * 4;
                        const unsigned bytes = (valid >> r) & 1u ? 4u : 0u;
                        if (idx < TILE * W) {
                            cp4(sdst + idx * 4, static_cast<const uint8_t *>(C.ks) + o, bytes);
                            cp4(sdst + TILE * S::SCB + idx * 4,
                                static_cast<const uint8_t *>(C.vs) + o, bytes);
                        }
                    }
                }
            }
            cp_commit();
        };
        // q of heads tid/16 and 8 more, issued ahead of everything that waits
        float qv[HT][D / 16];
#pragma unroll
        for (int hh = 0; hh < HT; ++hh) {
            const int h = (tid >> 4) + hh * 8;
            const int64_t q0 =
                int64_t(seq) * A.ldq + int64_t(head0 + min(h, nh - 1)) * D + (tid & 15);
            if (A.dtype == QMM_F32) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
                    qv[hh][i] = __ldg(static_cast<const float *>(A.q) + q0 + i * 16);
            } else if (A.dtype == QMM_F16) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
                    qv[hh][i] = load_io<__half>(A.q, q0 + i * 16);
            } else {
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
                    qv[hh][i] = load_io<__nv_bfloat16>(A.q, q0 + i * 16);
            }
        }
        int next_id;
        {
            int ids[STAGES];
#pragma unroll
            for (int i = 0; i < STAGES; ++i)
                ids[i] = page_id(i);
#pragma unroll
            for (int i = 0; i < STAGES - 1; ++i)
                issue(i, ids[i]);
            next_id = ids[STAGES - 1];
        }

        // ---- q's pieces as A operands, by 16 threads a head
#pragma unroll
        for (int hh = 0; hh < HT; ++hh) {
            const int h = (tid >> 4) + hh * 8, lt = tid & 15;
            float mx = 0.f, sum = 0.f;  // sum: 0, or NaN
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                qv[hh][i] = h < nh ? qv[hh][i] : 0.f;
                mx = fmaxf(mx, fabsf(qv[hh][i]));
                // A NaN in q is its answer, and so is an infinity but under a cap.
                sum += A.softcap > 0.f && fabsf(qv[hh][i]) > FLT_MAX ? 0.f : qv[hh][i] * 0.f;
            }
            int e = 0;
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) {
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
            }
            if constexpr (KIND != kBF16) {
                // the largest component to [2^13, 2^14)
                e = max(-126, min(126, 13 - (int(__float_as_uint(mx) >> 23) - 127)));
            }
            if (tid < 16 * NH) {  // (whole warps)
                if (lt == 0) {
                    qexp[h] = e;
                    settles[h] = sum == 0.f;
                }
                uint16_t *frag = reinterpret_cast<uint16_t *>(smem + hh * S::QF1);
                uint16_t *frag3 =
                    reinterpret_cast<uint16_t *>(smem + hh * S::QF1 + S::KSTEPS * 512);
                const float f = exp2i(e);
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const int d = i * 16 + lt;
                    int ks, tt, hi, lo;
                    if constexpr (KIND == kQ8) {
                        // lane t of a key holds codes 8t .. 8t+7 of a 32-block, in each
                        // four of them the even ones first
                        ks = (d >> 5) * 2 + ((d >> 2) & 1);
                        tt = (d & 31) >> 3;
                        hi = d & 1;
                        lo = (d >> 1) & 1;
                    } else {
                        ks = d >> 4;
                        tt = (d & 7) >> 1;
                        hi = (d >> 3) & 1;
                        lo = d & 1;
                    }
                    // row r of the operand: lane 4 (r % 8) + tt, register 2 hi + r / 8
                    auto put = [&](int r, H v) {
                        frag[(ks * 32 + (r & 7) * 4 + tt) * 8 + (2 * hi + (r >> 3)) * 2 + lo] =
                            *reinterpret_cast<const uint16_t *>(&v);
                    };
                    const float x = qv[hh][i] * f;
                    const H p0 = H(x);
                    const float r1 = x - float(p0);
                    const H p1 = H(r1);
                    const int hr = h & 7;  // the head's row of its operand
                    put(hr, p0);
                    put(hr + NH, p1);
                    if constexpr (NH == 4) {
                        put(hr + 8, KIND == kBF16 ? H(r1 - float(p1)) : H(0.f));
                        put(hr + 12, H(0.f));
                    } else if constexpr (S::THIRD) {
                        const H p2 = H(r1 - float(p1));
                        frag3[(ks * 32 + hr * 4 + tt) * 4 + hi * 2 + lo] =
                            *reinterpret_cast<const uint16_t *>(&p2);
                    }
                }
            }
        }
        __syncthreads();

        const int hg = g & (NH - 1);  // the head of an operand whose scores this lane holds
        float qscale[HT], slope[HT];
#pragma unroll
        for (int hh = 0; hh < HT; ++hh) {
            const int hd = hh * 8 + hg;
            qscale[hh] = A.scale * exp2i(-qexp[hd]);
            slope[hh] = A.alibi && hd < nh ? __ldg(A.alibi + head0 + hd) * kLog2e : 0.f;
        }
        // (a cap below 2^-128 has no finite reciprocal, and a score of 0 stays 0)
        const float cap_inv = A.softcap > 0.f ? fminf(1.f / A.softcap, FLT_MAX) : 0.f;
        // f16 probabilities are carried 2^14 times as large, clear of its subnormals
        constexpr float kBias = KIND == kF16 ? 14.f : 0.f;
        float m[HT], l[HT];  // of head hd
        int vexp[HT];        // Q8_0: exponent of the largest value scale so far
        float O[HT][D / 16][4] = {};
#pragma unroll
        for (int hh = 0; hh < HT; ++hh) {
            m[hh] = -INFINITY;
            l[hh] = 0.f;
            vexp[hh] = -126;
        }

        auto key_in = [&](int x) { return 2 * t + (x & 1) + (x >> 1) * 8; };  // of a group
        for (int i = 0; i < nw; ++i) {
            issue(i + STAGES - 1, next_id);
            next_id = page_id(i + STAGES);
            cp_wait<STAGES - 1>();
            __syncwarp();
            const int st = i % STAGES;
            const uint32_t kb = ring + st * S::STAGE, vb = kb + TILE * S::RS;
            const uint32_t ksb = vb + TILE * S::RS, vsb = ksb + TILE * S::SCB;

#pragma unroll
            for (int hh = 0; hh < HT; ++hh) {
            const int hd = hh * 8 + hg;
            const uint8_t *const qs = smem + hh * S::QF1;
            // ---- scores of head hd at keys 2t, 2t+1, 2t+8, 2t+9 of each group
            float s[KT][4];
            if constexpr (KIND == kQ8) {
                uint32_t ksc[KT][4][S::SP / 2];
#pragma unroll
                for (int u = 0; u < KT; ++u)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        s[u][x] = 0.f;
                        lds_words(ksc[u][x], ksb + (u * kGroup + key_in(x)) * S::SCB);
                    }
#pragma unroll
                for (int blk = 0; blk < D / 32; ++blk) {
                    uint4 a[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint8_t *fr = qs + ((2 * blk + h) * 32 + lane) * 16;
                        if constexpr (NH == 8) {
                            a[h] = *reinterpret_cast<const uint4 *>(fr);
                        } else {  // rows 8-15 are empty
                            a[h].x = *reinterpret_cast<const uint32_t *>(fr);
                            a[h].y = 0u;
                            a[h].z = *reinterpret_cast<const uint32_t *>(fr + 8);
                            a[h].w = 0u;
                        }
                    }
#pragma unroll
                    for (int u = 0; u < KT; ++u)
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            float c[4] = {};
                            uint2 w = lds64(
                                S::column(kb + (u * kGroup + n * 8) * S::RS + key_row, blk));
                            mma<KIND>(c, a[0].x, a[0].y, a[0].z, a[0].w, even_codes(w.x), odd_codes(w.x));
                            mma<KIND>(c, a[1].x, a[1].y, a[1].z, a[1].w, even_codes(w.y), odd_codes(w.y));
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const float2 sc = unpack2(ksc[u][2 * n + y][blk / 2], __half());
                                s[u][2 * n + y] += (NH == 8 ? c[y] + c[2 + y] : c[y]) *
                                                   (blk & 1 ? sc.y : sc.x);
                            }
                        }
                }
            } else {
                // two chains of sums a key block, for the instructions' latency
                float c[KT][2][2][4] = {}, third[KT][2][4] = {};
#pragma unroll
                for (int ks = 0; ks < S::KSTEPS; ++ks) {
                    const uint4 a =
                        *reinterpret_cast<const uint4 *>(qs + (ks * 32 + lane) * 16);
                    uint2 a3 = make_uint2(0u, 0u);
                    if constexpr (S::THIRD)
                        a3 = *reinterpret_cast<const uint2 *>(qs + S::KSTEPS * 512 +
                                                              (ks * 32 + lane) * 8);
#pragma unroll
                    for (int u = 0; u < KT; ++u) {
                        uint32_t b[4];
                        ldsm4(b, S::column(kb + u * kGroup * S::RS + frag_row, ks));
                        mma<KIND>(c[u][ks & 1][0], a.x, a.y, a.z, a.w, b[0], b[1]);
                        mma<KIND>(c[u][ks & 1][1], a.x, a.y, a.z, a.w, b[2], b[3]);
                        if constexpr (S::THIRD) {
                            mma<KIND>(third[u][0], a3.x, 0u, a3.y, 0u, b[0], b[1]);
                            mma<KIND>(third[u][1], a3.x, 0u, a3.y, 0u, b[2], b[3]);
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < KT; ++u)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int n = x >> 1, y = x & 1;
                        // the smaller pieces first
                        float v = c[u][0][n][y + 2] + c[u][1][n][y + 2];
                        if constexpr (S::THIRD)
                            v += third[u][n][y];
                        s[u][x] = v + (c[u][0][n][y] + c[u][1][n][y]);
                    }
            }
            float check = 0.f;
#pragma unroll
            for (int u = 0; u < KT; ++u)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    if constexpr (NH == 4)  // the other pieces' rows
                        s[u][x] += __shfl_xor_sync(0xffffffffu, s[u][x], 16);
                    check += s[u][x] * 0.f;
                }
            const unsigned valid = valid_ring[warp][st];
            const int key0 = (sp.t0 + ta + warp + i * kWarps) * TILE;
            // An infinite component of a key times pieces of q, or an infinite one
            // of q in pieces, gives NaN where the product with q itself is infinite:
            // settle it with q itself.
            if (__any_sync(0xffffffffu, check != 0.f && settles[hd])) {
#pragma unroll
                for (int u = 0; u < KT; ++u)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        uint32_t row;
                        if (!settles[hd] || hd >= nh || s[u][x] == s[u][x] ||
                            !row_of(key0 + u * kGroup + key_in(x), row))
                            continue;
                        s[u][x] = slow_dot(hd, row) * exp2i(qexp[hd]);
                    }
            }
            // scores in base 2
            float tmax = -INFINITY;
#pragma unroll
            for (int u = 0; u < KT; ++u) {
                if (A.softcap > 0.f) {
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        s[u][x] = A.softcap * kLog2e * tanhf(s[u][x] * qscale[hh] * cap_inv);
                } else {
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        s[u][x] *= qscale[hh] * kLog2e;
                }
                if (A.alibi) {
                    const float back = float(key0 + u * kGroup + 2 * t - (sp.hi - 1));
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        s[u][x] += slope[hh] * (back + float((x & 1) + (x >> 1) * 8));
                }
                if (valid != S::ALL) {
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        s[u][x] = (valid >> (u * kGroup + key_in(x))) & 1u ? s[u][x] : -INFINITY;
                }
                tmax = fmaxf(tmax, fmaxf(fmaxf(s[u][0], s[u][1]), fmaxf(s[u][2], s[u][3])));
            }
            tmax = fmaxf(tmax, __shfl_xor_sync(0xffffffffu, tmax, 1));
            tmax = fmaxf(tmax, __shfl_xor_sync(0xffffffffu, tmax, 2));
            const float mn = fmaxf(m[hh], tmax);
            const float base = mn == -INFINITY ? 0.f : mn;
            const float corr = ex2(m[hh] - base);  // 0 while nothing was seen
            m[hh] = mn;
            float p[KT][4], psum = 0.f;
#pragma unroll
            for (int u = 0; u < KT; ++u)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    p[u][x] = ex2(s[u][x] - (base - kBias));
                    psum += p[u][x];
                }
            l[hh] = l[hh] * corr + psum;
            // O's columns 2t and 2t+1 are heads (and with four heads, pieces)
            float f0 = __shfl_sync(0xffffffffu, corr, 8 * t),
                  f1 = __shfl_sync(0xffffffffu, corr, 8 * t + 4);

            // ---- values
            if constexpr (KIND == kQ8) {
                // the largest value scale of the tile moves the common exponent up
                __half2 mx = __half2half2(__ushort_as_half(0));
                uint32_t vsc[KT][4][S::SP / 2];
#pragma unroll
                for (int u = 0; u < KT; ++u)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        lds_words(vsc[u][x], vsb + (u * kGroup + key_in(x)) * S::SCB);
                        if (D % 64 != 0)
                            vsc[u][x][S::SP / 2 - 1] &= 0xffffu;  // the odd half is padding
#pragma unroll
                        for (int w = 0; w < S::SP / 2; ++w)
                            mx = __hmax2(
                                mx, __habs2(*reinterpret_cast<const __half2 *>(&vsc[u][x][w])));
                    }
                float dm = __half2float(__hmax(__low2half(mx), __high2half(mx)));
                dm = fmaxf(dm, __shfl_xor_sync(0xffffffffu, dm, 1));
                dm = fmaxf(dm, __shfl_xor_sync(0xffffffffu, dm, 2));
                if (__any_sync(0xffffffffu, dm > FLT_MAX)) {  // an infinite scale: the largest of the others
                    unsigned most = 0;
#pragma unroll 1
                    for (int i = lane; i < TILE * S::SP; i += 32) {
                        const unsigned d = lds16(vsb + 2 * i) & 0x7fffu;
                        if (d < 0x7c00u && (D % 64 == 0 || i % S::SP < D / 32))
                            most = max(most, d);
                    }
                    most = __reduce_max_sync(0xffffffffu, most);
                    dm = __half2float(__ushort_as_half(uint16_t(most)));
                }
                const int ve = max(vexp[hh], int(__float_as_uint(dm) >> 23) - 127);
                const float fe = exp2i(max(-126, vexp[hh] - ve));
                f0 *= fe;
                f1 *= fe;
                vexp[hh] = ve;
                const float up = exp2i(min(126, 14 - ve));
#pragma unroll
                for (int u = 0; u < KT; ++u)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        p[u][x] *= up;
#pragma unroll
                for (int blk = 0; blk < D / 32; ++blk) {
                    float c[2][4] = {};
#pragma unroll
                    for (int u = 0; u < KT; ++u) {
                        uint32_t bp[2][2];
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            const float2 s0 = unpack2(vsc[u][2 * n][blk / 2], __half());
                            const float2 s1 = unpack2(vsc[u][2 * n + 1][blk / 2], __half());
                            const float u0 = p[u][2 * n] * (blk & 1 ? s0.y : s0.x);
                            const float u1 = p[u][2 * n + 1] * (blk & 1 ? s1.y : s1.x);
                            bp[0][n] = pack2(u0, u1, H());
                            const float2 hf = unpack2(bp[0][n], H());
                            bp[1][n] = pack2(u0 - hf.x, u1 - hf.y, H());
                            if constexpr (NH == 4)  // columns 4-7 carry the second piece
                                bp[0][n] = g < 4 ? bp[0][n] : bp[1][n];
                        }
                        uint32_t w[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            w[x] = lds32(S::column(vb + (u * kGroup + (x >> 1) * 8) * S::RS +
                                                       val_row[x & 1], blk)) ^ 0x80808080u;
                        const uint32_t e01 = __byte_perm(w[0], w[1], 0x5140),
                                       e23 = __byte_perm(w[0], w[1], 0x7362),
                                       o01 = __byte_perm(w[2], w[3], 0x5140),
                                       o23 = __byte_perm(w[2], w[3], 0x7362);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t a0 = codes_f16(h ? e23 : e01, 0x4140);
                            const uint32_t a1 = codes_f16(h ? e23 : e01, 0x4342);
                            const uint32_t a2 = codes_f16(h ? o23 : o01, 0x4140);
                            const uint32_t a3 = codes_f16(h ? o23 : o01, 0x4342);
                            if constexpr (NH == 8)
                                mma<KIND>(c[h], a0, a1, a2, a3, bp[1][0], bp[1][1]);
                            mma<KIND>(c[h], a0, a1, a2, a3, bp[0][0], bp[0][1]);
                        }
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float(&o)[4] = O[hh][blk * 2 + h];
                        o[0] = o[0] * f0 + c[h][0];
                        o[1] = o[1] * f1 + c[h][1];
                        o[2] = o[2] * f0 + c[h][2];
                        o[3] = o[3] * f1 + c[h][3];
                    }
                }
            } else {
                constexpr int PIECES = KIND == kBF16 ? 3 : 2;
                constexpr int MMAS = NH == 4 ? PIECES - 1 : PIECES;
                uint32_t b[KT][PIECES][2];
#pragma unroll
                for (int u = 0; u < KT; ++u)
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        float u0 = p[u][2 * n], u1 = p[u][2 * n + 1];
#pragma unroll
                        for (int q = 0; q < PIECES; ++q) {
                            b[u][q][n] = pack2(u0, u1, H());
                            const float2 hf = unpack2(b[u][q][n], H());
                            u0 -= hf.x;
                            u1 -= hf.y;
                        }
                        if constexpr (NH == 4) {  // columns 4-7 carry the second piece
                            b[u][0][n] = g < 4 ? b[u][0][n] : b[u][1][n];
                            if constexpr (PIECES == 3)
                                b[u][1][n] = g < 4 ? b[u][2][n] : 0u;
                        }
                    }
#pragma unroll
                for (int ds = 0; ds < S::KSTEPS; ++ds) {
                    float c[4] = {};
#pragma unroll
                    for (int u = 0; u < KT; ++u) {
                        uint32_t a[4];
                        ldsm4t(a, S::column(vb + u * kGroup * S::RS + frag_row, ds));
#pragma unroll
                        for (int q = MMAS - 1; q >= 0; --q)
                            mma<KIND>(c, a[0], a[1], a[2], a[3], b[u][q][0], b[u][q][1]);
                    }
                    O[hh][ds][0] = O[hh][ds][0] * f0 + c[0];
                    O[hh][ds][1] = O[hh][ds][1] * f1 + c[1];
                    O[hh][ds][2] = O[hh][ds][2] * f0 + c[2];
                    O[hh][ds][3] = O[hh][ds][3] * f1 + c[3];
                }
            }
            }
            __syncwarp();
        }
        cp_wait<0>();
#pragma unroll
        for (int hh = 0; hh < HT; ++hh) {
            l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], 1);
            l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], 2);
        }
        __syncthreads();  // every warp is done with its ring: it becomes the joining space

        // ---- the warps' results joined
        // An infinite value times pieces of a probability (some of them 0 or
        // negative) gives NaN where the sum is infinite, and a key whose score is
        // -infinity has probability 0, which makes an infinite value NaN: such
        // sums, if any, are settled by looking at the values again.
        auto settle_sum = [&](int h, int d, float4 &sum) {
            float inf[4] = {};  // sums of the infinities and NaNs
#pragma unroll 1
            for (int j = (sp.t0 + ta) * TILE; j < (sp.t0 + tb) * TILE; ++j) {
                uint32_t row;
                if (!row_of(j, row))
                    continue;
                float v[4];
                bool any = false;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    v[x] = value_at<KIND, D>(C.v, C.vs, row, d + x);
                    v[x] = fabsf(v[x]) <= FLT_MAX ? 0.f : v[x];
                    any |= v[x] != 0.f;
                }
                if (!any)
                    continue;
                const bool never = A.softcap == 0.f && slow_dot(h, row) * A.scale == -INFINITY;
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    inf[x] += never && v[x] != 0.f ? NAN : v[x];
            }
            sum.x = inf[0] != 0.f ? inf[0] : sum.x;
            sum.y = inf[1] != 0.f ? inf[1] : sum.y;
            sum.z = inf[2] != 0.f ? inf[2] : sum.z;
            sum.w = inf[3] != 0.f ? inf[3] : sum.w;
        };
        auto finish = [&](int h, int d, float4 sum, float M, float tot) {
            const float inv = tot == 0.f ? 0.f : 1.f / tot;
            store4_any(A.out, int64_t(seq) * A.ldo + int64_t(head0 + h) * D + d,
                       make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv), A.dtype);
            if (A.lse && d == 0)
                A.lse[int64_t(seq) * A.n_q + head0 + h] =
                    tot == 0.f ? -INFINITY : (M + log2f(tot) - kBias) * kLn2;
        };
#pragma unroll
        for (int hh = 0; hh < HT; ++hh) {
            float undo = 1.f;
            if constexpr (KIND == kQ8)
                undo = exp2i(max(-126, vexp[hh] - 14));
            float *o = join + (warp * HEADS + hh * 8) * S::OSTRIDE;
#pragma unroll
            for (int ds = 0; ds < D / 16; ++ds) {
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    float v = O[hh][ds][x];
                    if constexpr (NH == 4)
                        v += __shfl_xor_sync(0xffffffffu, v, 2);
                    if (NH == 8 || t < 2)
                        o[(2 * t + (x & 1)) * S::OSTRIDE + dim_of<KIND>(ds, g, x >> 1)] = v * undo;
                }
            }
            if (t == 0 && g < NH) {
                join_ml[(warp * HEADS + hh * 8 + g) * 2] = m[hh];
                join_ml[(warp * HEADS + hh * 8 + g) * 2 + 1] = l[hh];
            }
        }
        __syncthreads();
        const bool whole = ta == 0 && tb == sp.n;
        // blocks that share the item
        const int64_t c0 = whole ? blk : uint64_t(tiles_at) / uint64_t(per);
        const int64_t c1 = whole ? blk : uint64_t(tiles_at + sp.n - 1) / uint64_t(per);
        constexpr int PART = HEADS * (D + 2);  // floats of a partial: sums, m and l of each head
        constexpr int QUADS = D / 4;
        // A block may be the last of one item and the first of another: a
        // partial that starts its item goes to the block's second place.
        float *mine_ws = A.ws + (2 * blk + (ta > 0 ? 0 : 1)) * PART;
        for (int i = tid; i < nh * QUADS; i += kThreads) {
            const int h = i / QUADS, d = i % QUADS * 4;
            float mw[kWarps], M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                mw[w] = join_ml[(w * HEADS + h) * 2];
                M = fmaxf(M, mw[w]);
            }
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
            float tot = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = mw[w] == -INFINITY ? 0.f : ex2(mw[w] - M);
                add4(sum, f, *reinterpret_cast<const float4 *>(
                                 join + (w * HEADS + h) * S::OSTRIDE + d));
                tot += f * join_ml[(w * HEADS + h) * 2 + 1];
            }
            // (where the probabilities are NaN there is nothing to settle)
            if (!(fabsf(sum.x) + fabsf(sum.y) + fabsf(sum.z) + fabsf(sum.w) <= FLT_MAX) &&
                tot == tot)
                settle_sum(h, d, sum);
            if (whole) {
                finish(h, d, sum, M, tot);
            } else {
                __stcg(reinterpret_cast<float4 *>(mine_ws + h * D + d), sum);
                if (d == 0) {
                    __stcg(mine_ws + HEADS * D + h, M);
                    __stcg(mine_ws + HEADS * D + HEADS + h, tot);
                }
            }
        }
        if (!whole) {
            // ---- the item's last block joins the blocks' partials in block
            // order; many blocks first join in groups, each group's last block
            // leaving the group's result in the place of its first
            const int n = int(c1 - c0) + 1, k = int(blk - c0);
            const int gs = n <= 16 ? n : (n <= 256 ? 16 : 32);  // blocks of a group
            float *const start = A.ws + 2 * c0 * PART;
            auto place = [&](int c) { return start + int64_t(2 * c + (c == 0)) * PART; };
            // Is this block the last of `of` to count on the ticket?  The
            // barrier puts every thread's stores before thread 0's release.
            auto last_of = [&](unsigned *ticket, int of) {
                __syncthreads();
                if (tid == 0) {
                    unsigned before;
                    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;"
                                 : "=r"(before)
                                 : "l"(ticket)
                                 : "memory");
                    last_block = before == unsigned(of - 1);
                    if (last_block)
                        *ticket = 0;
                }
                __syncthreads();
                return last_block;
            };
            // Sum of `count` partials `step` blocks apart, from block `from`
            // of the item on; sixteen are under way at once.
            auto join_parts = [&](int from, int step, int count, int h, int d, float4 &sum,
                                  float &M, float &tot) {
                sum = make_float4(0.f, 0.f, 0.f, 0.f);
                M = -INFINITY;
                tot = 0.f;
                for (int c = 0; c < count; c += 16) {
                    float4 o[16];
                    float pm[16], pl[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float *w = place(from + min(c + j, count - 1) * step);
                        o[j] = __ldcg(reinterpret_cast<const float4 *>(w + h * D + d));
                        pm[j] = c + j < count ? __ldcg(w + HEADS * D + h) : -INFINITY;
                        pl[j] = __ldcg(w + HEADS * D + HEADS + h);
                    }
                    float mn = M;
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        mn = fmaxf(mn, pm[j]);
                    // (never 0: an infinite sum stays infinite)
                    const float f = M == -INFINITY ? 0.f : fmaxf(ex2(M - mn), FLT_MIN);
                    sum = make_float4(sum.x * f, sum.y * f, sum.z * f, sum.w * f);
                    tot *= f;
                    M = mn;
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        if (c + j >= count)
                            continue;
                        const float fj =
                            pm[j] == -INFINITY ? 0.f : fmaxf(ex2(pm[j] - mn), FLT_MIN);
                        add4(sum, fj, o[j]);
                        tot += fj * pl[j];
                    }
                }
            };
            const int grp = k / gs, first = grp * gs, size = min(gs, n - first);
            bool mine_to_join = last_of(
                A.tickets + (grp ? A.max_blocks + c0 + first : c0), size);
            if (mine_to_join && gs < n) {
                constexpr int PER = (HEADS * QUADS + kThreads - 1) / kThreads;
                float4 sum[PER];
                float M[PER], tot[PER];
#pragma unroll
                for (int u = 0; u < PER; ++u) {
                    const int i = tid + u * kThreads;
                    if (i < nh * QUADS)
                        join_parts(first, 1, size, i / QUADS, i % QUADS * 4, sum[u], M[u], tot[u]);
                }
                __syncthreads();  // everything is read before the first place is overwritten
                float *w = place(first);
#pragma unroll
                for (int u = 0; u < PER; ++u) {
                    const int i = tid + u * kThreads, h = i / QUADS, d = i % QUADS * 4;
                    if (i >= nh * QUADS)
                        continue;
                    __stcg(reinterpret_cast<float4 *>(w + h * D + d), sum[u]);
                    if (d == 0) {
                        __stcg(w + HEADS * D + h, M[u]);
                        __stcg(w + HEADS * D + HEADS + h, tot[u]);
                    }
                }
                mine_to_join = last_of(A.tickets + 2 * A.max_blocks + c0, (n + gs - 1) / gs);
            }
            if (mine_to_join) {
                for (int i = tid; i < nh * QUADS; i += kThreads) {
                    const int h = i / QUADS, d = i % QUADS * 4;
                    float4 sum;
                    float M, tot;
                    if (gs < n)
                        join_parts(0, gs, (n + gs - 1) / gs, h, d, sum, M, tot);
                    else
                        join_parts(0, 1, n, h, d, sum, M, tot);
                    finish(h, d, sum, M, tot);
                }
            }
        }
        __syncthreads();  // the joining space becomes the ring again
    }
    fill_empty();
}

template <Kind KIND, int D, int HEADS, int WARPS>
cudaError_t launch_warps(AttnParams &p, int sm_count, cudaStream_t s)
{
    using Sh = Shape<KIND, D, HEADS, WARPS>;
    const auto kern = attn_kernel<KIND, D, HEADS, WARPS>;
    // Resident blocks of an SM, asked for once a device.
    static std::atomic<int> resident[64];
    const unsigned dev = unsigned(p.a.device);
    int occ = dev < 64 ? resident[dev].load(std::memory_order_relaxed) : 0;
    if (occ == 0) {
        const void *f = reinterpret_cast<const void *>(kern);
        cudaError_t e = func_smem(f, Sh::SMEM, true);
        if (e == cudaSuccess)
            e = func_occupancy(f, Sh::THREADS, Sh::SMEM, &occ);
        if (e != cudaSuccess)
            return e;
        if (occ < 1)
            return cudaErrorInvalidConfiguration;
        if (dev < 64)
            resident[dev].store(occ, std::memory_order_relaxed);
    }
    p.head_tiles = (p.group + HEADS - 1) / HEADS;
    p.items = p.a.c.n_heads * p.head_tiles;
    const int64_t longest = std::min<int64_t>(p.a.ld_table * p.a.c.page_size, kMostKeys);
    const int64_t items = int64_t(p.a.n_seqs) * p.items;
    const int64_t units = items * ((longest + Sh::TILE - 1) / Sh::TILE + 1 + Sh::COST);
    // (the workspace is sized to Shape's blocks: attn_space)
    int64_t grid = int64_t(std::min<int>(occ, Sh::BLOCKS)) * sm_count;
    grid = std::max<int64_t>(1, std::min(grid, std::max(items, units / Sh::MIN_UNITS) + 1));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(grid));
    cfg.blockDim = dim3(Sh::THREADS);
    cfg.dynamicSmemBytes = Sh::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
    return counted(cudaLaunchKernelEx(&cfg, kern, p));
}

// Warps of a block.  Narrow rows: eight, two blocks on an SM (24 sequences of
// 1024 keys, head_dim 64: 16.2 us, with four warps 20).  Rows of 128: four, three
// blocks, which overlap one another's starts and joins; with few items, whose
// parts all have to be joined, one block of twelve (one sequence of 131071 keys:
// 50.3 us, with four 53.5; 337 keys: 6.9 us, with four 8.0; Q8_0, four sequences of
// 8000 keys: 14.4 us, with four 20.6).  Rows of 96, and 16-bit rows of 256: six
// fill the shared memory better.
constexpr int attn_warps(Kind k, int D)
{
    return D == 64 && k != kQ8 ? 8 : D == 96 || (D == 256 && k != kQ8) ? 6 : 4;
}
constexpr bool attn_has_twelve(int D, int heads) { return D == 128 && heads <= 8; }

template <Kind KIND, int D, int HEADS>
cudaError_t launch_heads(AttnParams &p, int sm_count, cudaStream_t s)
{
    if constexpr (attn_has_twelve(D, HEADS)) {
        const int64_t items =
            int64_t(p.a.n_seqs) * p.a.c.n_heads * ((p.group + HEADS - 1) / HEADS);
        if (items * 4 <= sm_count)
            return launch_warps<KIND, D, HEADS, 12>(p, sm_count, s);
    }
    return launch_warps<KIND, D, HEADS, attn_warps(KIND, D)>(p, sm_count, s);
}

// Heads that a block takes together.  Up to four that share a key: their pieces
// of q and of the probabilities fill the operands' other four rows and columns,
// half the instructions of the eight-head form.  Over eight: sixteen, so that
// keys and values are fetched once for them, where the second operand's
// instructions and registers cost less than the second fetch out of L2 (16
// sequences of 4096 keys, 16 heads a key: head_dim 64 in f16 28 us, bf16 35, with
// eight heads 37 and 40; f16 128: 54, with eight 55; bf16 128: 57, with eight 55).
constexpr bool attn_has_sixteen(Kind k, int D)
{
    return (D == 64 && k != kQ8) || (D == 128 && k == kF16);
}

template <Kind KIND, int D>
cudaError_t launch_dim(AttnParams &p, int sm_count, cudaStream_t s)
{
    if (p.group <= 4)
        return launch_heads<KIND, D, 4>(p, sm_count, s);
    if constexpr (attn_has_sixteen(KIND, D)) {
        if (p.group > 8)
            return launch_heads<KIND, D, 16>(p, sm_count, s);
    }
    return launch_heads<KIND, D, 8>(p, sm_count, s);
}

// What an SM's blocks need of the workspace, whichever form is launched: two
// partial results a block.
template <Kind KIND, int D, int HEADS, int WARPS>
constexpr AttnSpace with_form(AttnSpace s)
{
    using Sh = Shape<KIND, D, HEADS, WARPS>;
    return {std::max(s.blocks, int(Sh::BLOCKS)),
            std::max(s.floats, size_t(2) * Sh::BLOCKS * HEADS * (D + 2))};
}
template <Kind KIND, int D>
constexpr AttnSpace space_dim()
{
    constexpr int W = attn_warps(KIND, D);
    AttnSpace s = with_form<KIND, D, 8, W>(with_form<KIND, D, 4, W>({0, 0}));
    if constexpr (attn_has_twelve(D, 8))
        s = with_form<KIND, D, 8, 12>(with_form<KIND, D, 4, 12>(s));
    if constexpr (attn_has_sixteen(KIND, D))
        s = with_form<KIND, D, 16, W>(s);
    return s;
}
template <Kind KIND>
AttnSpace space_kind(int D)
{
    switch (D) {
    case 64: return space_dim<KIND, 64>();
    case 96: return space_dim<KIND, 96>();
    case 128: return space_dim<KIND, 128>();
    case 192: return space_dim<KIND, 192>();
    default: return space_dim<KIND, 256>();
    }
}

template <Kind KIND>
cudaError_t launch_kind(AttnParams &p, int sm_count, cudaStream_t s)
{
    switch (p.a.c.D) {
    case 64: return launch_dim<KIND, 64>(p, sm_count, s);
    case 96: return launch_dim<KIND, 96>(p, sm_count, s);
    case 128: return launch_dim<KIND, 128>(p, sm_count, s);
    case 192: return launch_dim<KIND, 192>(p, sm_count, s);
    case 256: return launch_dim<KIND, 256>(p, sm_count, s);
    }
    return cudaErrorInvalidValue;
}

} // namespace

} // namespace qmm
