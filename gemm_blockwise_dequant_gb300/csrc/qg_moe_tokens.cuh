// qg_moe_tokens.cuh -- the expert products of a mixture-of-experts layer over a few tokens (one instance file for each
// width of the codes).
//
//   fc1  h[p][i] = silu(g) u,  g, u = dequant(W1[e]) . x[token] + b1[e]     (rows i of both halves)
//   fc2  o[p][n] = dequant(W2[e]) . h[p] + b2[e]                            (p: one of the token's experts, e)
//
// Bound by memory: every chosen expert's weights are read once, and with few rows each there are few operations to a
// byte.  The pairs (token, slot) are grouped by expert, up to 16 rows to a group; a group's activations are laid out
// once in shared memory, as fp16 with a power of two for each row (so fp16 and bf16 rows keep what they have).  h, which is
// fp32, takes two rows of fp16 for a pair, neighbouring columns of the MMAs, where y is not bf16: with one, an fp16 y was up to 1.5
// times as far off as its own rounding has it; with two no further (2 tokens 77 us instead of 75).  The weights go through
// m16n8k16 MMAs as the wide operand, 16 weight rows by 8 tokens: codes less the midpoint are whole numbers that fp16 holds
// exactly, one block's products are summed by the MMA and its scale is applied to the fp32 sums, so that nothing is rounded
// on the way.  A zero point other than the midpoint enters through the sum of the block's activations.
//
// Each warp streams its weights through a ring of its own (cp.async, no barrier between warps); S warps share a tile
// of 16 rows, each with a slice of K, and G = 16 / S tiles are worked on at a time.  S is chosen from the number of
// tiles, so that few of them still fill the warps.  A tile of fc1 is 8 gate rows and their 8 up rows: both values of an
// output meet in one lane.
//
// Measured (128 experts, top 8, 2880 x 2880, 4 bits in blocks of 32; the whole layer): 64 tokens 448 us, 1.76 GB of weights at
// 3.9 TB/s, of which the copies alone, in pieces of 128 bytes through two stages, take 396; 2 tokens 76 us.
#pragma once

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "qg_device.cuh"
#include "qg_moe_tokens.h"

namespace qg {
namespace moe {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxRows = 16;  // of activations in shared memory at a time

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// The same where a condition holds, without a branch.
template <int BYTES>
__device__ __forceinline__ void cp_async_if(bool is, uint32_t dst, const void *src) {
    if constexpr (BYTES == 16)
        asm volatile("{\n .reg .pred p;\n setp.ne.s32 p, %2, 0;\n @p cp.async.cg.shared.global [%0], [%1], 16;\n}" ::"r"(dst), "l"(src), "r"(static_cast<int>(is)) : "memory");
    else
        asm volatile("{\n .reg .pred p;\n setp.ne.s32 p, %2, 0;\n @p cp.async.ca.shared.global [%0], [%1], %3;\n}" ::"r"(dst), "l"(src), "r"(static_cast<int>(is)), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t add2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("add.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
// Without a C operand, or on top of one.
template <bool FIRST>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (FIRST)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// (a & MASK) | b as one operation, b in a register.
template <uint32_t MASK>
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "n"(MASK), "r"(b));
    return d;
}

// Codes of a width, SB values (32, or 64 where the blocks have them) of one row of a tile at a time: lane t of four
// holds SB / 4 neighbouring ones.  A stage of the ring holds kChunk values of 16 rows, which lie kStride bytes apart: that
// keeps the reads of eight rows free of bank conflicts.
template <int BITS, int SB>
struct Codes {
    static constexpr int kChunk = BITS == 8 ? 128 : 256;
    static constexpr int kUnits = kChunk / SB;
    static constexpr int kLane = SB / 4 * BITS / 8;            // bytes of a lane and unit
    static constexpr int kRow = kChunk * BITS / 8;             // bytes of a row in a stage
    static constexpr int kCopy = BITS == 2 && SB == 32 ? 8 : 16;
    static constexpr int kCopies = kRow / kCopy;               // of a row: 4 or 8
    static constexpr int kStride = kRow + (kLane == 2 ? 8 : kLane == 4 ? 16 : kLane == 8 ? 32 : 64);
    static constexpr int kPerLane = kCopies / 2;               // copies of a lane: 16 rows, 32 lanes
    static constexpr int kParWords = (kChunk / SB + 2) / 2;    // words of two scales that may hold a chunk's, of a row
    static constexpr float kMid = static_cast<float>(1 << (BITS - 1));
    static_assert(kCopies == 4 || kCopies == 8, "a lane's copies are of rows four or eight apart");
};

// Eight codes less the midpoint, as four pairs of fp16.  An fp16 of 1024 and more has its unit in the last place, so a
// code put there is 1024 + q; masked in place higher up, 1024 + 16 q (or 4 q), which one fma brings back.  Pair j holds
// the values order<BITS>(2 j) and order<BITS>(2 j + 1) of the eight.
// m: 1024 twice, in a register.
template <int BITS>
__device__ __forceinline__ void unpack(uint32_t lo, uint32_t hi, uint32_t m, uint32_t (&p)[4]) {
    if constexpr (BITS == 4) {
        const uint32_t w = lo >> 8;
        p[0] = add2(and_or<0x000F000Fu>(lo, m), 0xE408E408u);                   // - 1032
        p[1] = fma2(and_or<0x00F000F0u>(lo, m), 0x2C002C00u, 0xD480D480u);      // / 16 - 72
        p[2] = add2(and_or<0x000F000Fu>(w, m), 0xE408E408u);
        p[3] = fma2(and_or<0x00F000F0u>(w, m), 0x2C002C00u, 0xD480D480u);
    } else if constexpr (BITS == 2) {
        const uint32_t v = (lo & 0xFFFFu) | (lo << 12), w = v >> 8;
        p[0] = add2(and_or<0x00030003u>(v, m), 0xE402E402u);                    // - 1026
        p[1] = fma2(and_or<0x000C000Cu>(v, m), 0x34003400u, 0xDC08DC08u);       // / 4 - 258
        p[2] = add2(and_or<0x00030003u>(w, m), 0xE402E402u);
        p[3] = fma2(and_or<0x000C000Cu>(w, m), 0x34003400u, 0xDC08DC08u);
    } else {
        p[0] = add2(__byte_perm(lo, m, 0x5150), 0xE480E480u);                   // - 1152
        p[1] = add2(__byte_perm(lo, m, 0x5352), 0xE480E480u);
        p[2] = add2(__byte_perm(hi, m, 0x5150), 0xE480E480u);
        p[3] = add2(__byte_perm(hi, m, 0x5352), 0xE480E480u);
    }
}
template <int BITS>
__device__ __forceinline__ constexpr int order(int i) {
    return BITS == 4 ? (i >> 1) + 4 * (i & 1) : BITS == 2 ? (i & 4) + ((i >> 1) & 1) + 2 * (i & 1) : i;
}

// Shared memory: the ring of every warp, the partial sums, the plan, the activations and their block sums.
template <int BITS, int SB, bool ZP, int NT>
struct Layout {
    using C = Codes<BITS, SB>;
    static constexpr int kParRow = C::kParWords * 4;
    static constexpr int kParams = 16 * kParRow;
    static constexpr int kStage = 16 * C::kStride + kParams * (ZP ? 2 : 1);
    static constexpr int kStages = BITS == 2 ? (NT == 1 ? 4 : 3) : (NT == 1 ? 3 : 2);
    static constexpr int kRing = kWarps * kStages * kStage;
    static constexpr int kPartial = 2 * kWarps * 32 * NT * 16;
    static constexpr int kPlan = kMaxPairs * 2 + kMaxExperts * 4 + kMaxPairs * 4 + kMaxRows * 16 + 64;
    static constexpr int kFixed = kRing + kPartial + kPlan;
    static __host__ __device__ int x_stride(int K) { return SB == 32 ? K * 2 + (K % 64 == 0 ? 64 : 0) : K * 2 + 16; }
    static __host__ __device__ int x_bytes(int K, int rows) { return rows * (x_stride(K) + (ZP ? K / SB * 4 : 0)); }
    static_assert(kFixed % 16 == 0 && kStage % 16 == 0 && kPlan % 16 == 0, "alignment");
};

struct Plan {
    int16_t *ids;       // [pairs], -1: none
    int *count;         // [experts]
    uint32_t *group;    // [groups]: expert << 20 | groups of two columns before << 10 | first row's rank
    int *rows;          // [kMaxRows]: the pairs whose activations are here
    unsigned *top;      // [kMaxRows]: largest magnitude of a row, as bits
    float *back;        // [kMaxRows]: the power of two that undoes its scale
    int *base;          // [kMaxRows]: where a group's rows begin, by its place in the span
    int *num;           // groups, those of two columns, and where this CTA's and the next one's first tile is
};
__device__ __forceinline__ int expert_of(uint32_t group) { return static_cast<int>(group >> 20); }
__device__ __forceinline__ int wide_before(uint32_t group) { return static_cast<int>(group >> 10 & 0x3FFu); }
__device__ __forceinline__ int rank_of(uint32_t group) { return static_cast<int>(group & 0x3FFu); }

// Groups the pairs by expert, at most `limit` to a group; more than `narrow` take two columns.
__device__ __forceinline__ void make_plan(const Args &a, const Plan &p, int limit, int narrow) {
    const int tid = threadIdx.x;
    for (int e = tid; e < a.E; e += kThreads) p.count[e] = 0;
    __syncthreads();
    bool bad = false;
    for (int i = tid; i < a.P; i += kThreads) {
        const int e = __ldcg(a.ids + i);  // from the L2: fc 2 comes here before its own wait
        const bool ok = e >= 0 && e < a.E;
        p.ids[i] = static_cast<int16_t>(ok ? e : -1);
        if (ok) atomicAdd(&p.count[e], 1);
        bad |= !ok;
    }
    if (bad && a.status && blockIdx.x == 0) *a.status = 1;
    __syncthreads();
    if (tid < 32) {
        int before = 0;  // groups, and << 16 those of them of two columns
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + tid, rows = e < a.E ? p.count[e] : 0, n = (rows + limit - 1) / limit;
            const int full = rows / limit, wide = (limit > narrow ? full : 0) + (rows - full * limit > narrow ? 1 : 0);
            const int own = n | wide << 16;
            int sum = own;
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(~0u, sum, o);
                if (tid >= o) sum += v;
            }
            const int at = before + sum - own;
            for (int j = 0; j < n; ++j)  // the full ones first
                p.group[(at & 0xFFFF) + j] = static_cast<uint32_t>(e) << 20 | static_cast<uint32_t>((at >> 16) + (limit > narrow ? j : 0)) << 10 | static_cast<uint32_t>(j * limit);
            before += __shfl_sync(~0u, sum, 31);
        }
        if (tid == 0) p.num[0] = before & 0xFFFF, p.num[1] = before >> 16;
    }
    __syncthreads();
}

__device__ __forceinline__ int rows_of(const Plan &p, uint32_t group, int limit) {
    return min(limit, p.count[expert_of(group)] - rank_of(group));
}

// This CTA's tiles, num[2] .. num[3] - 1 of all groups' in a row: equal shares, where a tile of a group of two columns
// (more than eight rows) counts for kWide / kNarrow of another: with shares of as many tiles each, the CTA with most rows was
// done 26% after the others (64 tokens, 128 experts, top 8, 2880 x 2880, the one layer it was measured on: 541 us, and 446 us this way).
constexpr int kNarrow = 3, kWide = 4;
__device__ __forceinline__ void take_share(const Plan &p, int per) {
    const int groups = p.num[0], all = kNarrow * groups + (kWide - kNarrow) * p.num[1];
    for (int i = threadIdx.x; i < 2 * groups; i += kThreads) {
        const int g = i >> 1, which = i & 1, block = blockIdx.x + which;
        const auto cost_before = [&](int j) { return j == groups ? all : kNarrow * j + (kWide - kNarrow) * wide_before(p.group[j]); };
        const int from = cost_before(g), tile = cost_before(g + 1) - from;
        const int64_t begin = static_cast<int64_t>(all) * per * block / gridDim.x - static_cast<int64_t>(from) * per;
        if (begin >= 0 && begin < static_cast<int64_t>(tile) * per) p.num[2 + which] = g * per + static_cast<int>(begin / tile);
        else if (g == groups - 1 && begin >= 0) p.num[2 + which] = groups * per;
    }
    __syncthreads();
}

// The pairs of the groups g0 .. g1-1, in their order, one warp to a group.
__device__ __forceinline__ void find_rows(const Args &a, const Plan &p, int g0, int g1, int limit) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x < kMaxRows) p.top[threadIdx.x] = 0;
    for (int g = g0 + warp; g < g1; g += kWarps) {
        int base = 0;
        for (int i = g0; i < g; ++i) base += rows_of(p, p.group[i], limit);
        if (lane == 0) p.base[g - g0] = base;
        const uint32_t group = p.group[g];
        const int e = expert_of(group), first = rank_of(group);
        int n = 0;
        for (int i0 = 0; i0 < a.P && n < first + limit; i0 += 32) {
            const bool is = i0 + lane < a.P && p.ids[i0 + lane] == e;
            const unsigned who = __ballot_sync(~0u, is);
            const int at = n + __popc(who & ((1u << lane) - 1u));
            if (is && at >= first && at < first + limit) p.rows[base + at - first] = i0 + lane;
            n += __popc(who);
        }
    }
    __syncthreads();
}

__device__ __forceinline__ void load_values(const void *src, int dtype, size_t at, float (&x)[8]) {
    if (dtype == 0) {
        const float4 u = *reinterpret_cast<const float4 *>(static_cast<const float *>(src) + at), v = *reinterpret_cast<const float4 *>(static_cast<const float *>(src) + at + 4);
        x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w, x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
        return;
    }
    const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(src) + at);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = dtype == 1 ? h2f(static_cast<uint16_t>(w[i] & 0xFFFFu)) : __uint_as_float(w[i] << 16);
        x[2 * i + 1] = dtype == 1 ? h2f(static_cast<uint16_t>(w[i] >> 16)) : __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// The second of two terms is what the first leaves, times kSecond (11 bits more).
constexpr float kSecond = 2048.f;
// The activations of n pairs as scaled fp16, eight at a time in the order of the codes' pairs: a row for each, or two.  A row is the work of as many
// threads as there are for it; with up to kHeld vectors each they read it once.
template <int BITS, int SB, bool ZP, int NT>
__device__ __forceinline__ void stage_rows(const Args &a, const Plan &p, int n, char *xs, float *sums) {
    constexpr int kHeld = 3;
    int per = kThreads / kMaxRows;  // threads of a row: a warp or more
    while (per * 2 * n <= kThreads) per *= 2;
    const int r = threadIdx.x / per, lane = threadIdx.x % per, stride = Layout<BITS, SB, ZP, NT>::x_stride(a.K), vecs = a.K / 8;
    const size_t row = r < n ? static_cast<size_t>(a.fc == 1 ? p.rows[r] / a.k : p.rows[r]) * a.K : 0;
    float held[kHeld][8];
    float top = 0.f;
    if (r < n) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            if (lane + i * per < vecs) load_values(a.src, a.src_dtype, row + (lane + i * per) * 8, held[i]);
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            if (lane + i * per < vecs)
#pragma unroll
                for (int k = 0; k < 8; ++k) top = fmaxf(top, finite_abs(held[i][k]));
        for (int q = lane + kHeld * per; q < vecs; q += per) {
            float x[8];
            load_values(a.src, a.src_dtype, row + q * 8, x);
#pragma unroll
            for (int k = 0; k < 8; ++k) top = fmaxf(top, finite_abs(x[k]));
        }
        for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
        if ((threadIdx.x & 31) == 0) atomicMax(&p.top[r], __float_as_uint(top));
    }
    __syncthreads();
    if (r < n) {
        // the largest between 2^14 and 2^15: fp16 keeps 11 bits of whatever is above 2^-29 of it, and sums stay far from fp32's range
        const unsigned bits = p.top[r];
        const int e = bits >= 0x00800000u ? 14 - (static_cast<int>(bits >> 23) - 127) : bits ? 127 : 0, up = min(e, 127);
        const float scale = exp2i(max(up, -126)), low = e > 127 ? exp2i(e - 127) : 1.f;
        if (lane == 0) p.back[r] = exp2i(-max(up, -126)) / low;
        const auto put = [&](int q, const float (&x)[8]) {
            uint32_t w[4];
            uint16_t h[8], l[8];
            float sum = 0.f, sum2 = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float y = x[i] * scale * low;
                h[i] = f2h(y);
                l[i] = a.terms == 2 ? f2h((y - h2f(h[i])) * kSecond) : 0;
                if constexpr (ZP) sum += h2f(h[i]), sum2 += h2f(l[i]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = h[order<BITS>(2 * i)] | static_cast<uint32_t>(h[order<BITS>(2 * i + 1)]) << 16;
            *reinterpret_cast<uint4 *>(xs + r * a.terms * stride + q * 16) = make_uint4(w[0], w[1], w[2], w[3]);
            if (a.terms == 2) {
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = l[order<BITS>(2 * i)] | static_cast<uint32_t>(l[order<BITS>(2 * i + 1)]) << 16;
                *reinterpret_cast<uint4 *>(xs + (2 * r + 1) * stride + q * 16) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            if constexpr (ZP) {
                // SB / 8 neighbouring threads hold a block, and all of them are here: K / 8 is a multiple of SB / 8
                const unsigned quad = ((1u << (SB / 8)) - 1u) << (threadIdx.x & 31 & ~(SB / 8 - 1));
                for (int o = 1; o < SB / 8; o <<= 1) sum += __shfl_xor_sync(quad, sum, o), sum2 += __shfl_xor_sync(quad, sum2, o);
                if (q % (SB / 8) == 0) {
                    sums[r * a.terms * (a.K / SB) + q / (SB / 8)] = sum;
                    if (a.terms == 2) sums[(2 * r + 1) * (a.K / SB) + q / (SB / 8)] = sum2;
                }
            }
        };
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            if (lane + i * per < vecs) put(lane + i * per, held[i]);
        for (int q = lane + kHeld * per; q < vecs; q += per) {
            float x[8];
            load_values(a.src, a.src_dtype, row + q * 8, x);
            put(q, x);
        }
    }
    __syncthreads();
}

template <int BITS, int SB, bool ZP, int NTMAX>
__global__ void __launch_bounds__(kThreads, 1) expert_kernel(const __grid_constant__ Args a) {
    using C = Codes<BITS, SB>;
    using L = Layout<BITS, SB, ZP, NTMAX>;
    constexpr int D = L::kStages, CU = C::kUnits;
    extern __shared__ __align__(128) char smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g8 = lane >> 2, t4 = lane & 3;
    char *ring = smem + warp * (D * L::kStage);
    float4 *partial = reinterpret_cast<float4 *>(smem + L::kRing);
    char *at = smem + L::kRing + L::kPartial;
    Plan plan;
    plan.ids = reinterpret_cast<int16_t *>(at);
    plan.count = reinterpret_cast<int *>(at + kMaxPairs * 2);
    plan.group = reinterpret_cast<uint32_t *>(at + kMaxPairs * 2 + kMaxExperts * 4);
    plan.rows = reinterpret_cast<int *>(at + kMaxPairs * 6 + kMaxExperts * 4);
    plan.top = reinterpret_cast<unsigned *>(plan.rows + kMaxRows);
    plan.back = reinterpret_cast<float *>(plan.rows + 2 * kMaxRows);
    plan.base = plan.rows + 3 * kMaxRows;
    plan.num = plan.rows + 4 * kMaxRows;
    const int x_stride = L::x_stride(a.K), units = a.K / SB;
    char *xs = smem + L::kFixed;
    float *sums = reinterpret_cast<float *>(xs + a.room * x_stride);

    // fc 2 begins when all of fc 1 has waited for what is before it, the ids among them: only h is still to wait for, and
    // the plan and the first codes are fetched meanwhile, past the first-level cache: that may hold what the same addresses had before a kernel
    // ahead of this layer wrote there, and only the wait says that it does not.
    if (a.fc == 1) {
        pdl_wait();
        pdl_launch_dependents();
    }
    const int two = a.terms - 1, room = a.room >> two;  // pairs whose rows fit
    const int most_rows = min(8 * NTMAX >> two, room);
    make_plan(a, plan, most_rows, 8 / a.terms);
    const int per = a.N / 16, total = plan.num[0] * per;
    if (total) take_share(plan, per);
    const int first = total ? plan.num[2] : 0, last = total ? plan.num[3] : 0;
    if (first >= last) {
        if (a.fc == 2) pdl_wait();
        return;
    }
    // Slices of K: the fewest rounds of G tiles, a round's cost being its units and what opening and joining a tile takes
    const int most = (total + gridDim.x - 1) / gridDim.x;
    int S = 1, cost = 1 << 30;
    for (int s = 1; s <= kWarps; s *= 2) {
        const int c = ((most * s + kWarps - 1) / kWarps) * ((units + s - 1) / s + 4 * 32 / SB);
        if (c < cost) cost = c, S = s;
    }
    const int G = kWarps / S, mine = warp / S, slice = warp % S;
    const int u0 = units * slice / S, u1 = units * (slice + 1) / S;
    const int shift = SB == 32 ? 0 : 31 - __clz(a.bs / SB);  // units of a block, as a power of two

    // The weight rows of a tile: 16 neighbours, or 8 of each half (neighbours in pairs, where they are interleaved).
    const int nb = a.K / a.bs, row_bytes = a.K * BITS / 8;
    const int step = a.fc == 1 && a.interleaved ? 2 : 1, across = a.fc == 2 ? 8 : a.interleaved ? 1 : a.N / 2;  // r -> r + 1 within eight, r -> r + 8
    const auto first_row = [&](int tile) { return a.fc == 2 ? tile * 16 : tile * 8 * step; };

    // What this lane copies: pieces of the rows cr and further ones `across` and four apart, and its share of the scales.
    const int cr = lane / C::kCopies;
    const int64_t far8 = static_cast<int64_t>(across) * row_bytes, far4 = static_cast<int64_t>(4 * step) * row_bytes;
    const uint32_t code_to = smem_u32(ring) + cr * C::kStride + (lane % C::kCopies) * C::kCopy;
    const uint32_t par_to = smem_u32(ring) + 16 * C::kStride + (lane >> 1) * L::kParRow + (lane & 1) * 4;
    int ahead = first + mine, ahead_g = first / per, ahead_u = u0;
    const char *src = nullptr;
    const uint16_t *ssrc = nullptr;
    const int64_t zfar = ZP ? a.zp - a.scales : 0;
    const auto open = [&]() {
        while (ahead >= (ahead_g + 1) * per) ++ahead_g;
        const int64_t row = static_cast<int64_t>(expert_of(plan.group[ahead_g])) * a.N + first_row(ahead - ahead_g * per);
        src = reinterpret_cast<const char *>(a.w) + (row + cr * step) * row_bytes + (lane % C::kCopies) * C::kCopy + u0 * (SB * BITS / 8);
        ssrc = a.scales + (row + (lane >> 1 & 7) * step + (lane >> 4) * across) * nb;
    };
    if (ahead < last && u0 < u1) open();
    uint32_t fill = 0;  // bytes
    // A stage of the ring: its codes, its scales and zero points, or both.
    const auto issue = [&](auto codes_tag, auto params_tag) {
        constexpr bool CODES = decltype(codes_tag)::value, PARAMS = decltype(params_tag)::value;
        if (ahead < last) {
            const int left = u1 - ahead_u;  // units
            const bool there = (lane % C::kCopies) * (C::kCopy * 8 / BITS) < left * SB;
#pragma unroll
            for (int i = 0; i < (CODES ? C::kPerLane : 0); ++i) {
                // kCopies 4: rows cr, cr + 8; 8: cr, cr + 4, cr + 8, cr + 12
                const char *from = src + (C::kCopies == 4 ? (i ? far8 : 0) : (i & 1 ? far4 : 0) + (i & 2 ? far8 : 0));
                cp_async_if<C::kCopy>(there, code_to + fill + i * (32 / C::kCopies) * C::kStride, from);
            }
            // words of two scales, from the one that holds the chunk's first to the one that holds its last
            const int b0 = ahead_u >> shift, b1 = (ahead_u + min(left, CU) - 1) >> shift;
            const uintptr_t s0 = reinterpret_cast<uintptr_t>(ssrc + b0);
            const int behind = (static_cast<int>(s0 >> 1 & 1) + b1 - b0) >> 1;
            const char *word = reinterpret_cast<const char *>(s0 & ~static_cast<uintptr_t>(3)) + (lane & 1) * 4;
#pragma unroll
            for (int i = 0; i < (PARAMS ? (C::kParWords + 1) / 2 : 0); ++i) {
                cp_async_if<4>((lane & 1) + 2 * i <= behind, par_to + fill + 8 * i, word + 8 * i);
                if constexpr (ZP) cp_async_if<4>((lane & 1) + 2 * i <= behind, par_to + fill + L::kParams + 8 * i, word + 2 * zfar + 8 * i);
            }
            src += C::kRow;
            fill += L::kStage;
            if (fill == D * L::kStage) fill = 0;
            ahead_u += CU;
            if (ahead_u >= u1) {
                ahead_u = u0;
                ahead += G;
                if (ahead < last) open();
            }
        }
        if constexpr (PARAMS) cp_commit();
    };
    constexpr std::true_type yes{};
    constexpr std::false_type no{};
    if (a.fc == 2) {
        constexpr bool EARLY = C::kCopy == 16;  // smaller copies go through the first-level cache
        const int ahead0 = ahead, ahead_g0 = ahead_g;
        const char *const src0 = src;
        const uint16_t *const ssrc0 = ssrc;
        if constexpr (EARLY) {
#pragma unroll 1
            for (int i = 0; i < D - 1 && u0 < u1; ++i) issue(yes, no);
            ahead = ahead0, ahead_g = ahead_g0, ahead_u = u0, src = src0, ssrc = ssrc0, fill = 0;
        }
        pdl_wait();
        pdl_launch_dependents();
        // the codes of all these stages are waited for with the scales of the first
#pragma unroll 1
        for (int i = 0; i < D - 1; ++i)
            if (u0 < u1) issue(std::bool_constant<!EARLY>{}, yes);
            else cp_commit();
    } else {
#pragma unroll 1
        for (int i = 0; i < D - 1; ++i)
            if (u0 < u1) issue(yes, yes);
            else cp_commit();
    }

    int drain = 0, flip = 0;
    uint32_t magic;  // a value that the compiler does not know stays in its register
    asm volatile("mov.b32 %0, 0x64006400;" : "=r"(magic));
    const char *codes = ring + g8 * C::kStride + t4 * C::kLane;

    // One tile of a group of `rows` rows that begin at `base`.
    const auto run_tile = [&](auto nt_tag, int expert, int tile, int base, int rows) {
        constexpr int NT = decltype(nt_tag)::value;
        const int n0 = first_row(tile) + g8 * step, n1 = n0 + across;
        const int odd0 = static_cast<int>((static_cast<int64_t>(expert) * a.N + n0) * nb & 1), odd1 = odd0 ^ (across & nb & 1);
        const char *xlane[NT];
        [[maybe_unused]] const float *xsum[NT][2];
        float sum[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) {  // columns past the last row are not looked at
            xlane[j] = xs + (base + min(j * 8 + g8, rows - 1)) * x_stride + t4 * (SB / 4) * 2 + u0 * (SB * 2);
            if constexpr (ZP)
                for (int c = 0; c < 2; ++c) xsum[j][c] = sums + (base + min(j * 8 + 2 * t4 + c, rows - 1)) * units + u0;
            sum[j][0] = sum[j][1] = sum[j][2] = sum[j][3] = 0.f;
        }
        // one unit of K: its products, and the scale on their sum
        const auto unit = [&](const char *row0, const uint16_t *sp0, const uint16_t *sp1, int v, int b) {
            uint32_t c0[4], c1[4];
            row0 += v * (C::kLane * 4);
            const char *row1 = row0 + 8 * C::kStride;
            if constexpr (C::kLane == 2) {
                c0[0] = *reinterpret_cast<const uint16_t *>(row0), c1[0] = *reinterpret_cast<const uint16_t *>(row1);
            } else if constexpr (C::kLane == 4) {
                c0[0] = *reinterpret_cast<const uint32_t *>(row0), c1[0] = *reinterpret_cast<const uint32_t *>(row1);
            } else if constexpr (C::kLane == 8) {
                const uint2 p = *reinterpret_cast<const uint2 *>(row0), q = *reinterpret_cast<const uint2 *>(row1);
                c0[0] = p.x, c0[1] = p.y, c1[0] = q.x, c1[1] = q.y;
            } else {
                const uint4 p = *reinterpret_cast<const uint4 *>(row0), q = *reinterpret_cast<const uint4 *>(row1);
                c0[0] = p.x, c0[1] = p.y, c0[2] = p.z, c0[3] = p.w, c1[0] = q.x, c1[1] = q.y, c1[2] = q.z, c1[3] = q.w;
            }
            float acc[NT][4];
#pragma unroll
            for (int h = 0; h < SB / 32; ++h) {
                uint32_t p[4], q[4];
                if constexpr (BITS == 8) {
                    unpack<8>(c0[2 * h], c0[2 * h + 1], magic, p);
                    unpack<8>(c1[2 * h], c1[2 * h + 1], magic, q);
                } else if constexpr (BITS == 4) {
                    unpack<4>(c0[h], 0, magic, p);
                    unpack<4>(c1[h], 0, magic, q);
                } else {
                    unpack<2>(c0[0] >> (16 * h), 0, magic, p);
                    unpack<2>(c1[0] >> (16 * h), 0, magic, q);
                }
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const uint4 b4 = *reinterpret_cast<const uint4 *>(xlane[j] + (v * SB + h * 8) * 2);
                    if (h == 0) mma16816<true>(acc[j], p[0], q[0], p[1], q[1], b4.x, b4.y);
                    else mma16816<false>(acc[j], p[0], q[0], p[1], q[1], b4.x, b4.y);
                    mma16816<false>(acc[j], p[2], q[2], p[3], q[3], b4.z, b4.w);
                }
            }
            const float s0 = h2f(sp0[b]), s1 = h2f(sp1[b]);
            [[maybe_unused]] float z0 = 0.f, z1 = 0.f;
            if constexpr (ZP) {
                z0 = C::kMid - h2f(sp0[b + L::kParams / 2]);
                z1 = C::kMid - h2f(sp1[b + L::kParams / 2]);
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                if constexpr (ZP) {
                    const float x0 = xsum[j][0][v], x1 = xsum[j][1][v];
                    acc[j][0] = fmaf(z0, x0, acc[j][0]);
                    acc[j][1] = fmaf(z0, x1, acc[j][1]);
                    acc[j][2] = fmaf(z1, x0, acc[j][2]);
                    acc[j][3] = fmaf(z1, x1, acc[j][3]);
                }
                sum[j][0] = fmaf(s0, acc[j][0], sum[j][0]);
                sum[j][1] = fmaf(s0, acc[j][1], sum[j][1]);
                sum[j][2] = fmaf(s1, acc[j][2], sum[j][2]);
                sum[j][3] = fmaf(s1, acc[j][3], sum[j][3]);
            }
        };
#pragma unroll 1
        for (int u = u0; u < u1; u += CU) {
            cp_wait<D - 2>();
            __syncwarp();  // also: everyone has read the stage before, which the next copy goes to
            issue(yes, yes);
            const char *row0 = codes + drain;
            const uint16_t *sc = reinterpret_cast<const uint16_t *>(ring + drain + 16 * C::kStride) + g8 * (L::kParRow / 2);
            const int b0 = u >> shift;
            const uint16_t *sp0 = sc + ((odd0 + b0) & 1), *sp1 = sc + 8 * (L::kParRow / 2) + ((odd1 + b0) & 1);
            if (u + CU <= u1) {
                if (SB == 32 || shift == 0) {  // a scale for each unit
#pragma unroll
                    for (int v = 0; v < CU; ++v) unit(row0, sp0, sp1, v, v);
                } else {
#pragma unroll
                    for (int v = 0; v < CU; ++v) unit(row0, sp0, sp1, v, ((u + v) >> shift) - b0);
                }
            } else {
#pragma unroll 1
                for (int v = 0; u + v < u1; ++v) unit(row0, sp0, sp1, v, ((u + v) >> shift) - b0);
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                xlane[j] += C::kChunk * 2;
                if constexpr (ZP) xsum[j][0] += CU, xsum[j][1] += CU;
            }
            drain += L::kStage;
            if (drain == D * L::kStage) drain = 0;
        }
        // join the slices, in their order
        if (S > 1) {
            float4 *buf = partial + (flip * kWarps + warp) * (32 * NTMAX);
#pragma unroll
            for (int j = 0; j < NT; ++j) buf[j * 32 + lane] = make_float4(sum[j][0], sum[j][1], sum[j][2], sum[j][3]);
            named_bar_sync(1 + mine, S * 32);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            if (slice != (S > 1 ? j % S : 0)) continue;
            float4 v = make_float4(sum[j][0], sum[j][1], sum[j][2], sum[j][3]);
            if (S > 1) {
                const float4 *buf = partial + (flip * kWarps + mine * S) * (32 * NTMAX) + j * 32 + lane;
                v = buf[0];
                for (int i = 1; i < S; ++i) {
                    const float4 o = buf[i * (32 * NTMAX)];
                    v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
                }
            }
            const float bias0 = a.bias ? h2f(a.bias[static_cast<int64_t>(expert) * a.N + n0]) : 0.f, bias1 = a.bias ? h2f(a.bias[static_cast<int64_t>(expert) * a.N + n1]) : 0.f;
            const auto store = [&](int r, float x0, float x1) {  // a pair's values of rows g8 and g8 + 8
                const float back = plan.back[(base >> two) + r];
                const float p = fmaf(x0, back, bias0), q = fmaf(x1, back, bias1);
                const int64_t pair = plan.rows[(base >> two) + r];
                if (a.fc == 1) {
                    a.out[pair * (a.N / 2) + tile * 8 + g8] = p / (1.f + __expf(-p)) * q;
                } else {
                    a.out[pair * a.N + n0] = p;
                    a.out[pair * a.N + n1] = q;
                }
            };
            const int col = j * 8 + 2 * t4;
            if (two) {  // the terms of a pair are neighbouring columns
                if (col < rows) store(col >> 1, fmaf(v.y, 1.f / kSecond, v.x), fmaf(v.w, 1.f / kSecond, v.z));
            } else {
                if (col < rows) store(col, v.x, v.z);
                if (col + 1 < rows) store(col + 1, v.y, v.w);
            }
        }
        flip ^= 1;
    };

    // Spans: neighbouring groups whose rows are in shared memory together.
    int tile = first + mine, g0 = first / per;
    const int g_end = (last + per - 1) / per;
#pragma unroll 1
    while (g0 < g_end) {
        int g1 = g0, rows = 0;
        while (g1 < g_end) {
            const int n = rows_of(plan, plan.group[g1], most_rows);
            if (rows + n > room) break;
            rows += n;
            ++g1;
        }
        __syncthreads();  // the span before is done with
        find_rows(a, plan, g0, g1, most_rows);
        stage_rows<BITS, SB, ZP, NTMAX>(a, plan, rows, xs, sums);
        const int end = min(last, g1 * per);
        int g = g0;
#pragma unroll 1
        for (; tile < end; tile += G) {
            while (tile >= (g + 1) * per) ++g;
            const uint32_t group = plan.group[g];
            const int n = rows_of(plan, group, most_rows) << two, base = plan.base[g - g0] << two;
            if (NTMAX == 1 || n <= 8) run_tile(std::integral_constant<int, 1>{}, expert_of(group), tile - g * per, base, n);
            else run_tile(std::integral_constant<int, NTMAX>{}, expert_of(group), tile - g * per, base, n);
        }
        g0 = g1;
    }
    cp_wait<0>();
}

template <int BITS, int SB, bool ZP, int NT>
cudaError_t launch_one(Args a, cudaStream_t s) {
    using L = Layout<BITS, SB, ZP, NT>;
    const auto kern = expert_kernel<BITS, SB, ZP, NT>;
    const int avail = device_info().max_smem_optin - L::kFixed;
    int room = std::min(kMaxRows, a.P * a.terms);
    while (room > 0 && L::x_bytes(a.K, room) > avail) --room;
    if (room == 0) return cudaErrorNotSupported;
    if (room < a.terms) a.terms = 1;  // rows so long that one fits
    if (NT == 2 && room < kMaxRows && room < a.P * a.terms) return launch_one<BITS, SB, ZP, 1>(a, s);
    a.room = room;
    static std::atomic<unsigned long long> done{0};  // a bit for each device
    const int slot = device_slot();
    if (slot < 0 || !(done.load(std::memory_order_relaxed) >> slot & 1)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, device_info().max_smem_optin);
        if (e != cudaSuccess) return e;
        if (slot >= 0) done.fetch_or(1ull << slot, std::memory_order_relaxed);
    }
    return launch_pdl(kern, dim3(device_info().sm_count), dim3(kThreads), L::kFixed + L::x_bytes(a.K, room), s, a);
}

template <int BITS>
bool experts_fit(int K, int bs, bool zp) {
    const int most = device_info().max_smem_optin;
    if (bs == 32) return zp ? Layout<BITS, 32, true, 1>::kFixed + Layout<BITS, 32, true, 1>::x_bytes(K, 1) <= most : Layout<BITS, 32, false, 1>::kFixed + Layout<BITS, 32, false, 1>::x_bytes(K, 1) <= most;
    return zp ? Layout<BITS, 64, true, 1>::kFixed + Layout<BITS, 64, true, 1>::x_bytes(K, 1) <= most : Layout<BITS, 64, false, 1>::kFixed + Layout<BITS, 64, false, 1>::x_bytes(K, 1) <= most;
}

// Two columns of MMAs where more than eight tokens may meet at one expert.
template <int BITS>
cudaError_t launch_experts(const Args &a, cudaStream_t s) {
    const bool two = a.most_rows * a.terms > 8;
    if (a.bs == 32) {
        if (a.zp) return two ? launch_one<BITS, 32, true, 2>(a, s) : launch_one<BITS, 32, true, 1>(a, s);
        return two ? launch_one<BITS, 32, false, 2>(a, s) : launch_one<BITS, 32, false, 1>(a, s);
    }
    if (a.zp) return two ? launch_one<BITS, 64, true, 2>(a, s) : launch_one<BITS, 64, true, 1>(a, s);
    return two ? launch_one<BITS, 64, false, 2>(a, s) : launch_one<BITS, 64, false, 1>(a, s);
}

}  // namespace moe
}  // namespace qg
