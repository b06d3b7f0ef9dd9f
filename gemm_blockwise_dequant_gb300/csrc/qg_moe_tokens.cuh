// qg_moe_tokens.cuh -- the expert products of a mixture-of-experts layer over a few tokens (one instance file for each
// width of the codes).
//
//   fc1  h[p][i] = silu(g) u,  g, u = dequant(W1[e]) . x[token] + b1[e]     (rows i of both halves)
//   fc2  o[p][n] = dequant(W2[e]) . h[p] + b2[e]                            (p: one of the token's experts, e)
//
// Bound by memory: every chosen expert's weights are read once, and with few rows each there are few operations to a
// byte.  The pairs (token, slot) are grouped by expert, up to 16 rows to a group; a group's activations are laid out
// once in shared memory, as fp16 with a power of two for each row (so fp16, bf16 and fp32 rows alike keep 11 bits or
// more).  The weights go through m16n8k16 MMAs as the wide operand, 16 weight rows by 8 tokens: codes less the midpoint
// are whole numbers that fp16 holds exactly, one block's products are summed by the MMA and its scale is applied to
// the fp32 sums, so that nothing is rounded on the way.  A zero point other than the midpoint enters through the sum
// of the block's activations.
//
// Each warp streams its weights through a ring of its own (cp.async, no barrier between warps); S warps share a tile
// of 16 rows, each with a slice of K, and G = 16 / S tiles are worked on at a time.  S is chosen from the number of
// tiles, so that few of them still fill the warps.  A tile of fc1 is 8 gate rows and their 8 up rows: both values of an
// output meet in one lane.
#pragma once

#include <type_traits>

#include "qg_device.cuh"
#include "qg_moe_tokens.h"

namespace qg {
namespace moe {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kChunk = 128;  // values of K in a ring stage

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
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
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Codes of a width, SB values (32, or 64 where the blocks have them) of one row of a tile at a time: lane t of four
// holds SB / 4 neighbouring ones.  Rows in a stage lie kStride bytes apart, which keeps their reads free of bank conflicts.
template <int BITS, int SB>
struct Codes {
    static constexpr int kLane = SB / 4 * BITS / 8;            // bytes of a lane
    static constexpr int kRow = kChunk * BITS / 8;             // bytes of a row in a stage
    static constexpr int kCopy = BITS == 2 && SB == 32 ? 8 : 16;
    static constexpr int kCopies = kRow / kCopy;               // of a row
    static constexpr int kStride = BITS == 4 ? (SB == 32 ? 80 : 96) : BITS == 2 ? (SB == 32 ? 40 : 48) : (SB == 32 ? 160 : 192);
    static constexpr int kPerLane = kCopies / 2;               // copies of a lane: 16 rows, 32 lanes
    static constexpr float kMid = static_cast<float>(1 << (BITS - 1));
};

// Eight codes less the midpoint, as four pairs of fp16.  An fp16 of 1024 and more has its unit in the last place, so a
// code put there is 1024 + q; masked in place higher up, 1024 + 16 q (or 4 q), which one fma brings back.  Pair j holds
// the values order<BITS>(2 j) and order<BITS>(2 j + 1) of the eight.
template <int BITS>
__device__ __forceinline__ void unpack(uint32_t lo, uint32_t hi, uint32_t (&p)[4]) {
    constexpr uint32_t M = 0x64006400u;  // 1024, twice
    if constexpr (BITS == 4) {
        const uint32_t w = lo >> 8;
        p[0] = add2((lo & 0x000F000Fu) | M, 0xE408E408u);                       // - 1032
        p[1] = fma2((lo & 0x00F000F0u) | M, 0x2C002C00u, 0xD480D480u);          // / 16 - 72
        p[2] = add2((w & 0x000F000Fu) | M, 0xE408E408u);
        p[3] = fma2((w & 0x00F000F0u) | M, 0x2C002C00u, 0xD480D480u);
    } else if constexpr (BITS == 2) {
        const uint32_t v = (lo & 0xFFFFu) | (lo << 12), w = v >> 8;
        p[0] = add2((v & 0x00030003u) | M, 0xE402E402u);                        // - 1026
        p[1] = fma2((v & 0x000C000Cu) | M, 0x34003400u, 0xDC08DC08u);           // / 4 - 258
        p[2] = add2((w & 0x00030003u) | M, 0xE402E402u);
        p[3] = fma2((w & 0x000C000Cu) | M, 0x34003400u, 0xDC08DC08u);
    } else {
        p[0] = add2(__byte_perm(lo, 0x64646464u, 0x4140), 0xE480E480u);         // - 1152
        p[1] = add2(__byte_perm(lo, 0x64646464u, 0x4342), 0xE480E480u);
        p[2] = add2(__byte_perm(hi, 0x64646464u, 0x4140), 0xE480E480u);
        p[3] = add2(__byte_perm(hi, 0x64646464u, 0x4342), 0xE480E480u);
    }
}
template <int BITS>
__device__ __forceinline__ constexpr int order(int i) {
    return BITS == 4 ? (i >> 1) + 4 * (i & 1) : BITS == 2 ? (i & 4) + ((i >> 1) & 1) + 2 * (i & 1) : i;
}

// Shared memory: the ring of every warp, the partial sums, the group's activations and their block sums, the plan.
template <int BITS, int SB, bool ZP, int NT>
struct Layout {
    using C = Codes<BITS, SB>;
    static constexpr int kParRow = SB == 32 ? 12 : 8;          // words of two scales: up to four scales at any place, or two
    static constexpr int kParams = 16 * kParRow;
    static constexpr int kStage = 16 * C::kStride + kParams * (ZP ? 2 : 1);
    // enough in flight to cover the latency: about 3 KB of codes a warp
    static constexpr int kStages = BITS == 8 ? (NT == 1 ? 3 : 2) : BITS == 4 ? (NT == 1 ? 5 : 4) : (NT == 1 ? 8 : 6);
    static constexpr int kRing = kWarps * kStages * kStage;
    static constexpr int kPartial = 2 * kWarps * 32 * NT * 16;
    static constexpr int kPlan = kMaxPairs * 2 + kMaxExperts * 4 + kMaxPairs * 4 + 16 * 16;
    static constexpr int kFixed = kRing + kPartial + kPlan + 256;
    static __host__ __device__ int x_stride(int K) { return SB == 32 ? K * 2 + (K % 64 == 0 ? 64 : 0) : K * 2 + 16; }
    static __host__ __device__ int x_bytes(int K, int rows) { return rows * x_stride(K) + (ZP ? K / SB * NT * 8 * 4 : 0); }
    static_assert(kFixed % 16 == 0 && kStage % 16 == 0, "alignment");
};

struct Plan {
    int16_t *ids;       // [pairs], -1: none
    int *count;         // [experts], then the groups before
    uint32_t *group;    // [groups]: expert << 16 | first row's rank
    int *rows;          // [16]: the pairs of the current group
    unsigned *top;      // [16]: largest magnitude of a row, as bits
    float *back;        // [16]: the power of two that undoes its scale
    int *num;           // groups
};

// Groups the pairs by expert, at most `limit` rows to a group.
__device__ __forceinline__ void make_plan(const Args &a, const Plan &p, int limit) {
    const int tid = threadIdx.x;
    for (int e = tid; e < a.E; e += kThreads) p.count[e] = 0;
    __syncthreads();
    bool bad = false;
    for (int i = tid; i < a.P; i += kThreads) {
        const int e = a.ids[i];
        const bool ok = e >= 0 && e < a.E;
        p.ids[i] = static_cast<int16_t>(ok ? e : -1);
        if (ok) atomicAdd(&p.count[e], 1);
        bad |= !ok;
    }
    if (bad && a.status && blockIdx.x == 0) *a.status = 1;
    __syncthreads();
    if (tid < 32) {
        int before = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + tid, n = e < a.E ? (p.count[e] + limit - 1) / limit : 0;
            int sum = n;
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(~0u, sum, o);
                if (tid >= o) sum += v;
            }
            for (int j = 0; j < n; ++j) p.group[before + sum - n + j] = static_cast<uint32_t>(e) << 16 | static_cast<uint32_t>(j * limit);
            before += __shfl_sync(~0u, sum, 31);
        }
        if (tid == 0) *p.num = before;
    }
    __syncthreads();
}

// The pairs of a group, in their order; returns how many.
__device__ __forceinline__ int find_rows(const Args &a, const Plan &p, uint32_t group, int limit) {
    const int tid = threadIdx.x, e = static_cast<int>(group >> 16), first = static_cast<int>(group & 0xFFFFu);
    __syncthreads();  // the group before is done with
    if (tid < 32) {
        int n = 0;
        for (int i0 = 0; i0 < a.P && n < first + limit; i0 += 32) {
            const bool is = i0 + tid < a.P && p.ids[i0 + tid] == e;
            const unsigned who = __ballot_sync(~0u, is);
            const int at = n + __popc(who & ((1u << tid) - 1u));
            if (is && at >= first && at < first + limit) p.rows[at - first] = i0 + tid;
            n += __popc(who);
        }
        if (tid < 16) p.top[tid] = 0;
        if (tid == 0) p.num[1] = min(limit, n - first);
    }
    __syncthreads();
    return p.num[1];
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

// The group's activations as scaled fp16, eight at a time in the order of the codes' pairs; rows past the last are zero.
template <int BITS, int SB, bool ZP, int NT>
__device__ void stage_rows(const Args &a, const Plan &p, int n, int room, char *xs, float *sums) {
    constexpr int R = 8 * NT, TPR = kThreads / R;
    const int tid = threadIdx.x, r = tid / TPR, lane = tid % TPR, stride = Layout<BITS, SB, ZP, NT>::x_stride(a.K);
    const int64_t row = r < n ? (a.fc == 1 ? p.rows[r] / a.k : p.rows[r]) : 0;
    float top = 0.f;
    if (r < n)
        for (int q = lane; q < a.K / 8; q += TPR) {
            float x[8];
            load_values(a.src, a.src_dtype, static_cast<size_t>(row) * a.K + q * 8, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, finite_abs(x[i]));
        }
    for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    if ((tid & 31) == 0) atomicMax(&p.top[r], __float_as_uint(top));
    __syncthreads();
    // the largest between 2^14 and 2^15: fp16 keeps 11 bits of whatever is above 2^-29 of it, and sums stay far from fp32's range
    const unsigned bits = p.top[r];
    const int e = bits >= 0x00800000u ? 14 - (static_cast<int>(bits >> 23) - 127) : bits ? 127 : 0, up = min(e, 127);
    const float scale = exp2i(max(up, -126)), low = e > 127 ? exp2i(e - 127) : 1.f;
    if (lane == 0) p.back[r] = exp2i(-max(up, -126)) / low;
    for (int q = lane; q < a.K / 8; q += TPR) {
        uint32_t w[4] = {0, 0, 0, 0};
        float sum = 0.f;
        if (r < n) {
            float x[8];
            load_values(a.src, a.src_dtype, static_cast<size_t>(row) * a.K + q * 8, x);
            uint16_t h[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h[i] = f2h(x[i] * scale * low);
                if constexpr (ZP) sum += h2f(h[i]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = h[order<BITS>(2 * i)] | static_cast<uint32_t>(h[order<BITS>(2 * i + 1)]) << 16;
        }
        if (r < room) *reinterpret_cast<uint4 *>(xs + r * stride + q * 16) = make_uint4(w[0], w[1], w[2], w[3]);
        if constexpr (ZP) {
            // SB / 8 neighbouring threads hold a block, and all of them are here: K / 8 is a multiple of SB / 8
            const unsigned quad = ((1u << (SB / 8)) - 1u) << (tid & 31 & ~(SB / 8 - 1));
            for (int o = 1; o < SB / 8; o <<= 1) sum += __shfl_xor_sync(quad, sum, o);
            if (q % (SB / 8) == 0) sums[(q / (SB / 8)) * (8 * NT) + r] = sum;
        }
    }
    __syncthreads();
}

// Where a warp is in its sequence of tiles and chunks.
struct Cursor {
    int g, tile, end, u;  // group, tile of all, the CTA's end in this group, unit of K
};

template <int BITS, int SB, bool ZP, int NTMAX>
__global__ void __launch_bounds__(kThreads, 1) expert_kernel(const __grid_constant__ Args a) {
    using C = Codes<BITS, SB>;
    using L = Layout<BITS, SB, ZP, NTMAX>;
    constexpr int D = L::kStages, CU = kChunk / SB;
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
    plan.top = reinterpret_cast<unsigned *>(plan.rows + 16);
    plan.back = reinterpret_cast<float *>(plan.rows + 32);
    plan.num = plan.rows + 48;
    char *xs = smem + L::kFixed;
    float *sums = reinterpret_cast<float *>(xs + a.room * L::x_stride(a.K));
    const int x_stride = L::x_stride(a.K);

    pdl_wait();
    pdl_launch_dependents();
    make_plan(a, plan, a.room);
    const int groups = *plan.num, per = a.fc == 1 ? a.N / 16 : (a.N + 15) / 16;
    const int total = groups * per;
    const int first = static_cast<int>(static_cast<int64_t>(total) * blockIdx.x / gridDim.x), last = static_cast<int>(static_cast<int64_t>(total) * (blockIdx.x + 1) / gridDim.x);
    if (first >= last) return;
    // Slices of K: the fewest rounds of G tiles, a round's cost being its units and about four more to join the slices
    const int units = a.K / SB, most = (total + gridDim.x - 1) / gridDim.x;
    int S = 1, cost = 1 << 30;
    for (int s = 1; s <= kWarps; s *= 2) {
        const int c = ((most * s + kWarps - 1) / kWarps) * ((units + s - 1) / s + 4 * 32 / SB);
        if (c < cost) cost = c, S = s;
    }
    const int G = kWarps / S, mine = warp / S, slice = warp % S;
    const int u0 = units * slice / S, u1 = units * (slice + 1) / S;

    const int nb = a.K / a.bs, row_bytes = a.K * BITS / 8;
    const auto weight_row = [&](int tile, int r) {  // the weight row of a tile's row r
        if (a.fc == 2) return tile * 16 + r;
        const int i = tile * 8 + (r & 7);
        return a.interleaved ? 2 * i + (r >> 3) : (r >> 3) * (a.N / 2) + i;
    };
    const auto settle = [&](Cursor &c) {  // on to the group that has a tile for this warp
        while (c.tile >= c.end && c.end < last) {
            ++c.g;
            c.tile = c.end + mine;
            c.end = min(last, c.end + per);
        }
    };
    Cursor ahead{first / per, first + mine, min(last, (first / per + 1) * per), u0}, now = ahead;
    settle(ahead);

    // what this lane copies of the tile at `ahead`
    const char *src[C::kPerLane];
    const uint16_t *ssrc = nullptr, *zsrc = nullptr;
    size_t srow = 0;  // index of the row's first scale
    const auto open = [&]() {
        if (ahead.tile >= last) return;
        const int64_t e = plan.group[ahead.g] >> 16;
        const int tile = ahead.tile - ahead.g * per;
#pragma unroll
        for (int i = 0; i < C::kPerLane; ++i) {
            const int r = lane / C::kCopies + i * (32 / C::kCopies);
            src[i] = reinterpret_cast<const char *>(a.w) + (e * a.N + weight_row(tile, r)) * row_bytes + (lane % C::kCopies) * C::kCopy;
        }
        srow = static_cast<size_t>(e * a.N + weight_row(tile, lane >> 1)) * nb;
        ssrc = a.scales;
        zsrc = a.zp;
    };
    open();
    int fill = 0;
    const auto issue = [&]() {
        if (ahead.tile < last) {
            const uint32_t stage = smem_u32(ring + fill * L::kStage);
            const int left = (u1 - ahead.u) * SB;  // values of K still there
            const int kb = ahead.u * SB * BITS / 8;
#pragma unroll
            for (int i = 0; i < C::kPerLane; ++i) {
                const int r = lane / C::kCopies + i * (32 / C::kCopies), part = lane % C::kCopies;
                if (part * (C::kCopy * 8 / BITS) < left) {
                    if constexpr (C::kCopy == 16) cp_async16(stage + r * C::kStride + part * 16, src[i] + kb);
                    else cp_async8(stage + r * C::kStride + part * 8, src[i] + kb);
                }
            }
            // words of two scales from the one that holds the chunk's first
            const int k0 = ahead.u * SB, k1 = k0 + min(left, kChunk) - 1;
            const size_t w0 = (srow + k0 / a.bs) >> 1, w1 = (srow + k1 / a.bs) >> 1;
#pragma unroll
            for (int i = 0; i < (SB == 32 ? 2 : 1); ++i) {
                const int w = (lane & 1) + 2 * i;
                if (w0 + w <= w1) {
                    cp_async4(stage + 16 * C::kStride + (lane >> 1) * L::kParRow + w * 4, reinterpret_cast<const uint32_t *>(ssrc) + w0 + w);
                    if constexpr (ZP) cp_async4(stage + 16 * C::kStride + L::kParams + (lane >> 1) * L::kParRow + w * 4, reinterpret_cast<const uint32_t *>(zsrc) + w0 + w);
                }
            }
            if (++fill == D) fill = 0;
            ahead.u += CU;
            if (ahead.u >= u1) {
                ahead.u = u0;
                ahead.tile += G;
                settle(ahead);
                open();
            }
        }
        cp_commit();
    };
#pragma unroll 1
    for (int i = 0; i < D - 1; ++i)
        if (u0 < u1) issue();
        else cp_commit();

    int drain = 0, flip = 0;
    const auto run_group = [&](auto nt_tag, int expert, int rows, int begin, int end) {
        constexpr int NT = decltype(nt_tag)::value;
#pragma unroll 1
        for (int tile_all = begin + mine; tile_all < end; tile_all += G) {
            const int tile = tile_all - now.g * per;
            const int n0 = weight_row(tile, g8), n1 = weight_row(tile, g8 + 8);
            const int odd0 = static_cast<int>((static_cast<int64_t>(expert) * a.N + n0) * nb & 1), odd1 = static_cast<int>((static_cast<int64_t>(expert) * a.N + n1) * nb & 1);
            float sum[NT][4];
#pragma unroll
            for (int j = 0; j < NT; ++j) sum[j][0] = sum[j][1] = sum[j][2] = sum[j][3] = 0.f;
#pragma unroll 1
            for (int u = u0; u < u1; u += CU) {
                cp_wait<D - 2>();
                __syncwarp();
                const char *stage = ring + drain * L::kStage;
                const int b0 = u * SB / a.bs;
                const uint16_t *sc = reinterpret_cast<const uint16_t *>(stage + 16 * C::kStride);
                const uint16_t *sp0 = sc + g8 * (L::kParRow / 2) + ((odd0 + b0) & 1) - b0, *sp1 = sc + (g8 + 8) * (L::kParRow / 2) + ((odd1 + b0) & 1) - b0;
#pragma unroll
                for (int v = 0; v < CU; ++v) {
                    if (u + v < u1) {
                        uint32_t c0[4], c1[4];
                        const char *row0 = stage + g8 * C::kStride + v * (C::kLane * 4) + t4 * C::kLane, *row1 = row0 + 8 * C::kStride;
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
                        for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
#pragma unroll
                        for (int h = 0; h < SB / 32; ++h) {
                            uint32_t p[4], q[4];
                            if constexpr (BITS == 8) {
                                unpack<8>(c0[2 * h], c0[2 * h + 1], p);
                                unpack<8>(c1[2 * h], c1[2 * h + 1], q);
                            } else if constexpr (BITS == 4) {
                                unpack<4>(c0[h], 0, p);
                                unpack<4>(c1[h], 0, q);
                            } else {
                                unpack<2>(c0[0] >> (16 * h), 0, p);
                                unpack<2>(c1[0] >> (16 * h), 0, q);
                            }
#pragma unroll
                            for (int j = 0; j < NT; ++j) {
                                const int token = min(j * 8 + g8, a.room - 1);  // columns past the last row are not looked at
                                const uint4 b = *reinterpret_cast<const uint4 *>(xs + token * x_stride + ((u + v) * SB + t4 * (SB / 4) + h * 8) * 2);
                                mma16816(acc[j], p[0], q[0], p[1], q[1], b.x, b.y);
                                mma16816(acc[j], p[2], q[2], p[3], q[3], b.z, b.w);
                            }
                        }
                        const int b = (u + v) * SB / a.bs;
                        const float s0 = h2f(sp0[b]), s1 = h2f(sp1[b]);
                        [[maybe_unused]] float z0 = 0.f, z1 = 0.f;
                        if constexpr (ZP) {
                            z0 = C::kMid - h2f(sp0[b + L::kParams / 2]);
                            z1 = C::kMid - h2f(sp1[b + L::kParams / 2]);
                        }
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            if constexpr (ZP) {
                                const float2 xsum = *reinterpret_cast<const float2 *>(sums + (u + v) * (8 * NTMAX) + j * 8 + 2 * t4);
                                acc[j][0] = fmaf(z0, xsum.x, acc[j][0]);
                                acc[j][1] = fmaf(z0, xsum.y, acc[j][1]);
                                acc[j][2] = fmaf(z1, xsum.x, acc[j][2]);
                                acc[j][3] = fmaf(z1, xsum.y, acc[j][3]);
                            }
                            sum[j][0] = fmaf(s0, acc[j][0], sum[j][0]);
                            sum[j][1] = fmaf(s0, acc[j][1], sum[j][1]);
                            sum[j][2] = fmaf(s1, acc[j][2], sum[j][2]);
                            sum[j][3] = fmaf(s1, acc[j][3], sum[j][3]);
                        }
                    }
                }
                __syncwarp();  // everyone has read the stage that the next copy goes to
                if (++drain == D) drain = 0;
                issue();
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
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int r = j * 8 + 2 * t4 + c;
                    if (r >= rows) continue;
                    const float back = plan.back[r];
                    const float p = fmaf(c ? v.y : v.x, back, bias0), q = fmaf(c ? v.w : v.z, back, bias1);
                    const int64_t pair = plan.rows[r];
                    if (a.fc == 1) {
                        a.out[pair * (a.N / 2) + tile * 8 + g8] = p / (1.f + __expf(-p)) * q;
                    } else {
                        a.out[pair * a.N + n0] = p;
                        a.out[pair * a.N + n1] = q;
                    }
                }
            }
            flip ^= 1;
        }
    };
#pragma unroll 1
    for (int begin = first; begin < last; begin = now.end, ++now.g, now.end = min(last, begin + per)) {
        const uint32_t group = plan.group[now.g];
        const int rows = find_rows(a, plan, group, a.room);
        stage_rows<BITS, SB, ZP, NTMAX>(a, plan, rows, a.room, xs, sums);
        if (NTMAX == 1 || rows <= 8) run_group(std::integral_constant<int, 1>{}, static_cast<int>(group >> 16), rows, begin, now.end);
        else run_group(std::integral_constant<int, NTMAX>{}, static_cast<int>(group >> 16), rows, begin, now.end);
    }
    cp_wait<0>();
}

template <int BITS, int SB, bool ZP, int NT>
cudaError_t launch_one(Args a, cudaStream_t s) {
    using L = Layout<BITS, SB, ZP, NT>;
    const auto kern = expert_kernel<BITS, SB, ZP, NT>;
    const int avail = device_info().max_smem_optin - L::kFixed;
    int room = 8 * NT;
    while (room > 0 && L::x_bytes(a.K, room) > avail) --room;
    if (room == 0) return cudaErrorNotSupported;
    if (NT == 2 && room < 16) return launch_one<BITS, SB, ZP, 1>(a, s);
    a.room = room;
    const int smem = L::kFixed + L::x_bytes(a.K, room);
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(device_info().sm_count), dim3(kThreads), smem, s, a);
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
    const bool two = a.most_rows > 8;
    if (a.bs == 32) {
        if (a.zp) return two ? launch_one<BITS, 32, true, 2>(a, s) : launch_one<BITS, 32, true, 1>(a, s);
        return two ? launch_one<BITS, 32, false, 2>(a, s) : launch_one<BITS, 32, false, 1>(a, s);
    }
    if (a.zp) return two ? launch_one<BITS, 64, true, 2>(a, s) : launch_one<BITS, 64, true, 1>(a, s);
    return two ? launch_one<BITS, 64, false, 2>(a, s) : launch_one<BITS, 64, false, 1>(a, s);
}

}  // namespace moe
}  // namespace qg
