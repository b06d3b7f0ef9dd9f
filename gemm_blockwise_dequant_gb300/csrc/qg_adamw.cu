// qg_adamw.cu -- one AdamW step over a list of tensors, with states in fp32 or in 8 bits, and the clipping of the
// gradients by their global norm in the same call.
//
//   c  = min(1, max_norm / (norm + norm_eps)),  g' = c g          (1 without clipping)
//   m' = b1 m + (1 - b1) g',  v' = b2 v + (1 - b2) g'^2
//   p' = p (1 - lr wd) - lr (m' / (1 - b1^step)) / (sqrt(v' / (1 - b2^step)) + eps)
//
// 8-bit states are e4m3 codes of m' and of u' = sqrt(v') times an fp32 scale for every 256 values (the largest
// magnitude / 448): u' needs half of v's range of exponents, which e4m3 has.  The step itself uses m' and u' before
// that rounding.  A u' above zero is never stored as zero, which m' / u' of a later step could not bear.
//
// Bound by memory.  The list is cut into chunks of 4096 values; a thread owns 8 neighbouring ones and a warp one
// block of 256 at a time, so that a block's largest magnitude is a warp reduction.  With clipping a first launch reads the
// gradients alone and leaves one sum of squares for each CTA; the second takes the chunks from the last one on, where
// the L2 still holds the gradients that were read last.
//
// Measured: 56.5 million bf16 values with 8-bit states, clipped, 149 us (the norm 30 us for 113 MB; the step alone 111, 4.6 TB/s, the L1 busy
// for 79% of it and 59% of the issue slots taken); 419 million with fp32 states and master copies, clipped, 2.0 ms (6 TB/s over
// both launches); 1.4 million fp32 values 8.6 us, which is latency.
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>

#include "../../include/qgemm.h"
#include "qg_device.cuh"
#include "qg_internal.h"

namespace qg {
namespace {

constexpr int kThreads = 256;              // of a group: a CTA is kGroups of them, one CTA on each SM
constexpr int kGroups = 3;
constexpr int kVals = 8;                   // of a thread
constexpr int kPart = kThreads * kVals;    // values that a group takes at a time
constexpr int kChunk = 2 * kPart;          // looked up at a time
constexpr float kCodeMax = 448.f;          // the largest e4m3 value
constexpr float kTinyBlock = 1e-30f;       // a block with no larger magnitude is stored as zeros (448 / it stays finite)

__device__ __forceinline__ uint4 load128(const void *p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// Eight values at element e of an array as they lie there (n: those that exist, zero where there are none): one vector
// of 16-bit values, two of fp32.  They become numbers apart from this, so that a thread's loads are all on their way
// before it waits for the first.  WIDE: eight there, at whole vectors.
struct Eight {
    uint4 a, b;
};
template <bool WIDE>
__device__ __forceinline__ Eight raw8(const void *base, int dtype, int64_t e, int n) {
    Eight r;
    const char *p = static_cast<const char *>(base) + e * (dtype == 0 ? 4 : 2);
    if constexpr (WIDE) {
        r.a = load128(p);
        if (dtype == 0) r.b = load128(p + 16);
        return r;
    }
    uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (dtype == 0) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < n) w[k] = reinterpret_cast<const uint32_t *>(p)[k];
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < n) w[k >> 1] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(p)[k]) << (16 * (k & 1));
    }
    r.a = make_uint4(w[0], w[1], w[2], w[3]), r.b = make_uint4(w[4], w[5], w[6], w[7]);
    return r;
}
__device__ __forceinline__ void numbers(const Eight &r, int dtype, float (&x)[8]) {
    const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
    if (dtype == 0) {  // the types apart: a choice of each value would convert it every way
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = __uint_as_float(w[k]);
    } else if (dtype == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i] = h2f(static_cast<uint16_t>(w[i] & 0xFFFFu)), x[2 * i + 1] = h2f(static_cast<uint16_t>(w[i] >> 16));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

template <bool WIDE = false>
__device__ __forceinline__ void store8(void *base, int dtype, int64_t e, int n, const float (&x)[8]) {
    if (dtype == 0) {
        float *p = static_cast<float *>(base) + e;
        if (WIDE || (n == 8 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0)) {
            reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
            reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < n) p[k] = x[k];
        }
        return;
    }
    uint16_t *p = static_cast<uint16_t *>(base) + e;
    uint32_t w[4];
    if (dtype == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    if (WIDE || (n == 8 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0)) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < n) p[k] = static_cast<uint16_t>(w[k >> 1] >> (16 * (k & 1)));
    }
}

// Eight e4m3 codes.
template <bool WIDE>
__device__ __forceinline__ uint2 load_codes(const void *base, int64_t e, int n) {
    const uint8_t *p = static_cast<const uint8_t *>(base) + e;
    if constexpr (WIDE) {
        uint2 v;
        asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
        return v;
    }
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (k < n) w[k >> 2] |= static_cast<uint32_t>(p[k]) << (8 * (k & 3));
    return make_uint2(w[0], w[1]);
}
template <bool WIDE>
__device__ __forceinline__ void store_codes(void *base, int64_t e, int n, uint2 c) {
    uint8_t *p = static_cast<uint8_t *>(base) + e;
    if (WIDE || (n == 8 && (reinterpret_cast<uintptr_t>(p) & 7u) == 0)) {
        *reinterpret_cast<uint2 *>(p) = c;
        return;
    }
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (k < n) p[k] = static_cast<uint8_t>(w[k >> 2] >> (8 * (k & 3)));
}
__device__ __forceinline__ void decode(uint2 c, float (&x)[8]) {
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
        x[2 * i] = h2f(h.x), x[2 * i + 1] = h2f(h.y);
    }
}
// The largest of a warp's values that are not negative (a NaN is one: its bits are above all).
__device__ __forceinline__ float warp_top(float x) { return __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(x))); }

// To a unit in the last place; of 2^126 and more 0.
__device__ __forceinline__ float reciprocal(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two products at a time (packed fp32).
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n .reg .b64 ra, rb, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %5};\n mul.rn.f32x2 rd, ra, rb;\n mov.b64 {%0, %1}, rd;\n}\n"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// Codes of x / scale for the warp's block of 256 values; scale is what goes with them.
template <bool KEEP>
__device__ __forceinline__ uint2 encode(const float (&x)[8], float &scale) {
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(x[k]));
    top = warp_top(top);
    // infinities: the codes of the others are zeros, and the state shows it (0 * inf is NaN); a NaN is a code of its own
    // x * (448 / top) and top / 448 as reciprocals and products, each rounded by itself, as a plain fp32 program has them: which of two evaluations
    // is nearer matters less than that they are the same (a unit in the last place moves one of a million values to the next code).
    const float inv = top >= kTinyBlock ? kCodeMax * __frcp_rn(top) : 0.f;
    scale = top >= kTinyBlock ? top * (1.f / kCodeMax) : 0.f;
    uint32_t w[2] = {0, 0};
    float2 y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = mul2(make_float2(x[2 * i], x[2 * i + 1]), both(inv));
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i >> 1] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(y[i].x, y[i].y), __NV_SATFINITE, __NV_E4M3)) << (16 * (i & 1));
    if constexpr (KEEP) {  // what is above zero stays above
        if (((w[0] - 0x01010101u) & ~w[0] & 0x80808080u) | ((w[1] - 0x01010101u) & ~w[1] & 0x80808080u)) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (x[k] * inv > 0.f && !(w[k >> 2] >> (8 * (k & 3)) & 0xFFu)) w[k >> 2] |= 1u << (8 * (k & 3));
        }
    }
    return make_uint2(w[0], w[1]);
}

// The list as a CTA sees it, in shared memory (longer lists take more launches).  The chunks of all tensors, one after
// another, are dealt out in turn, so that all SMs work side by side in memory: each with a run of its own they would open
// as many DRAM pages at a time as there are runs and arrays (55.7 million values with 8-bit states: 153 us, 93 side by
// side).  Every warp looks up each chunk's tensor.
constexpr int kTable = 512;  // entries
struct Entry {
    void *param;
    const void *grad;
    void *m, *v;
    float *sm, *sv;
    float *master;
    int64_t numel;
    int first;  // chunk
    float decay;
    short kind, state, param_dtype, grad_dtype;
};
enum Kind { ANY, WIDE_F32, WIDE_E4M3, WIDE_E4M3_F16, WIDE_E4M3_BF16 };  // WIDE: every array at whole vectors

__device__ __forceinline__ int kind_of(const qg_adamw_tensor &t) {
    const uintptr_t all = reinterpret_cast<uintptr_t>(t.param) | reinterpret_cast<uintptr_t>(t.grad) | reinterpret_cast<uintptr_t>(t.master);
    const uintptr_t states = reinterpret_cast<uintptr_t>(t.exp_avg) | reinterpret_cast<uintptr_t>(t.exp_avg_sq);
    if ((all & 15u) != 0 || (states & (t.state == QG_STATE_E4M3 ? 7u : 15u)) != 0) return ANY;
    if (t.state != QG_STATE_E4M3) return WIDE_F32;
    if (t.master || t.param_dtype == 0 || t.param_dtype != t.grad_dtype) return WIDE_E4M3;
    return t.param_dtype == 1 ? WIDE_E4M3_F16 : WIDE_E4M3_BF16;
}

struct List {
    const Entry *t;
    int count;

    // All threads call it.
    __device__ __forceinline__ List(const qg_adamw_tensor *list, int n, char *room) : t(reinterpret_cast<const Entry *>(room)), count(n) {
        for (int i = threadIdx.x; i < n; i += kThreads * kGroups) {
            const qg_adamw_tensor &q = list[i];
            reinterpret_cast<Entry *>(room)[i] = {q.param, q.grad, q.exp_avg, q.exp_avg_sq, q.exp_avg_scale, q.exp_avg_sq_scale, q.master, q.numel,
                                                  static_cast<int>(q.first_chunk), q.weight_decay, static_cast<short>(kind_of(q)), static_cast<short>(q.state),
                                                  static_cast<short>(q.param_dtype), static_cast<short>(q.grad_dtype)};
        }
        __syncthreads();
    }
    // The tensor owning chunk c: the last one with first <= c (a warp finds it, 32 steps at a time).
    __device__ __forceinline__ int find(int c) const {
        const int lane = threadIdx.x & 31;
        int lo = 0, n = count;
        while (n > 1) {
            const int step = (n + 31) / 32, i = lo + lane * step;
            const unsigned who = __ballot_sync(~0u, lane * step < n && t[i].first <= c);  // ones first
            const int last = __popc(who) - 1;
            n = min(step, n - last * step);
            lo += last * step;
        }
        return lo;
    }
    // The same where it is not behind entry i, and likely near.
    __device__ __forceinline__ int find_before(int i, int c) const {
        const int at = i - static_cast<int>(threadIdx.x & 31);
        const unsigned who = __ballot_sync(~0u, at >= 0 && t[max(at, 0)].first <= c);
        return who ? i - (__ffs(who) - 1) : find(c);
    }
};
int list_bytes(int count) { return std::min(count, kTable) * static_cast<int>(sizeof(Entry)); }
static_assert(sizeof(Entry) % 16 == 0, "read in 16-byte pieces");

// Nothing but zeros: eight squares whose sum is 0 may also have left fp32's range.
__device__ __forceinline__ bool all_zero(const float (&g)[8]) {
    uint32_t any = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) any |= __float_as_uint(g[k]);
    return any << 1 == 0;
}
// The sum of squares of eight values in fp32, or in fp64 where that leaves its range.
__device__ __forceinline__ double squares(const float (&g)[8]) {
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 8; ++k) s[k & 1] = fmaf(g[k], g[k], s[k & 1]);
    const float sum = s[0] + s[1];
    if ((sum >= 1e-30f && sum <= 3e38f) || all_zero(g)) return sum;
    double wide = 0.0;
#pragma unroll
    for (int k = 0; k < 8; ++k) wide += static_cast<double>(g[k]) * g[k];
    return wide;
}

// The sum of squares of whole parts of one tensor, of eight at most (four of fp32): all loads of a thread together.
template <int DT>
__device__ __forceinline__ double squares_of_some(const void *grad, int64_t e, int parts) {
    constexpr int U = DT == 0 ? 2 : 1, N = 8 / U;
    uint4 v[N][U];
    const char *p = static_cast<const char *>(grad) + e * (DT == 0 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int u = 0; u < U; ++u) v[i][u] = i < parts ? load128(p + i * (kPart * (DT == 0 ? 4 : 2)) + u * 16) : make_uint4(0, 0, 0, 0);
    double total = 0.0;
    float s = 0.f;
    bool fits = true;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float g[8], q[2] = {0.f, 0.f};
        numbers({v[i][0], v[i][U - 1]}, DT, g);
#pragma unroll
        for (int k = 0; k < 8; ++k) q[k & 1] = fmaf(g[k], g[k], q[k & 1]);
        const float sum = q[0] + q[1];
        // zeros (of tensors that no token reached) are as quick as other gradients: they took 2.8 times as long one by one
        fits = fits && ((sum >= 1e-30f && sum <= 3e37f) || all_zero(g));
        s += sum;
    }
    if (fits) return s;
#pragma unroll 1
    for (int i = 0; i < parts; ++i) {  // again, one by one
        float g[8];
        numbers(raw8<true>(grad, DT, e + static_cast<int64_t>(i) * kPart, 8), DT, g);
        total += squares(g);
    }
    return total;
}

// One sum of squares for each CTA; added to what is there (the entries before these).
__global__ void __launch_bounds__(kThreads * kGroups, 1) sumsq_kernel(const qg_adamw_tensor *__restrict__ list, int count, int more, int64_t chunks,
                                                                     double *__restrict__ partial, int add) {
    __shared__ double red[kThreads * kGroups / 32];
    extern __shared__ __align__(16) char room[];
    pdl_wait();
    pdl_launch_dependents();
    double total = 0.0;
    const List l(list, count, room);
    const int begin = l.t[0].first / 4, last = static_cast<int>(more ? list[count].first_chunk : chunks);  // of four chunks; chunks
    for (int turn = begin + blockIdx.x * kGroups + threadIdx.x / kThreads; turn * 4 < last; turn += gridDim.x * kGroups) {
        const int end = min(last, turn * 4 + 4);
        for (int c = max(turn * 4, l.t[0].first); c < end;) {
            const Entry &t = l.t[l.find(c)];
            const void *grad = t.grad;
            const int dt = t.grad_dtype, after = min(end, t.first + static_cast<int>((t.numel + kChunk - 1) / kChunk));
            const bool wide = (reinterpret_cast<uintptr_t>(grad) & 15u) == 0;
            const int64_t e0 = static_cast<int64_t>(c - t.first) * kChunk, e1 = std::min<int64_t>(t.numel, static_cast<int64_t>(after - t.first) * kChunk);
            for (int64_t e = e0; e < e1;) {
                const int64_t mine = e + threadIdx.x % kThreads * kVals;
                const int some = wide ? static_cast<int>(std::min<int64_t>((e1 - e) / kPart, dt == 0 ? 4 : 8)) : 0;
                if (some > 0) {
                    total += dt == 0 ? squares_of_some<0>(grad, mine, some) : dt == 1 ? squares_of_some<1>(grad, mine, some) : squares_of_some<2>(grad, mine, some);
                    e += static_cast<int64_t>(some) * kPart;
                    continue;
                }
                const int64_t left = t.numel - mine;
                if (left > 0) {
                    float g[8];
                    numbers(wide && left >= 8 ? raw8<true>(grad, dt, mine, 8) : raw8<false>(grad, dt, mine, left < 8 ? static_cast<int>(left) : 8), dt, g);
                    total += squares(g);
                }
                e += kPart;
            }
            c = after;
        }
    }
    for (int o = 16; o >= 1; o >>= 1) total += __shfl_xor_sync(~0u, total, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = total;
    __syncthreads();
    if (threadIdx.x == 0) {
        total = add ? partial[blockIdx.x] : 0.0;
        for (int w = 0; w < kThreads * kGroups / 32; ++w) total += red[w];
        partial[blockIdx.x] = total;
    }
}

struct StepArgs {
    const qg_adamw_tensor *list;
    int count, more;  // entries of this launch, and whether others follow
    int64_t chunks;
    float lr, beta1, beta2, keep1, keep2, ln1, ln2, eps, one;  // keep = 1 - beta, ln = log(beta), one = 1
    const float *lr_dev;
    float step;
    const int64_t *step_dev;
    const double *partial;  // null: no clipping
    int parts;
    float max_norm, norm_eps;
    float *norm;
};

// What a step multiplies with.
struct Rates {
    float clip;               // of a gradient
    float rate, widen, lr;    // lr / (1 - b1^step), 1 / sqrt(1 - b2^step)
};

// What a thread reads of a chunk.
struct Raw {
    Eight w, g, m, v;
    uint2 cm, cv;
    float sm, sv;
};
template <bool WIDE, bool EIGHT>
__device__ __forceinline__ void fetch8(Raw &x, const Entry &t, int64_t e, int n) {
    x.g = raw8<WIDE>(t.grad, t.grad_dtype, e, n);
    x.w = t.master ? raw8<WIDE>(t.master, 0, e, n) : raw8<WIDE>(t.param, t.param_dtype, e, n);
    if constexpr (EIGHT) {
        x.cm = load_codes<WIDE>(t.m, e, n), x.cv = load_codes<WIDE>(t.v, e, n);
        const int64_t block = e >> 8;
        const bool there = WIDE || block << 8 < t.numel;
        x.sm = there ? t.sm[block] : 0.f, x.sv = there ? t.sv[block] : 0.f;
    } else {
        x.m = raw8<WIDE>(t.m, 0, e, n);
        x.v = raw8<WIDE>(t.v, 0, e, n);
    }
}

// Two roots: a step of Newton's iteration, s + (x - s s) / (2 sqrt(x)), from the approximate s = x / sqrt(x).  Compared with the IEEE root for every fp32 x: the
// same from 2^-102 on, off by a unit in the last place for some below, by two for some subnormal ones.
// The product at the end is below every root and stands in where the step gives NaN: of 0, infinity and NaN.
// (56.5 million values with 8-bit states, clipped: 149 us, 147 were subnormal x to count as 0; with the IEEE root, which is a dozen instructions and
// a branch, 205.)
__device__ __forceinline__ float2 roots(float2 x) {
    float2 y;
    asm("rsqrt.approx.f32 %0, %1;" : "=f"(y.x) : "f"(x.x));
    asm("rsqrt.approx.f32 %0, %1;" : "=f"(y.y) : "f"(x.y));
    const float2 s = mul2(x, y), low = mul2(x, both(0x1p-65f));
    const float2 u = ffma2(ffma2(make_float2(-s.x, -s.y), s, x), mul2(y, both(0.5f)), s);
    return make_float2(fmaxf(u.x, low.x), fmaxf(u.y, low.y));
}

// What a step multiplies with, twice each.
struct Factors {
    float2 b1, b2, k1, k2, clip, rate, widen, eps, decay, one;
    float2 sm, sv;  // scales of the codes
};
// The step of two values: w, m and v are replaced, u is the root of v'.  EIGHT: m comes as a code, v as that of its root.
// Moments are evaluated as the formula stands, each product and sum rounded by itself.  A code that another order moves to its neighbour is up to 7% of
// its value and may decide a later scale: with factors folded into one another and approximate roots, 1 to 3 of 220,795 blocks were 3 to 6% off
// a plain evaluation after eight steps, of either moment.  The sums are fmas with a one that the compiler does not know: of a packed product and a packed
// sum it makes an fma although both name their rounding.  The quotient of p' is fed back nowhere and is approximate.
template <bool EIGHT>
__device__ __forceinline__ void step2(const Factors &f, float2 &w, float2 g, float2 &m, float2 &v, float2 &u) {
    g = mul2(g, f.clip);
    if constexpr (EIGHT) {
        m = mul2(m, f.sm), v = mul2(v, f.sv);
        v = mul2(v, v);
    }
    m = ffma2(mul2(f.b1, m), f.one, mul2(f.k1, g));
    v = ffma2(mul2(f.b2, v), f.one, mul2(f.k2, mul2(g, g)));
    u = roots(v);
    if constexpr (!EIGHT) {  // a v that was given below zero has no root
        if (v.x < 0.f) u.x = __int_as_float(0x7FFFFFFF);
        if (v.y < 0.f) u.y = __int_as_float(0x7FFFFFFF);
    }
    const float2 d = ffma2(u, f.widen, f.eps);
    w = ffma2(mul2(m, make_float2(reciprocal(d.x), reciprocal(d.y))), f.rate, mul2(w, f.decay));
}
__device__ __forceinline__ Factors factors(const StepArgs &p, const Rates &r, float weight_decay) {
    return {both(p.beta1), both(p.beta2), both(p.keep1), both(p.keep2), both(r.clip), both(-r.rate), both(r.widen), both(p.eps), both(fmaf(-r.lr, weight_decay, 1.f)), both(p.one), {}, {}};
}

// The step of eight values, n of them there, and their stores.  WIDE: all there, at whole vectors.
template <bool WIDE, bool EIGHT>
__device__ __forceinline__ void step8(const Raw &x, const Entry &t, const StepArgs &p, const Rates &r, int64_t e, int n) {
    float w[8], g[8], m[8], v[8], u[8];
    numbers(x.g, t.grad_dtype, g);
    numbers(x.w, t.master ? 0 : t.param_dtype, w);
    Factors f = factors(p, r, t.decay);
    if constexpr (EIGHT) {
        f.sm = both(x.sm), f.sv = both(x.sv);
        decode(x.cm, m);
        decode(x.cv, v);
    } else {
        numbers(x.m, 0, m);
        numbers(x.v, 0, v);
    }
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
        float2 w2 = make_float2(w[k], w[k + 1]), m2 = make_float2(m[k], m[k + 1]), v2 = make_float2(v[k], v[k + 1]), u2;
        step2<EIGHT>(f, w2, make_float2(g[k], g[k + 1]), m2, v2, u2);
        w[k] = w2.x, w[k + 1] = w2.y, m[k] = m2.x, m[k + 1] = m2.y, v[k] = v2.x, v[k + 1] = v2.y, u[k] = u2.x, u[k + 1] = u2.y;
    }
    store8<WIDE>(t.param, t.param_dtype, e, n, w);
    if (t.master) store8<WIDE>(t.master, 0, e, n, w);
    if constexpr (EIGHT) {
        const int64_t block = e >> 8;
        float sm, sv;
        const uint2 cm = encode<false>(m, sm), cv = encode<true>(u, sv);
        store_codes<WIDE>(t.m, e, n, cm);
        store_codes<WIDE>(t.v, e, n, cv);
        if ((threadIdx.x & 31) == 0 && n > 0) {
            t.sm[block] = sm;
            t.sv[block] = sv;
        }
    } else {
        store8<WIDE>(t.m, 0, e, n, m);
        store8<WIDE>(t.v, 0, e, n, v);
    }
}

// A whole chunk of a tensor with 8-bit states, and parameters and gradients of one 16-bit type, at whole vectors.  There is
// as much to compute here as to move, so that the next chunk is on its way meanwhile.
struct Half {
    uint4 w, g;
    uint2 m, v;
    float sm, sv;
};
// The chunk to come waits in shared memory, each thread's values in places of its own (so nobody waits for anybody).
constexpr int kAll = kThreads * kGroups;
constexpr int kPlace = kAll * (16 + 16 + 8 + 8 + 4 + 4), kSlot = 2 * kPlace;
template <int N>
__device__ __forceinline__ void copy_async(uint32_t to, const void *from) {
    if constexpr (N == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(N) : "memory");
}
struct Places {  // of this thread in the first place
    uint32_t wg, mv, s;
    __device__ __forceinline__ Places(uint32_t ring) : wg(ring + threadIdx.x * 16), mv(ring + kAll * 32 + threadIdx.x * 8), s(ring + kAll * 48 + threadIdx.x * 4) {}
};
__device__ __forceinline__ void request_half(const Places &p, uint32_t place, const Entry &t, int64_t e) {
    const char *w = static_cast<const char *>(t.param) + e * 2, *g = static_cast<const char *>(t.grad) + e * 2;
    const char *m = static_cast<const char *>(t.m) + e, *v = static_cast<const char *>(t.v) + e;
    const float *sm = t.sm + (e >> 8), *sv = t.sv + (e >> 8);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t to = place + i * kPlace;
        copy_async<16>(p.wg + to, w + i * (kPart * 2));
        copy_async<16>(p.wg + to + kAll * 16, g + i * (kPart * 2));
        copy_async<8>(p.mv + to, m + i * kPart);
        copy_async<8>(p.mv + to + kAll * 8, v + i * kPart);
        copy_async<4>(p.s + to, sm + i * (kPart / 256));
        copy_async<4>(p.s + to + kAll * 4, sv + i * (kPart / 256));
    }
}
__device__ __forceinline__ Half receive_half(const Places &p, uint32_t place) {
    Half x;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.w.x), "=r"(x.w.y), "=r"(x.w.z), "=r"(x.w.w) : "r"(p.wg + place) : "memory");
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.g.x), "=r"(x.g.y), "=r"(x.g.z), "=r"(x.g.w) : "r"(p.wg + place + kAll * 16) : "memory");
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(x.m.x), "=r"(x.m.y) : "r"(p.mv + place) : "memory");
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(x.v.x), "=r"(x.v.y) : "r"(p.mv + place + kAll * 8) : "memory");
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x.sm) : "r"(p.s + place) : "memory");
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x.sv) : "r"(p.s + place + kAll * 4) : "memory");
    return x;
}
template <int DT>
__device__ __forceinline__ void step_half(const Places &places, uint32_t place, const Entry &t, int64_t e, const StepArgs &p, const Rates &r) {
    Factors f = factors(p, r, t.decay);
    char *to = static_cast<char *>(t.param) + e * 2, *tm = static_cast<char *>(t.m) + e, *tv = static_cast<char *>(t.v) + e;
    float *sm = t.sm + (e >> 8), *sv = t.sv + (e >> 8);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const Half x = receive_half(places, place + i * kPlace);
        f.sm = both(x.sm), f.sv = both(x.sv);
        float m[8], u[8], w[8], g[8];
        numbers({x.w, x.w}, DT, w);
        numbers({x.g, x.g}, DT, g);
        decode(x.m, m);
        decode(x.v, u);
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
            float2 w2 = make_float2(w[k], w[k + 1]), m2 = make_float2(m[k], m[k + 1]), v2 = make_float2(u[k], u[k + 1]), u2;
            step2<true>(f, w2, make_float2(g[k], g[k + 1]), m2, v2, u2);
            w[k] = w2.x, w[k + 1] = w2.y, m[k] = m2.x, m[k + 1] = m2.y, u[k] = u2.x, u[k + 1] = u2.y;
        }
        store8<true>(to + i * (kPart * 2), DT, 0, 8, w);
        float s0, s1;
        store_codes<true>(tm, i * kPart, 8, encode<false>(m, s0));
        store_codes<true>(tv, i * kPart, 8, encode<true>(u, s1));
        if ((threadIdx.x & 31) == 0) sm[i * (kPart / 256)] = s0, sv[i * (kPart / 256)] = s1;
    }
}

__global__ void __launch_bounds__(kThreads * kGroups, 1) step_kernel(const __grid_constant__ StepArgs p) {
    __shared__ float factor;
    extern __shared__ __align__(16) char room[];
    pdl_launch_dependents();
    pdl_wait();
    float clip = 1.f;
    if (p.partial) {
        if (threadIdx.x < 32) {
            double sum = 0.0;
            for (int i = threadIdx.x; i < p.parts; i += 32) sum += p.partial[i];
            for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
            if (threadIdx.x == 0) {
                const float norm = static_cast<float>(sqrt(sum));
                if (blockIdx.x == 0 && p.norm) *p.norm = norm;
                const float c = p.max_norm / (norm + p.norm_eps);
                factor = norm < INFINITY ? (c <= 1.f ? c : 1.f) : -1.f;  // 0 / 0: nothing to clip
            }
        }
        __syncthreads();
        clip = factor;
        if (clip < 0.f) return;  // a norm that is infinite or NaN: no step
    }
    Rates r;
    r.clip = clip;
    r.lr = p.lr_dev ? *p.lr_dev : p.lr;
    const float step = p.step_dev ? fmaxf(static_cast<float>(*p.step_dev), 1.f) : p.step;
    r.rate = r.lr / -expm1f(step * p.ln1);
    r.widen = rsqrtf(-expm1f(step * p.ln2));
    const List l(p.list, p.count, room + 2 * kSlot);
    // from the last chunk on: the gradients that the norm's launch read last are still in the L2
    const int first = l.t[0].first, back = static_cast<int>(gridDim.x) * kGroups;
    int c = static_cast<int>(p.more ? p.list[p.count].first_chunk : p.chunks) - 1 - static_cast<int>(blockIdx.x * kGroups + threadIdx.x / kThreads);
    int i = p.count - 1;
    const Places mine(smem_u32(room));
    struct Where {
        int i;      // entry, or -1: no more
        int64_t e;  // this thread's first value
        bool half;
    };
    const auto request = [&](uint32_t place) {
        Where w{-1, 0, false};
        if (c >= first) {
            i = l.find_before(i, c);
            const Entry &t = l.t[i];
            const int64_t begin = static_cast<int64_t>(c - t.first) * kChunk;
            w = {i, begin + threadIdx.x % kThreads * kVals, t.kind >= WIDE_E4M3_F16 && begin + kChunk <= t.numel};
            if (w.half) request_half(mine, place, t, w.e);
            c -= back;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        return w;
    };
    uint32_t place = 0;
    for (Where at = request(0); at.i >= 0; place ^= kSlot) {
        const Where next = request(place ^ kSlot);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        const Entry &t = l.t[at.i];
        if (at.half) {
            if (t.kind == WIDE_E4M3_F16) step_half<1>(mine, place, t, at.e, p, r);
            else step_half<2>(mine, place, t, at.e, p, r);
        } else {
#pragma unroll 1
            for (int64_t e = at.e; e < at.e + kChunk; e += kPart) {
                const int64_t left = t.numel - e;
                const int n = left >= 8 ? 8 : left > 0 ? static_cast<int>(left) : 0;
                if (!__any_sync(~0u, n > 0)) break;
                Raw x;
                const bool wide = t.kind != ANY && __all_sync(~0u, n == 8);
                if (t.state == QG_STATE_E4M3) {
                    if (wide) {
                        fetch8<true, true>(x, t, e, 8);
                        step8<true, true>(x, t, p, r, e, 8);
                    } else {
                        fetch8<false, true>(x, t, e, n);
                        step8<false, true>(x, t, p, r, e, n);
                    }
                } else if (wide) {
                    fetch8<true, false>(x, t, e, 8);
                    step8<true, false>(x, t, p, r, e, 8);
                } else {
                    fetch8<false, false>(x, t, e, n);
                    step8<false, false>(x, t, p, r, e, n);
                }
            }
        }
        at = next;
    }
}

int parts_of(int64_t chunks) {
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((chunks + kGroups - 1) / kGroups, device_info().sm_count)));
}

}  // namespace

int64_t adamw_chunks(int64_t numel) { return (numel + kChunk - 1) / kChunk; }

size_t adamw_workspace_bytes(int64_t chunks) { return sizeof(double) * parts_of(chunks); }

cudaError_t adamw_step(const AdamwStep &q, void *ws, cudaStream_t s) {
    // no values: nothing but, perhaps, the norm of nothing
    if (q.chunks == 0) return q.clip && q.norm ? cudaMemsetAsync(q.norm, 0, sizeof(float), s) : cudaSuccess;
    const qg_adamw_tensor *list = static_cast<const qg_adamw_tensor *>(q.list);
    const int parts = parts_of(q.chunks);
    static std::atomic<unsigned long long> done{0};  // a bit for each device
    const int slot = device_slot();
    if (slot < 0 || !(done.load(std::memory_order_relaxed) >> slot & 1)) {
        cudaError_t e = cudaFuncSetAttribute(step_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * kSlot + list_bytes(kTable));
        if (e == cudaSuccess) e = cudaFuncSetAttribute(sumsq_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, list_bytes(kTable));
        if (e != cudaSuccess) return e;
        if (slot >= 0) done.fetch_or(1ull << slot, std::memory_order_relaxed);
    }
    if (q.clip)
        for (int at = 0; at < q.count; at += kTable) {
            const int n = std::min(kTable, q.count - at);
            const cudaError_t e = launch_pdl(sumsq_kernel, dim3(parts), dim3(kAll), list_bytes(n), s, list + at, n, at + n < q.count ? 1 : 0, q.chunks,
                                             static_cast<double *>(ws), at > 0 ? 1 : 0);
            if (e != cudaSuccess) return e;
        }
    StepArgs a{};
    a.chunks = q.chunks;
    a.lr = static_cast<float>(q.lr);
    a.beta1 = static_cast<float>(q.beta1);
    a.beta2 = static_cast<float>(q.beta2);
    a.keep1 = static_cast<float>(1.0 - q.beta1);
    a.keep2 = static_cast<float>(1.0 - q.beta2);
    a.ln1 = static_cast<float>(std::log(q.beta1));  // -inf for 0: 1 - 0^step is 1
    a.ln2 = static_cast<float>(std::log(q.beta2));
    a.eps = static_cast<float>(q.eps);
    a.one = 1.f;
    a.lr_dev = q.lr_dev;
    a.step = static_cast<float>(q.step);
    a.step_dev = q.step_dev;
    a.partial = q.clip ? static_cast<const double *>(ws) : nullptr;
    a.parts = parts;
    a.max_norm = q.max_norm;
    a.norm_eps = q.norm_eps;
    a.norm = q.norm;
    for (int at = 0; at < q.count; at += kTable) {
        a.list = list + at;
        a.count = std::min(kTable, q.count - at);
        a.more = at + a.count < q.count ? 1 : 0;
        const cudaError_t e = launch_pdl(step_kernel, dim3(parts), dim3(kAll), 2 * kSlot + list_bytes(a.count), s, a);
        if (e != cudaSuccess) return e;
    }
    return cudaGetLastError();
}

}  // namespace qg
