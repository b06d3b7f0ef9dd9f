// qg_logprobs.cu -- log probabilities of given tokens from logits, with the entropy of every row and its k most
// probable alternatives, and the gradient of the logits.
//
//   z = x * inv_temperature,  M = max z,  S = sum exp(z - M),  A = sum exp(z - M) (z - M)
//   lse = M + log S,  logprob = z[target] - lse,  entropy = log S - A / S
//   dx[v] = inv_temperature * ( d ([v = target] - p_v) - h p_v (log p_v + entropy) ),  p_v = exp(z_v - lse)
//
// Both are bound by memory.  Forward: one pass over the logits; a thread keeps a running reference (the largest value
// it has met), S and A, and rescales them when the reference grows.  A row is the work of one CTA or, where there are
// few rows, of a cluster whose CTAs join their sums through distributed shared memory.
// Measured, vocabulary 100352: 4096 rows of bf16 151 us (5.4 TB/s), their gradient with entropies 278 us (5.9 TB/s); a few
// rows by latency: 64 of bf16 with 5 alternatives 14 us, one of fp32 with 20 alternatives 9.5 us.
//
// Alternatives in the same pass: the k-th largest of the threads' first maxima is a value that at least k logits
// reach, so only what reaches it can be among the k largest.  What does goes to a small list in shared memory (about
// k for each further stretch of the row that is as long as the first), as keys (value, then lower index) that are
// all different; a list that gets full is cut to its k largest, which raises the bound.
#include <cooperative_groups.h>

#include <algorithm>

#include "qg_device.cuh"
#include "qg_internal.h"

namespace qg {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kVecs = 4;       // 16-byte vectors of a thread and step
constexpr int kList = 2048;    // candidates that the list holds
constexpr int kMaxTop = 64;
constexpr uint32_t kOrdNegInf = 0x007FFFFFu;  // ordered(-inf)

// Unsigned integers in the order of the values: -inf < ... < -0 = +0 < ... < inf < NaN.
__device__ __forceinline__ uint32_t ordered(float x) {
    if (x != x) return 0xFFFFFFFFu;
    const uint32_t b = __float_as_uint(x + 0.f);  // one zero
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) {
    if (k == 0xFFFFFFFFu) return __int_as_float(0x7FFFFFFF);
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Packed fp32 pairs.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n .reg .b64 ra, rb, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %5};\n add.rn.f32x2 rd, ra, rb;\n mov.b64 {%0, %1}, rd;\n}\n"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n .reg .b64 ra, rb, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %5};\n mul.rn.f32x2 rd, ra, rb;\n mov.b64 {%0, %1}, rd;\n}\n"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// Words of logits as they lie in memory: largest() keeps a NaN, at_least() does not.
template <int XT>
struct Logits;  // f32, f16, bf16
template <>
struct Logits<0> {
    static constexpr int VE = 4, ES = 4;
    static constexpr uint32_t NEG_INF = 0xFF800000u;  // a word of them
    static __device__ __forceinline__ void floats(const uint4 &v, float (&x)[4]) {
        x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
    static __device__ __forceinline__ float one(const char *p) { return *reinterpret_cast<const float *>(p); }
    static __device__ __forceinline__ uint32_t largest(uint32_t a, uint32_t b) { return __float_as_uint(max_nan(__uint_as_float(a), __uint_as_float(b))); }
    static __device__ __forceinline__ uint32_t at_least(uint32_t a, uint32_t b) { return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b))); }
    static __device__ __forceinline__ float value(uint32_t w) { return __uint_as_float(w); }
    static __device__ __forceinline__ uint32_t word(float x) { return __float_as_uint(x); }
};
template <>
struct Logits<1> {
    static constexpr int VE = 8, ES = 2;
    static constexpr uint32_t NEG_INF = 0xFC00FC00u;
    static __device__ __forceinline__ void floats(const uint4 &v, float (&x)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ float one(const char *p) { return h2f(*reinterpret_cast<const uint16_t *>(p)); }
    static __device__ __forceinline__ uint32_t largest(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    static __device__ __forceinline__ uint32_t at_least(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    static __device__ __forceinline__ float value(uint32_t w) { return max_nan(h2f(static_cast<uint16_t>(w)), h2f(static_cast<uint16_t>(w >> 16))); }
    static __device__ __forceinline__ uint32_t word(float x) { return f2h(x) * 0x10001u; }
};
template <>
struct Logits<2> {
    static constexpr int VE = 8, ES = 2;
    static constexpr uint32_t NEG_INF = 0xFF80FF80u;
    static __device__ __forceinline__ void floats(const uint4 &v, float (&x)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ float one(const char *p) { return bf2f(*reinterpret_cast<const uint16_t *>(p)); }
    static __device__ __forceinline__ uint32_t largest(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    static __device__ __forceinline__ uint32_t at_least(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    static __device__ __forceinline__ float value(uint32_t w) { return max_nan(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }
    static __device__ __forceinline__ uint32_t word(float x) { return f2bf(x) * 0x10001u; }
};

__device__ __forceinline__ uint4 load_stream(const char *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// A row as 16-byte vectors at 16-byte boundaries: vector q holds the values q * VE - pad and on.
template <int XT>
struct Row {
    const char *at;
    int pad, V, vecs;
    __device__ __forceinline__ Row(const void *X, int64_t first, int V_) : V(V_) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(X) + static_cast<uint64_t>(first) * Logits<XT>::ES;
        pad = static_cast<int>(a & 15u) / Logits<XT>::ES;
        at = reinterpret_cast<const char *>(a & ~static_cast<uintptr_t>(15));
        vecs = (pad + V + Logits<XT>::VE - 1) / Logits<XT>::VE;
    }
    // -inf outside the row
    __device__ __forceinline__ uint4 load(int q) const {
        constexpr int VE = Logits<XT>::VE;
        const int e = q * VE - pad;
        if (e >= 0 && e + VE <= V) return load_stream(at + static_cast<int64_t>(q) * 16);
        uint32_t w[4] = {Logits<XT>::NEG_INF, Logits<XT>::NEG_INF, Logits<XT>::NEG_INF, Logits<XT>::NEG_INF};
#pragma unroll
        for (int k = 0; k < VE; ++k)
            if (e + k >= 0 && e + k < V) {
                const char *p = at + static_cast<int64_t>(q) * 16 + k * Logits<XT>::ES;
                if constexpr (XT == 0) w[k] = *reinterpret_cast<const uint32_t *>(p);
                else w[k >> 1] = (w[k >> 1] & (0xFFFFu << (16 * (1 - (k & 1))))) | static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(p)) << (16 * (k & 1));
            }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// Sums over exp2((x - ref) * c); ref = -inf: nothing yet.
struct Sums {
    float ref, s, a;
};
__device__ __forceinline__ void move_reference(Sums &t, float to, float c) {
    if (t.ref < to && t.ref > -INFINITY) {
        const float d = fmaxf((t.ref - to) * c, -150.f), f = ex2(d);
        t.a = f * fmaf(d, t.s, t.a);
        t.s *= f;
    }
    t.ref = fmaxf(t.ref, to);
}
__device__ __forceinline__ Sums joined(Sums t, Sums o, float c) {
    const float m = fmaxf(t.ref, o.ref);
    move_reference(t, m, c);
    move_reference(o, m, c);
    return {m, t.s + o.s, t.a + o.a};
}

// Of the lanes' sums, to all of them (adding is commutative, bit for bit).
template <int LANES>
__device__ __forceinline__ Sums joined_lanes(Sums w, float c) {
#pragma unroll
    for (int o = LANES / 2; o >= 1; o >>= 1) {
        const Sums other{__shfl_xor_sync(~0u, w.ref, o), __shfl_xor_sync(~0u, w.s, o), __shfl_xor_sync(~0u, w.a, o)};
        w = joined(w, other, c);
    }
    return w;
}

struct ScoreArgs {
    const void *X;
    int64_t ldx;
    const int64_t *target;
    int T, V, top;
    float inv_t, c;      // c = inv_t * log2(e)
    float reach, least;  // 130 / c; the least reference that a value of the type lies so far below (infinity: none)
    float *logprob, *entropy, *lse;
    int64_t *top_ids;
    float *top_logprobs;
    int *status;
};

// The n keys' k-th largest (n >= k >= 1; all threads get it): bit by bit from the top.
template <typename K, int PER>
__device__ K kth_largest(const K (&mine)[PER], int k, int low_bit) {
    K at = 0;
    for (int b = static_cast<int>(sizeof(K)) * 8 - 1; b >= low_bit; --b) {
        const K next = at | (static_cast<K>(1) << b);
        int n = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) n += __syncthreads_count(mine[i] >= next);
        if (n >= k) at = next;
    }
    return at;
}

struct Shared {
    unsigned long long list[kList];
    unsigned long long best[kMaxTop];
    Sums part[kThreads / 32];
    Sums sum;
    int bad, count, found;
};

// Cuts the list's first n keys (n <= kList) to the k largest; returns how many are left.
__device__ int cut_list(Shared &sh, int n, int k, unsigned long long &bound) {
    if (n <= k) return n;
    unsigned long long mine[kList / kThreads];
#pragma unroll
    for (int i = 0; i < kList / kThreads; ++i) {
        const int at = i * kThreads + threadIdx.x;
        mine[i] = at < n ? sh.list[at] : 0ull;
    }
    bound = kth_largest(mine, k, 0);
    if (threadIdx.x == 0) sh.count = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kList / kThreads; ++i)
        if (mine[i] >= bound) sh.list[atomicAdd(&sh.count, 1)] = mine[i];  // their order does not matter: the last step ranks them
    __syncthreads();
    return k;
}

// Writes the min(n, k) largest of n keys, in order, to out.
__device__ __forceinline__ void rank_keys(const unsigned long long *keys, int n, int k, unsigned long long *out) {
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const unsigned long long mine = keys[i];
        int above = 0;
        for (int j = 0; j < n; ++j) above += keys[j] > mine;
        if (above < k) out[above] = mine;
    }
}

template <int XT, bool TOP>
__global__ void __launch_bounds__(kThreads, 2) score_kernel(const __grid_constant__ ScoreArgs p) {
    using L = Logits<XT>;
    constexpr int VE = L::VE;
    __shared__ Shared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int parts = static_cast<int>(cluster.num_blocks()), part = static_cast<int>(cluster.block_rank());
    const int64_t row = blockIdx.x / parts;
    const int tid = threadIdx.x;
    pdl_launch_dependents();
    pdl_wait();
    const Row<XT> r(p.X, row * p.ldx, p.V);
    const int v0 = static_cast<int>(static_cast<int64_t>(r.vecs) * part / parts), v1 = static_cast<int>(static_cast<int64_t>(r.vecs) * (part + 1) / parts);
    Sums t{-INFINITY, 0.f, 0.f};
    bool bad = false;
    int kept = 0;                                                               // keys in the list
    unsigned long long bound = static_cast<unsigned long long>(kOrdNegInf + 1) << 32;  // what a key has to reach
    if (tid == 0) sh.count = 0, sh.found = 0;
    // the given token's logit, long before it is wanted
    int64_t target = -1;
    float given = 0.f;
    if (part == 0 && tid == 0 && p.target) {
        target = p.target[row];
        if (target >= 0 && target < p.V) given = L::one(static_cast<const char *>(p.X) + (row * p.ldx + target) * L::ES);
    }

    uint4 ahead[kVecs];
    const auto fetch = [&](int q0) {
#pragma unroll
        for (int u = 0; u < kVecs; ++u) {
            const int q = q0 + u * kThreads + tid;
            ahead[u] = q < v1 ? r.load(q) : make_uint4(L::NEG_INF, L::NEG_INF, L::NEG_INF, L::NEG_INF);
        }
    };
    fetch(v0);
    for (int q0 = v0; q0 < v1; q0 += kThreads * kVecs) {
        uint4 v[kVecs];
#pragma unroll
        for (int u = 0; u < kVecs; ++u) v[u] = ahead[u];
        if (q0 + kThreads * kVecs < v1) fetch(q0 + kThreads * kVecs);
        uint32_t best = L::NEG_INF;
#pragma unroll
        for (int u = 0; u < kVecs; ++u) best = L::largest(L::largest(best, v[u].x), L::largest(v[u].y, L::largest(v[u].z, v[u].w)));
        const float top = L::value(best);
        if (!(top < INFINITY)) bad = true;  // NaN, or an infinity whose differences are NaN
        if (top > -INFINITY) {
            move_reference(t, top, p.c);
            if (fabsf(t.ref) <= 16384.f && t.ref >= p.least) {
                // What is 2^-130 of the reference or less counts as about that, -inf too: its product with its logarithm is a
                // number.  |ref| / 64 is more than the type's step there.  Where the type has no such value (fp16 at temperatures
                // above some 700), -inf would count as its lowest one: those logits are taken one by one below.
                const uint32_t low = L::word(t.ref - fmaxf(p.reach, fabsf(t.ref) * 0.015625f));
                const float2 ref = make_float2(-t.ref, -t.ref), c = make_float2(p.c, p.c);
                float2 s0 = make_float2(0.f, 0.f), a0 = s0;
#pragma unroll
                for (int u = 0; u < kVecs; ++u) {
                    float x[VE];
                    L::floats(make_uint4(L::at_least(v[u].x, low), L::at_least(v[u].y, low), L::at_least(v[u].z, low), L::at_least(v[u].w, low)), x);
#pragma unroll
                    for (int k = 0; k < VE; k += 2) {
                        const float2 y = mul2(add2(make_float2(x[k], x[k + 1]), ref), c);
                        const float2 e = make_float2(ex2(y.x), ex2(y.y));
                        s0 = add2(s0, e);
                        a0 = ffma2(e, y, a0);
                    }
                }
                t.s += s0.x + s0.y;
                t.a += a0.x + a0.y;
            } else {
#pragma unroll 1
                for (int u = 0; u < kVecs; ++u) {
                    const uint4 w = u == 0 ? v[0] : u == 1 ? v[1] : u == 2 ? v[2] : v[3];
                    float x[VE];
                    L::floats(w, x);
#pragma unroll
                    for (int k = 0; k < VE; ++k) {
                        const float y = fmaxf((x[k] - t.ref) * p.c, -150.f), e = ex2(y);
                        t.s += e;
                        t.a = fmaf(e, y, t.a);
                    }
                }
            }
        }
        if constexpr (TOP) {
            const uint32_t most = ordered(top);
            if (q0 == v0) {  // the first step: a bound from the threads' maxima (its upper 16 bits will do)
                const uint32_t one[1] = {most};
                const uint32_t b = kth_largest(one, p.top, 16);
                if (b > kOrdNegInf) bound = static_cast<unsigned long long>(b) << 32;
            }
            for (;;) {
                if (most >= static_cast<uint32_t>(bound >> 32)) {
#pragma unroll
                    for (int u = 0; u < kVecs; ++u) {
                        float x[VE];
                        L::floats(v[u], x);
                        const int e = (q0 + u * kThreads + tid) * VE - r.pad;
#pragma unroll
                        for (int k = 0; k < VE; ++k) {
                            const unsigned long long key = static_cast<unsigned long long>(ordered(x[k])) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(e + k));
                            if (key >= bound) {
                                const int at = atomicAdd(&sh.count, 1);
                                if (at < kList) sh.list[at] = key;
                            }
                        }
                    }
                }
                __syncthreads();
                const int n = sh.count;
                __syncthreads();
                if (n <= kList) {
                    kept = n;
                    break;
                }
                // too many: the bound rises to the k-th largest of those in the list, and this step's are looked at again
                unsigned long long mine[kList / kThreads];
#pragma unroll
                for (int i = 0; i < kList / kThreads; ++i) mine[i] = sh.list[i * kThreads + tid];
                bound = kth_largest(mine, p.top, 0);
                if (tid == 0) sh.count = kept;
                __syncthreads();
            }
            if (kept > kList / 2) kept = cut_list(sh, kept, p.top, bound);
        }
    }

    // the CTA's sums
    bad = __syncthreads_or(bad);
    {
        const Sums w = joined_lanes<32>(t, p.c);
        if ((tid & 31) == 0) sh.part[tid >> 5] = w;
        __syncthreads();
        if (tid < 32) {
            const Sums all = joined_lanes<16>(sh.part[tid & 15], p.c);
            if (tid == 0) sh.sum = all, sh.bad = bad;
        }
    }
    if constexpr (TOP) {
        if (kept > kThreads) kept = cut_list(sh, kept, p.top, bound);
        rank_keys(sh.list, kept, p.top, sh.best);
        if (tid == 0) sh.found = min(kept, p.top);
    }
    if (parts > 1) cluster.sync();
    else __syncthreads();
    if (part == 0) {
        Sums all = sh.sum;
        bool any_bad = sh.bad;
        if (parts > 1) {  // a lane for each CTA
            const int i = tid & 7;
            all = {-INFINITY, 0.f, 0.f};
            if (i < parts) all = *cluster.map_shared_rank(&sh.sum, i), any_bad = *cluster.map_shared_rank(&sh.bad, i) != 0;
            all = joined_lanes<8>(all, p.c);
            any_bad = __any_sync(~0u, any_bad);
        }
        if (any_bad) all.s = all.ref = __int_as_float(0x7FFFFFFF);
        // a row without a finite value: lse -inf, entropy 0
        const bool none = all.ref == -INFINITY;
        const float log_s = none ? 0.f : logf(all.s), lse = fmaf(all.ref, p.inv_t, log_s);
        const auto logprob = [&](float x) { return none ? -INFINITY : (x - all.ref) * p.inv_t - log_s; };
        if (tid == 0) {
            float lp = 0.f;
            if (target >= p.V) {
                if (p.status) *p.status = 1;
            } else if (target >= 0) {
                lp = logprob(given);
            }
            if (p.logprob) p.logprob[row] = lp;
            if (p.entropy) p.entropy[row] = none ? 0.f : log_s - 0.69314718056f * (all.a / all.s);
            if (p.lse) p.lse[row] = lse;
        }
        if constexpr (TOP) {
            int found = sh.found;
            const unsigned long long *keys = sh.best;
            if (parts > 1) {  // every CTA's best, one after another
                const int lane = tid & 31, m = lane < parts ? *cluster.map_shared_rank(&sh.found, lane) : 0;
                int behind = m;  // the keys of this CTA and those before it
                for (int o = 1; o < 8; o <<= 1) {
                    const int v = __shfl_up_sync(~0u, behind, o);
                    if (lane >= o) behind += v;
                }
                const int n = __shfl_sync(~0u, behind, 7);
                for (int i = tid >> 5; i < parts; i += kThreads / 32) {  // a warp for each CTA
                    const int first = __shfl_sync(~0u, behind - m, i), mine = __shfl_sync(~0u, m, i);
                    const unsigned long long *from = cluster.map_shared_rank(sh.best, i);
                    for (int k = lane; k < mine; k += 32) sh.list[first + k] = from[k];
                }
                __syncthreads();  // sh.best is this CTA's own copy from here on: nobody else reads it
                rank_keys(sh.list, n, p.top, sh.best);
                __syncthreads();
                found = min(n, p.top);
            }
            if (tid < found) {
                const unsigned long long key = keys[tid];
                const float x = unordered(static_cast<uint32_t>(key >> 32));
                p.top_ids[row * p.top + tid] = 0xFFFFFFFFu - static_cast<uint32_t>(key);
                p.top_logprobs[row * p.top + tid] = logprob(x);
            }
            if (found < p.top && tid < 32) {  // fewer than k above -inf: the first of those at -inf follow
                int n = found;
                for (int e = 0; n < p.top && e < p.V; e += 32) {
                    const bool is = e + tid < p.V && L::one(static_cast<const char *>(p.X) + (row * p.ldx + e + tid) * L::ES) == -INFINITY;
                    const unsigned who = __ballot_sync(~0u, is);
                    const int at = n + __popc(who & ((1u << tid) - 1u));
                    if (is && at < p.top) {
                        p.top_ids[row * p.top + at] = e + tid;
                        p.top_logprobs[row * p.top + at] = any_bad ? __int_as_float(0x7FFFFFFF) : -INFINITY;
                    }
                    n += __popc(who);
                }
            }
        }
    }
    if (parts > 1) cluster.sync();  // the others' shared memory is read until here
}

// ---------------------------------------------------------------------------------------------------- gradient
struct LossArgs {
    const void *X;
    int64_t ldx;
    const int64_t *target;
    const float *lse, *entropy, *d_logprob, *d_entropy;
    void *dX;
    int64_t lddx;
    int V;
    float inv_t;
    unsigned segments;
};

constexpr int kLossThreads = 256;
constexpr int kLossVecs = 4;

template <int XT, bool ENT>
__global__ void __launch_bounds__(kLossThreads) loss_kernel(const __grid_constant__ LossArgs p) {
    using L = Logits<XT>;
    constexpr int VE = L::VE;
    pdl_launch_dependents();
    pdl_wait();
    const int64_t row = blockIdx.x / p.segments;
    const int q0 = static_cast<int>(blockIdx.x % p.segments) * (kLossThreads * kLossVecs) + threadIdx.x;
    const Row<XT> r(p.X, row * p.ldx, p.V);
    char *out = static_cast<char *>(p.dX) + row * p.lddx * L::ES - r.pad * L::ES;
    const bool wide = (reinterpret_cast<uintptr_t>(out) & 15u) == 0;
    const int64_t target = p.target ? p.target[row] : -1;
    const bool given = target >= 0 && target < p.V;
    const float d = given ? p.d_logprob[row] : 0.f, h = ENT ? p.d_entropy[row] : 0.f, lse = p.lse[row];
    // a row that no gradient enters, or without a finite logit: zeros
    const bool zero = (d == 0.f && h == 0.f) || lse == -INFINITY;
    const float H = ENT ? p.entropy[row] : 0.f;
    uint4 v[kLossVecs];
    if (!zero) {
#pragma unroll
        for (int u = 0; u < kLossVecs; ++u)
            if (q0 + u * kLossThreads < r.vecs) v[u] = r.load(q0 + u * kLossThreads);
    }
#pragma unroll
    for (int u = 0; u < kLossVecs; ++u) {
        const int q = q0 + u * kLossThreads, e = q * VE - r.pad;
        if (q >= r.vecs) break;
        float x[VE];
        if (zero) {
#pragma unroll
            for (int k = 0; k < VE; ++k) x[k] = 0.f;
        } else {
            L::floats(v[u], x);
#pragma unroll
            for (int k = 0; k < VE; ++k) {
                float lp = fmaf(x[k], p.inv_t, -lse);
                const float pr = ex2(lp * 1.44269504089f);
                float f = d;
                if constexpr (ENT) f = fmaf(h, (lp < -1e4f ? 0.f : lp) + H, d);  // p is 0 where its logarithm is -inf
                x[k] = -pr * f;
                if (given && e + k == static_cast<int>(target)) x[k] += d;
                x[k] *= p.inv_t;
            }
        }
        const uint4 w = L::pack(x);
        char *o = out + static_cast<int64_t>(q) * 16;
        if (wide && e >= 0 && e + VE <= p.V) {
            *reinterpret_cast<uint4 *>(o) = w;
        } else {
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < VE; ++k)
                if (e + k >= 0 && e + k < p.V) {
                    if constexpr (XT == 0) reinterpret_cast<uint32_t *>(o)[k] = ww[k];
                    else reinterpret_cast<uint16_t *>(o)[k] = static_cast<uint16_t>(ww[k >> 1] >> (16 * (k & 1)));
                }
        }
    }
}

template <int XT, bool TOP>
cudaError_t launch_score(const ScoreArgs &a, int want, cudaStream_t s) {
    static ClusterFit fit;
    const auto kern = score_kernel<XT, TOP>;
    const int parts = fitting_cluster(reinterpret_cast<const void *>(kern), fit, want, kThreads, 0);
    return launch_cluster(kern, dim3(static_cast<unsigned>(a.T) * parts), dim3(kThreads), 0, s, parts, a);
}

}  // namespace

cudaError_t token_logprobs(const TokenLogprobs &q, cudaStream_t s) {
    const double c = q.inv_t * 1.4426950408889634;
    const bool fits = c >= 1e-36 && c <= (q.x_dtype == 1 ? 1e9 : 1e36);  // 130 / c and c * 256 are finite, and 130 / c is above the type's least step
    const float reach = fits ? static_cast<float>(130.0 / c) : 0.f, least = fits ? reach - (q.x_dtype == 1 ? 65504.f : 3e38f) : INFINITY;
    const ScoreArgs a{q.X, q.ldx, q.target, q.T, q.V, q.top, q.inv_t, static_cast<float>(c), reach, least, q.logprob, q.entropy, q.lse, q.top_ids, q.top_logprobs, q.status};
    // CTAs of a row: as many as are on the SMs at a time, two on each, as long as each has a step of its own to do (64 rows of
    // 100352 bf16 with 5 alternatives: 4 CTAs each 14 us, 8 take two turns, 24; one row of 100352 fp32: 16 CTAs are 0.3 us
    // slower than 8, their join costs more)
    const int steps = static_cast<int>((static_cast<int64_t>(q.V) * (q.x_dtype == 0 ? 4 : 2) + kThreads * kVecs * 16 - 1) / (kThreads * kVecs * 16));
    int parts = 1;
    while (parts < 8 && parts < steps && static_cast<int64_t>(q.T) * parts <= device_info().sm_count) parts *= 2;
    cudaError_t e;
    if (q.x_dtype == 0) e = q.top ? launch_score<0, true>(a, parts, s) : launch_score<0, false>(a, parts, s);
    else if (q.x_dtype == 1) e = q.top ? launch_score<1, true>(a, parts, s) : launch_score<1, false>(a, parts, s);
    else e = q.top ? launch_score<2, true>(a, parts, s) : launch_score<2, false>(a, parts, s);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t token_logprobs_grad(const TokenLogprobsGrad &q, cudaStream_t s) {
    const int ve = q.x_dtype == 0 ? 4 : 8;
    const int vecs = (q.V + ve - 1) / ve + 1;  // a row may begin inside a vector
    const unsigned segments = static_cast<unsigned>((vecs + kLossThreads * kLossVecs - 1) / (kLossThreads * kLossVecs));
    const LossArgs a{q.X, q.ldx, q.target, q.lse, q.entropy, q.d_logprob, q.d_entropy, q.dX, q.lddx, q.V, q.inv_t, segments};
    if (static_cast<uint64_t>(segments) * q.T > 0x7FFFFFFFull) return cudaErrorNotSupported;
    const dim3 grid(segments * static_cast<unsigned>(q.T)), block(kLossThreads);
    cudaError_t e;
    if (q.x_dtype == 0) e = q.d_entropy ? launch_pdl(loss_kernel<0, true>, grid, block, 0, s, a) : launch_pdl(loss_kernel<0, false>, grid, block, 0, s, a);
    else if (q.x_dtype == 1) e = q.d_entropy ? launch_pdl(loss_kernel<1, true>, grid, block, 0, s, a) : launch_pdl(loss_kernel<1, false>, grid, block, 0, s, a);
    else e = q.d_entropy ? launch_pdl(loss_kernel<2, true>, grid, block, 0, s, a) : launch_pdl(loss_kernel<2, false>, grid, block, 0, s, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace qg
