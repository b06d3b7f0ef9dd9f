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
// Bound by memory.  The list is cut into chunks of 2048 values; a thread owns 8 neighbouring ones and a warp one
// block of 256, so that a block's largest magnitude is a warp reduction.  With clipping a first launch reads the
// gradients alone and leaves one sum of squares for each CTA; the second walks every CTA's run of chunks backwards,
// where the L2 still holds the gradients that were read last.
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>

#include "../../include/qgemm.h"
#include "qg_device.cuh"
#include "qg_internal.h"

namespace qg {
namespace {

constexpr int kThreads = 256;
constexpr int kCtas = 4;                   // of an SM
constexpr int kVals = 8;                   // of a thread
constexpr int kChunk = kThreads * kVals;   // values
constexpr float kCodeMax = 448.f, kCodeMin = 0.001953125f;  // e4m3: the largest value, the smallest above zero
constexpr float kTinyBlock = 1e-30f;       // a block with no larger magnitude is stored as zeros (448 / it stays finite)

// The tensor owning chunk c: the last one with first_chunk <= c (the block counts them).
__device__ int find_tensor(const qg_adamw_tensor *list, int count, int64_t c) {
    int n = 0;
    for (int i = 0; i < count; i += kThreads)
        n += __syncthreads_count(i + static_cast<int>(threadIdx.x) < count && list[i + threadIdx.x].first_chunk <= c);
    return n - 1;
}

// Eight values at element e of an array (n: those that exist), zero where there are none.
__device__ __forceinline__ void load8(const void *base, int dtype, int64_t e, int n, float (&x)[8]) {
    if (dtype == 0) {
        const float *p = static_cast<const float *>(base) + e;
        if (n == 8 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
            const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
            x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = k < n ? p[k] : 0.f;
        }
        return;
    }
    const uint16_t *p = static_cast<const uint16_t *>(base) + e;
    uint32_t w[4] = {0, 0, 0, 0};
    if (n == 8 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < n) w[k >> 1] |= static_cast<uint32_t>(p[k]) << (16 * (k & 1));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (dtype == 1) x[2 * i] = h2f(static_cast<uint16_t>(w[i] & 0xFFFFu)), x[2 * i + 1] = h2f(static_cast<uint16_t>(w[i] >> 16));
        else x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ void store8(void *base, int dtype, int64_t e, int n, const float (&x)[8]) {
    if (dtype == 0) {
        float *p = static_cast<float *>(base) + e;
        if (n == 8 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
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
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = dtype == 1 ? f2h(x[2 * i]) | static_cast<uint32_t>(f2h(x[2 * i + 1])) << 16 : f2bf(x[2 * i]) | static_cast<uint32_t>(f2bf(x[2 * i + 1])) << 16;
    if (n == 8 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < n) p[k] = static_cast<uint16_t>(w[k >> 1] >> (16 * (k & 1)));
    }
}

// Eight e4m3 codes.
__device__ __forceinline__ uint2 load_codes(const void *base, int64_t e, int n) {
    const uint8_t *p = static_cast<const uint8_t *>(base) + e;
    if (n == 8 && (reinterpret_cast<uintptr_t>(p) & 7u) == 0) return *reinterpret_cast<const uint2 *>(p);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (k < n) w[k >> 2] |= static_cast<uint32_t>(p[k]) << (8 * (k & 3));
    return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store_codes(void *base, int64_t e, int n, uint2 c) {
    uint8_t *p = static_cast<uint8_t *>(base) + e;
    if (n == 8 && (reinterpret_cast<uintptr_t>(p) & 7u) == 0) {
        *reinterpret_cast<uint2 *>(p) = c;
        return;
    }
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (k < n) p[k] = static_cast<uint8_t>(w[k >> 2] >> (8 * (k & 3)));
}
__device__ __forceinline__ void decode(uint2 c, float scale, float (&x)[8]) {
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
        x[2 * i] = h2f(h.x) * scale, x[2 * i + 1] = h2f(h.y) * scale;
    }
}
// Codes of x / scale for the warp's block of 256 values; scale is what goes with them.
template <bool KEEP>
__device__ __forceinline__ uint2 encode(const float (&x)[8], float &scale) {
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(x[k]));
    for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    // infinities and NaN: the codes of the others are zeros, and the state shows it (0 * inf is NaN)
    const float inv = top >= kTinyBlock ? kCodeMax / top : 0.f;
    scale = top >= kTinyBlock ? top / kCodeMax : 0.f;
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a = x[2 * i] * inv, b = x[2 * i + 1] * inv;
        if constexpr (KEEP) {
            a = a > 0.f ? fmaxf(a, kCodeMin) : a;
            b = b > 0.f ? fmaxf(b, kCodeMin) : b;
        }
        w[i >> 1] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3)) << (16 * (i & 1));
    }
    return make_uint2(w[0], w[1]);
}

// One sum of squares for each CTA.
__global__ void __launch_bounds__(kThreads, kCtas) sumsq_kernel(const qg_adamw_tensor *__restrict__ list, int count, int64_t chunks,
                                                               double *__restrict__ partial) {
    __shared__ double red[kThreads / 32];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t c0 = chunks * blockIdx.x / gridDim.x, c1 = chunks * (blockIdx.x + 1) / gridDim.x;
    double total = 0.0;
    if (c0 < c1) {
        int at = find_tensor(list, count, c0);
        int64_t next = at + 1 < count ? list[at + 1].first_chunk : chunks;
        for (int64_t c = c0; c < c1; ++c) {
            if (c >= next) {
                while (at + 1 < count && list[at + 1].first_chunk <= c) ++at;
                next = at + 1 < count ? list[at + 1].first_chunk : chunks;
            }
            const qg_adamw_tensor &t = list[at];
            const int64_t e = (c - t.first_chunk) * kChunk + threadIdx.x * kVals;
            const int64_t left = t.numel - e;
            float g[8];
            if (left > 0) load8(t.grad, t.grad_dtype, e, left < 8 ? static_cast<int>(left) : 8, g);
            if (left <= 0) continue;
            float s[2] = {0.f, 0.f};
            bool any = false;
#pragma unroll
            for (int k = 0; k < 8; ++k) s[k & 1] = fmaf(g[k], g[k], s[k & 1]), any |= g[k] != 0.f;
            const float sum = s[0] + s[1];
            if (sum >= 1e-30f && sum <= 3e38f) {
                total += sum;
            } else if (any) {  // squares that leave fp32's range
#pragma unroll
                for (int k = 0; k < 8; ++k) total += static_cast<double>(g[k]) * g[k];
            }
        }
    }
    for (int o = 16; o >= 1; o >>= 1) total += __shfl_xor_sync(~0u, total, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = total;
    __syncthreads();
    if (threadIdx.x == 0) {
        total = 0.0;
        for (int w = 0; w < kThreads / 32; ++w) total += red[w];
        partial[blockIdx.x] = total;
    }
}

struct StepArgs {
    const qg_adamw_tensor *list;
    int count;
    int64_t chunks;
    float lr, beta1, beta2, keep1, keep2, ln1, ln2, eps;  // keep = 1 - beta, ln = log(beta)
    const float *lr_dev;
    float step;
    const int64_t *step_dev;
    const double *partial;  // null: no clipping
    int parts;
    float max_norm, norm_eps;
    float *norm;
};

__global__ void __launch_bounds__(kThreads, kCtas) step_kernel(const __grid_constant__ StepArgs p) {
    __shared__ float factor;
    const int64_t c0 = p.chunks * blockIdx.x / gridDim.x, c1 = p.chunks * (blockIdx.x + 1) / gridDim.x;
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
                factor = norm < INFINITY ? (c > 1.f ? 1.f : c) : -1.f;
            }
        }
        __syncthreads();
        clip = factor;
        if (clip < 0.f) return;  // a norm that is infinite or NaN: no step
    }
    if (c0 >= c1) return;
    const float lr = p.lr_dev ? *p.lr_dev : p.lr, step = p.step_dev ? fmaxf(static_cast<float>(*p.step_dev), 1.f) : p.step;
    const float rate = lr / -expm1f(step * p.ln1);                  // lr / (1 - b1^step)
    const float widen = rsqrtf(-expm1f(step * p.ln2));              // 1 / sqrt(1 - b2^step)
    int at = find_tensor(p.list, p.count, c1 - 1);
    qg_adamw_tensor t = p.list[at];
    for (int64_t c = c1 - 1; c >= c0; --c) {
        if (c < t.first_chunk) {
            do --at;
            while (p.list[at].first_chunk > c || p.list[at].numel == 0);  // an empty tensor owns no chunk
            t = p.list[at];
        }
        const int64_t e = (c - t.first_chunk) * kChunk + threadIdx.x * kVals;
        const int64_t left = t.numel - e;
        const int n = left >= 8 ? 8 : left > 0 ? static_cast<int>(left) : 0;
        float w[8], g[8], m[8], v[8];
        const bool eight = t.state == QG_STATE_E4M3;
        const int64_t block = e >> 8;
        load8(t.grad, t.grad_dtype, e, n, g);
        if (t.master) load8(t.master, 0, e, n, w);
        else load8(t.param, t.param_dtype, e, n, w);
        if (eight) {
            const bool there = (block << 8) < t.numel;
            decode(load_codes(t.exp_avg, e, n), there ? t.exp_avg_scale[block] : 0.f, m);
            decode(load_codes(t.exp_avg_sq, e, n), there ? t.exp_avg_sq_scale[block] : 0.f, v);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] *= v[k];
        } else {
            load8(t.exp_avg, 0, e, n, m);
            load8(t.exp_avg_sq, 0, e, n, v);
        }
        const float decay = fmaf(-lr, t.weight_decay, 1.f);
        float u[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float gk = g[k] * clip;
            m[k] = fmaf(p.beta1, m[k], p.keep1 * gk);
            v[k] = fmaf(p.beta2, v[k], p.keep2 * gk * gk);
            u[k] = sqrtf(v[k]);
            w[k] = fmaf(w[k], decay, -rate * m[k] / fmaf(u[k], widen, p.eps));
        }
        store8(t.param, t.param_dtype, e, n, w);
        if (t.master) store8(t.master, 0, e, n, w);
        if (eight) {
            float sm, su;
            const uint2 cm = encode<false>(m, sm), cu = encode<true>(u, su);
            store_codes(t.exp_avg, e, n, cm);
            store_codes(t.exp_avg_sq, e, n, cu);
            if ((threadIdx.x & 31) == 0 && n > 0) {
                t.exp_avg_scale[block] = sm;
                t.exp_avg_sq_scale[block] = su;
            }
        } else {
            store8(t.exp_avg, 0, e, n, m);
            store8(t.exp_avg_sq, 0, e, n, v);
        }
    }
}

int parts_of(int64_t chunks) {
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(chunks, device_info().sm_count * kCtas)));
}

}  // namespace

int64_t adamw_chunks(int64_t numel) { return (numel + kChunk - 1) / kChunk; }

size_t adamw_workspace_bytes(int64_t chunks) { return sizeof(double) * parts_of(chunks); }

cudaError_t adamw_step(const AdamwStep &q, void *ws, cudaStream_t s) {
    const qg_adamw_tensor *list = static_cast<const qg_adamw_tensor *>(q.list);
    const int parts = parts_of(q.chunks);
    if (q.clip) {
        const cudaError_t e = launch_pdl(sumsq_kernel, dim3(parts), dim3(kThreads), 0, s, list, q.count, q.chunks, static_cast<double *>(ws));
        if (e != cudaSuccess) return e;
    }
    if (q.chunks == 0 && !(q.clip && q.norm)) return cudaSuccess;
    StepArgs a{};
    a.list = list;
    a.count = q.count;
    a.chunks = q.chunks;
    a.lr = static_cast<float>(q.lr);
    a.beta1 = static_cast<float>(q.beta1);
    a.beta2 = static_cast<float>(q.beta2);
    a.keep1 = static_cast<float>(1.0 - q.beta1);
    a.keep2 = static_cast<float>(1.0 - q.beta2);
    a.ln1 = static_cast<float>(std::log(q.beta1));  // -inf for 0: 1 - 0^step is 1
    a.ln2 = static_cast<float>(std::log(q.beta2));
    a.eps = static_cast<float>(q.eps);
    a.lr_dev = q.lr_dev;
    a.step = static_cast<float>(q.step);
    a.step_dev = q.step_dev;
    a.partial = q.clip ? static_cast<const double *>(ws) : nullptr;
    a.parts = parts;
    a.max_norm = q.max_norm;
    a.norm_eps = q.norm_eps;
    a.norm = q.norm;
    const cudaError_t e = launch_pdl(step_kernel, dim3(parts), dim3(kThreads), 0, s, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace qg
