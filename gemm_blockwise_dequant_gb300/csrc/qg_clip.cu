// qg_clip.cu -- the global gradient norm over a list of tensors, and clipping.
//
//   norm = sqrt( sum x^2 ),  out = x * min(1, max_norm / (norm + eps))
//
// Two passes over the gradients, bound by memory: for 839 MB of bf16 the first
// takes 120 us (7.0 TB/s), the second, which reads and writes, 274 us (6.1
// TB/s); for 111 MB 23 and 38 us.  The list is cut into chunks
// of 16 KB (a chunk never crosses a tensor, and its 16-byte vectors lie at
// 16-byte boundaries wherever the tensor begins); a CTA owns a run of
// consecutive chunks, so it searches the list once and then walks it.  The
// second pass walks each run backwards: what the first pass read last is still
// in the L2.
//
// A thread adds the squares of its 16 or 32 values of a chunk in fp32, then
// everything across chunks, threads and CTAs in fp64 in a fixed order.  Squares
// that overflow fp32 or fall below its normal range are added again in fp64, so
// the norm is right wherever it fits fp32.
#include <algorithm>

#include "../../include/qgemm.h"
#include "qg_device.cuh"
#include "qg_internal.h"

namespace qg {
namespace {

constexpr int kThreads = 256;
constexpr int kCtas = 4;                              // of an SM
constexpr int kVec = 4;                               // 16-byte vectors of a thread and chunk
constexpr int kChunkBytes = kThreads * kVec * 16;

// The tensor a CTA is at.  Vector q holds the values q * VE - pad .. of it.
struct Tensor {
    const char *grad;  // at a 16-byte boundary at or before the first value
    char *out;         // the place of that vector's first value (possibly before the tensor)
    int64_t numel, first;
    int dtype, pad;
    bool out_vec;
};

__device__ __forceinline__ Tensor open_tensor(const qg_grad_tensor *list, int i) {
    const qg_grad_tensor t = list[i];
    Tensor r;
    const int es = t.dtype == 0 ? 4 : 2;
    const uintptr_t g = reinterpret_cast<uintptr_t>(t.grad);
    const int off = static_cast<int>(g & 15u);
    r.pad = off / es;
    r.grad = static_cast<const char *>(t.grad) - off;
    r.out = static_cast<char *>(t.out) - off;
    r.out_vec = (reinterpret_cast<uintptr_t>(r.out) & 15u) == 0;
    r.numel = t.numel;
    r.first = t.first_chunk;
    r.dtype = t.dtype;
    return r;
}

// The tensor owning chunk c: the last one with first_chunk <= c (the block counts them).
__device__ int find_tensor(const qg_grad_tensor *list, int count, int64_t c) {
    int n = 0;
    for (int i = 0; i < count; i += kThreads)
        n += __syncthreads_count(i + static_cast<int>(threadIdx.x) < count && list[i + threadIdx.x].first_chunk <= c);
    return n - 1;
}

// The block's sum, valid in thread 0.
__device__ double block_sum(double v, double *red) {
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
        v = 0.0;
        for (int w = 0; w < kThreads / 32; ++w) v += red[w];
    }
    return v;
}

// Every vector of the chunk lies inside the tensor.
__device__ __forceinline__ bool whole_chunk(const Tensor &t, int64_t c) {
    const int ve = t.dtype == 0 ? 4 : 8;
    const int64_t q = (c - t.first) * (kThreads * kVec);
    return q * ve >= t.pad && (q + kThreads * kVec) * ve - t.pad <= t.numel;
}

// The chunk's vectors of this thread, zero outside the tensor.
__device__ __forceinline__ void load_chunk(const Tensor &t, int64_t c, uint4 (&v)[kVec]) {
    const int ve = t.dtype == 0 ? 4 : 8;
    const int64_t q0 = (c - t.first) * (kThreads * kVec) + threadIdx.x;
    if (whole_chunk(t, c)) {  // the loads of a thread together
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] = *reinterpret_cast<const uint4 *>(t.grad + (q0 + i * kThreads) * 16);
        return;
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int64_t q = q0 + i * kThreads, e = q * ve - t.pad;
        v[i] = make_uint4(0, 0, 0, 0);
        if (e >= 0 && e + ve <= t.numel) {
            v[i] = *reinterpret_cast<const uint4 *>(t.grad + q * 16);
        } else if (e < t.numel) {  // the first or last vector
            uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < ve && e + k >= 0 && e + k < t.numel) {
                    if (t.dtype == 0) w[k & 3] = reinterpret_cast<const uint32_t *>(t.grad + q * 16)[k];
                    else w[k >> 1] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(t.grad + q * 16)[k]) << (16 * (k & 1));
                }
            v[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

template <typename F>
__device__ __forceinline__ void for_values(int dtype, const uint4 &v, F f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if (dtype == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f(i, __uint_as_float(w[i]));
    } else if (dtype == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f(2 * i, h2f(static_cast<uint16_t>(w[i] & 0xFFFFu)));
            f(2 * i + 1, h2f(static_cast<uint16_t>(w[i] >> 16)));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f(2 * i, __uint_as_float(w[i] << 16));
            f(2 * i + 1, __uint_as_float(w[i] & 0xFFFF0000u));
        }
    }
}

__global__ void __launch_bounds__(kThreads, kCtas) norm_kernel(const qg_grad_tensor *__restrict__ list, int count, int64_t chunks,
                                                           double *__restrict__ partial) {
    __shared__ double red[kThreads / 32];
    pdl_wait();
    pdl_launch_dependents();  // only now: the second pass reads gradients before it waits for this kernel
    const int64_t c0 = chunks * blockIdx.x / gridDim.x, c1 = chunks * (blockIdx.x + 1) / gridDim.x;
    double total = 0.0;
    if (c0 < c1) {
        int at = find_tensor(list, count, c0);
        Tensor t = open_tensor(list, at);
        int64_t next = at + 1 < count ? list[at + 1].first_chunk : chunks;
        uint4 ahead[kVec];
        load_chunk(t, c0, ahead);
        for (int64_t c = c0; c < c1; ++c) {
            const int dtype = t.dtype;
            uint4 v[kVec];
#pragma unroll
            for (int i = 0; i < kVec; ++i) v[i] = ahead[i];
            if (c + 1 < c1) {  // the next chunk's loads before this one's sums
                if (c + 1 >= next) {
                    while (at + 1 < count && list[at + 1].first_chunk <= c + 1) ++at;
                    t = open_tensor(list, at);
                    next = at + 1 < count ? list[at + 1].first_chunk : chunks;
                }
                load_chunk(t, c + 1, ahead);
            }
            float s[4] = {};
            uint32_t any = 0;
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                for_values(dtype, v[i], [&](int k, float x) { s[k & 3] = fmaf(x, x, s[k & 3]); });
                any |= (v[i].x | v[i].y) | (v[i].z | v[i].w);
            }
            const float sum = (s[0] + s[1]) + (s[2] + s[3]);
            if (sum >= 1e-30f && sum <= 3e38f) {
                total += sum;
            } else if (any) {
#pragma unroll
                for (int i = 0; i < kVec; ++i)
                    for_values(dtype, v[i], [&](int, float x) { total += static_cast<double>(x) * x; });
            }
        }
    }
    total = block_sum(total, red);
    if (threadIdx.x == 0) partial[blockIdx.x] = total;
}

__device__ __forceinline__ void store_chunk(const Tensor &t, int64_t c, const uint4 (&v)[kVec], float coef) {
    const int ve = t.dtype == 0 ? 4 : 8;
    const int64_t q0 = (c - t.first) * (kThreads * kVec) + threadIdx.x;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int64_t q = q0 + i * kThreads, e = q * ve - t.pad;
        if (e >= t.numel) continue;
        uint32_t w[4];
        if (t.dtype == 0) {
            for_values(0, v[i], [&](int k, float y) { w[k] = __float_as_uint(y * coef); });
        } else {
            float x[8];
            for_values(t.dtype, v[i], [&](int k, float y) { x[k] = y * coef; });
#pragma unroll
            for (int k = 0; k < 4; ++k)
                w[k] = t.dtype == 1 ? f2h(x[2 * k]) | static_cast<uint32_t>(f2h(x[2 * k + 1])) << 16
                                    : f2bf(x[2 * k]) | static_cast<uint32_t>(f2bf(x[2 * k + 1])) << 16;
        }
        char *o = t.out + q * 16;
        if (t.out_vec && e >= 0 && e + ve <= t.numel) {
            *reinterpret_cast<uint4 *>(o) = make_uint4(w[0], w[1], w[2], w[3]);
        } else if (t.dtype == 0) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (e + k >= 0 && e + k < t.numel) reinterpret_cast<uint32_t *>(o)[k] = w[k];
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (e + k >= 0 && e + k < t.numel) reinterpret_cast<uint16_t *>(o)[k] = static_cast<uint16_t>(w[k >> 1] >> (16 * (k & 1)));
        }
    }
}

__global__ void __launch_bounds__(kThreads, kCtas) scale_kernel(const qg_grad_tensor *__restrict__ list, int count, int64_t chunks,
                                                            const double *__restrict__ partial, int parts, float max_norm, float eps,
                                                            float *norm_out) {
    __shared__ float factor;
    const int64_t c0 = chunks * blockIdx.x / gridDim.x, c1 = chunks * (blockIdx.x + 1) / gridDim.x;
    Tensor t;
    int at = 0;
    uint4 v[kVec];
    if (c0 < c1) {  // under the first pass: the first chunk of this one
        at = find_tensor(list, count, c1 - 1);
        t = open_tensor(list, at);
        load_chunk(t, c1 - 1, v);
    }
    pdl_launch_dependents();
    pdl_wait();
    if (threadIdx.x < 32) {  // one warp: fp64 is slow
        double sum = 0.0;
        for (int i = threadIdx.x; i < parts; i += 32) sum += partial[i];
        for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (threadIdx.x == 0) {
            const float norm = static_cast<float>(sqrt(sum));
            if (blockIdx.x == 0) *norm_out = norm;
            const float c = max_norm / (norm + eps);
            factor = c > 1.f ? 1.f : c;  // a NaN stays one
        }
    }
    __syncthreads();
    const float coef = factor;
    if (c0 >= c1) return;
    for (int64_t c = c1 - 1;; --c) {
        const Tensor here = t;
        uint4 ahead[kVec];
        if (c > c0) {
            if (c - 1 < t.first) {
                do --at;
                while (list[at].first_chunk > c - 1 || list[at].numel == 0);  // an empty tensor owns no chunk
                t = open_tensor(list, at);
            }
            load_chunk(t, c - 1, ahead);
        }
        store_chunk(here, c, v, coef);
        if (c == c0) break;
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] = ahead[i];
    }
}

int parts_of(int64_t chunks) {
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(chunks, device_info().sm_count * kCtas)));
}

}  // namespace

int64_t clip_chunks(const void *grad, int64_t numel, int elem_size) {
    if (numel == 0) return 0;
    return (numel * elem_size + static_cast<int64_t>(reinterpret_cast<uintptr_t>(grad) & 15u) + kChunkBytes - 1) / kChunkBytes;
}

size_t clip_workspace_bytes(int64_t chunks) { return sizeof(double) * parts_of(chunks); }

cudaError_t clip_grad_norm(const void *list, int count, int64_t chunks, float max_norm, float eps, float *norm, void *ws,
                           cudaStream_t s) {
    const qg_grad_tensor *l = static_cast<const qg_grad_tensor *>(list);
    const int parts = parts_of(chunks);
    double *partial = static_cast<double *>(ws);
    cudaError_t e = launch_pdl(norm_kernel, dim3(parts), dim3(kThreads), 0, s, l, count, chunks, partial);
    if (e != cudaSuccess) return e;
    e = launch_pdl(scale_kernel, dim3(parts), dim3(kThreads), 0, s, l, count, chunks, static_cast<const double *>(partial),
                   parts, max_norm, eps, norm);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace qg
