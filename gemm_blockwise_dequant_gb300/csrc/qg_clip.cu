// qg_clip.cu -- the global gradient norm over a list of tensors, and clipping.
//
//   norm = sqrt( sum x^2 ),  out = x * min(1, max_norm / (norm + eps))
//
// The list is cut into chunks of kChunk values (a chunk never crosses a
// tensor); a CTA owns a run of consecutive chunks, so it searches the list
// once and then walks it.  A thread adds the squares of its values of a chunk
// in fp32, then everything across chunks, threads and CTAs in fp64 in a fixed
// order.  The squares of a chunk that overflow fp32 or fall below its normal
// range are added again in fp64, so the norm is right wherever it fits fp32.
#include <algorithm>

#include "../../include/qgemm.h"
#include "qg_device.cuh"
#include "qg_internal.h"

namespace qg {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 16;                      // values per thread of a chunk
constexpr int kChunk = kThreads * kPer;

// The tensor owning chunk c: the last one with first_chunk <= c that has values.
__device__ int find_tensor(const qg_grad_tensor *list, int count, int64_t c) {
    int lo = 0, hi = count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (list[mid].first_chunk <= c) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ double block_sum(double v, double *red) {
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0;
    for (int w = 0; w < kThreads / 32; ++w) v += red[w];
    __syncthreads();
    return v;
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const qg_grad_tensor *__restrict__ list, int count,
                                                        int64_t chunks, double *__restrict__ partial) {
    __shared__ double red[kThreads / 32];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t c0 = chunks * blockIdx.x / gridDim.x, c1 = chunks * (blockIdx.x + 1) / gridDim.x;
    double total = 0.0;
    if (c0 < c1) {
        int t = find_tensor(list, count, c0);
        for (int64_t c = c0; c < c1; ++c) {
            while (t + 1 < count && list[t + 1].first_chunk <= c) ++t;
            const int64_t base = (c - list[t].first_chunk) * kChunk, n = list[t].numel;
            float v[kPer], s = 0.f, mx = 0.f;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int64_t e = base + i * kThreads + threadIdx.x;
                v[i] = e < n ? load_a_elem(list[t].grad, list[t].dtype, e) : 0.f;
                s = fmaf(v[i], v[i], s);
                mx = fmaxf(mx, fabsf(v[i]));
            }
            if (s >= 1e-30f && s <= 3e38f) {
                total += s;
            } else if (mx > 0.f || s != s) {
                for (int i = 0; i < kPer; ++i) total += static_cast<double>(v[i]) * v[i];
            }
        }
    }
    total = block_sum(total, red);
    if (threadIdx.x == 0) partial[blockIdx.x] = total;
}

__global__ void __launch_bounds__(kThreads) scale_kernel(const qg_grad_tensor *__restrict__ list, int count,
                                                         int64_t chunks, const double *__restrict__ partial, int parts,
                                                         float max_norm, float eps, float *norm_out) {
    __shared__ double red[kThreads / 32];
    pdl_wait();
    pdl_launch_dependents();
    double sum = 0.0;
    for (int i = threadIdx.x; i < parts; i += kThreads) sum += partial[i];
    sum = block_sum(sum, red);
    const float norm = static_cast<float>(sqrt(sum));
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm;
    float coef = max_norm / (norm + eps);
    if (coef > 1.f) coef = 1.f;  // a NaN stays one
    const int64_t c0 = chunks * blockIdx.x / gridDim.x, c1 = chunks * (blockIdx.x + 1) / gridDim.x;
    if (c0 >= c1) return;
    int t = find_tensor(list, count, c0);
    for (int64_t c = c0; c < c1; ++c) {
        while (t + 1 < count && list[t + 1].first_chunk <= c) ++t;
        const int64_t base = (c - list[t].first_chunk) * kChunk, n = list[t].numel;
        for (int i = 0; i < kPer; ++i) {
            const int64_t e = base + i * kThreads + threadIdx.x;
            if (e >= n) break;
            const int dt = list[t].dtype;
            const void *g = list[t].grad;
            const float v = dt == 0 ? static_cast<const float *>(g)[e]
                                    : dt == 1 ? h2f(static_cast<const uint16_t *>(g)[e]) : bf2f(static_cast<const uint16_t *>(g)[e]);
            store_y_elem(list[t].out, dt, e, v * coef);
        }
    }
}

int parts_of(int64_t chunks) {
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(chunks, device_info().sm_count * 8)));
}

}  // namespace

int64_t clip_chunks(int64_t numel) { return (numel + kChunk - 1) / kChunk; }

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
