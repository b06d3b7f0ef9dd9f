// qg_lora.cu -- low-rank adapters of many requests beside a shared projection:
// the forward pass (apply) and the backward pass (grad).
#include <algorithm>

#include "qg_device.cuh"
#include "qg_internal.h"

namespace qg {
namespace {

// A row of no request (at or past the last offset, or refused offsets): untouched.
constexpr int kNoRow = -2;

// Adapter of every row: one CTA checks the offsets and writes the map.
__global__ void __launch_bounds__(1024) row_map_kernel(const LoraProblem p, int *__restrict__ map) {
    pdl_wait();
    pdl_launch_dependents();
    int bad = threadIdx.x == 0 && p.offs[0] != 0;
    for (int s = threadIdx.x; s < p.S; s += blockDim.x) {
        if (p.offs[s + 1] < p.offs[s]) bad = 1;
        if (s == p.S - 1 && p.offs[s + 1] > p.T) bad = 1;
    }
    bad = __syncthreads_or(bad);
    const int end = bad ? 0 : static_cast<int>(p.offs[p.S]);
    for (int t = end + threadIdx.x; t < p.T; t += blockDim.x) map[t] = kNoRow;
    int strange = 0;
    if (!bad)
        for (int s = threadIdx.x >> 5; s < p.S; s += blockDim.x >> 5) {
            int a = p.ids[s];
            if (a >= p.na) strange = 1;
            if (a < 0 || a >= p.na) a = -1;
            for (int t = static_cast<int>(p.offs[s]) + (threadIdx.x & 31); t < p.offs[s + 1]; t += 32) map[t] = a;
        }
    if ((bad || strange) && p.status) *p.status = 1;
}

// V[t][j] = sum_k X[t][k] A[a][j][k]: one warp per (t, j)
__global__ void shrink_kernel(const LoraApply q, const int *__restrict__ map, float *__restrict__ V) {
    pdl_wait();
    pdl_launch_dependents();
    const LoraProblem &p = q.p;
    const int w = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int t = w / p.r, j = w - t * p.r;
    if (t >= p.T) return;
    const int a = map[t];
    if (a == kNoRow) return;
    float s = 0.f;
    if (a >= 0)
        for (int k = lane; k < p.K; k += 32)
            s = fmaf(load_a_elem(q.X, q.x_dtype, t * q.ldx + k), load_a_elem(p.A, p.w_dtype, (static_cast<size_t>(a) * p.r + j) * p.K + k), s);
    for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) {
        V[static_cast<size_t>(t) * p.r + j] = s;
        if (q.V) q.V[static_cast<size_t>(t) * p.r + j] = s;
    }
}

__global__ void expand_kernel(const LoraApply q, const int *__restrict__ map, const float *__restrict__ V) {
    pdl_wait();
    pdl_launch_dependents();
    const LoraProblem &p = q.p;
    const int t = blockIdx.y, n = blockIdx.x * blockDim.x + threadIdx.x;
    const int a = map[t];
    if (n >= p.N || a == kNoRow) return;
    float s = 0.f;
    if (a >= 0) {
        for (int j = 0; j < p.r; ++j)
            s = fmaf(V[static_cast<size_t>(t) * p.r + j], load_a_elem(p.B, p.w_dtype, (static_cast<size_t>(a) * p.N + n) * p.r + j), s);
        if (p.scaling) s *= p.scaling[a];
    }
    float y = 0.f;
    if (q.Yin) {
        const size_t i = t * q.ldyin + n;
        y = q.yin_dtype == 0 ? static_cast<const float *>(q.Yin)[i]
                             : q.yin_dtype == 1 ? h2f(static_cast<const uint16_t *>(q.Yin)[i]) : bf2f(static_cast<const uint16_t *>(q.Yin)[i]);
    }
    store_y_elem(q.Y, q.y_dtype, t * q.ldy + n, y + s);
}

// G[t][j] = scaling sum_n dY[t][n] B[a][n][j]: one warp per (t, j)
__global__ void grad_shrink_kernel(const LoraGrad q, const int *__restrict__ map, float *__restrict__ G) {
    pdl_wait();
    pdl_launch_dependents();
    const LoraProblem &p = q.p;
    const int w = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int t = w / p.r, j = w - t * p.r;
    if (t >= p.T) return;
    const int a = map[t];
    if (a < 0) return;
    float s = 0.f;
    for (int n = lane; n < p.N; n += 32)
        s = fmaf(load_a_elem(q.dY, q.x_dtype, t * q.lddy + n), load_a_elem(p.B, p.w_dtype, (static_cast<size_t>(a) * p.N + n) * p.r + j), s);
    for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) G[static_cast<size_t>(t) * p.r + j] = p.scaling ? s * p.scaling[a] : s;
}

__global__ void grad_input_kernel(const LoraGrad q, const int *__restrict__ map, const float *__restrict__ G) {
    pdl_wait();
    pdl_launch_dependents();
    const LoraProblem &p = q.p;
    const int t = blockIdx.y, k = blockIdx.x * blockDim.x + threadIdx.x;
    const int a = map[t];
    if (k >= p.K || a == kNoRow) return;
    float s = 0.f;
    if (a >= 0)
        for (int j = 0; j < p.r; ++j)
            s = fmaf(G[static_cast<size_t>(t) * p.r + j], load_a_elem(p.A, p.w_dtype, (static_cast<size_t>(a) * p.r + j) * p.K + k), s);
    const size_t i = t * q.lddx + k;
    float x = 0.f;
    if (q.dXin)
        x = q.x_dtype == 0 ? static_cast<const float *>(q.dXin)[i]
                           : q.x_dtype == 1 ? h2f(static_cast<const uint16_t *>(q.dXin)[i]) : bf2f(static_cast<const uint16_t *>(q.dXin)[i]);
    store_y_elem(q.dX, q.x_dtype, i, x + s);
}

// dA (which = 0) or dB (1): one thread per element, over all the rows
__global__ void grad_weight_kernel(const LoraGrad q, const int *__restrict__ map, const float *__restrict__ G, int which) {
    pdl_wait();
    pdl_launch_dependents();
    const LoraProblem &p = q.p;
    const int cols = which ? p.N : p.K;
    const int c = blockIdx.x * blockDim.x + threadIdx.x, j = blockIdx.y, a = blockIdx.z;
    if (c >= cols) return;
    const float *skinny = which ? q.V : G;
    float s = 0.f;
    for (int t = 0; t < p.T; ++t)
        if (map[t] == a)
            s = fmaf(skinny[static_cast<size_t>(t) * p.r + j],
                     which ? load_a_elem(q.dY, q.x_dtype, t * q.lddy + c) : load_a_elem(q.X, q.x_dtype, t * q.ldx + c), s);
    if (which && p.scaling) s *= p.scaling[a];
    const size_t i = which ? (static_cast<size_t>(a) * p.N + c) * p.r + j : (static_cast<size_t>(a) * p.r + j) * p.K + c;
    void *d = which ? q.dB : q.dA;
    if (q.accumulate) s += q.g_dtype == 0 ? static_cast<float *>(d)[i]
                                          : q.g_dtype == 1 ? h2f(static_cast<uint16_t *>(d)[i]) : bf2f(static_cast<uint16_t *>(d)[i]);
    store_y_elem(d, q.g_dtype, i, s);
}

size_t map_bytes(int T) { return (static_cast<size_t>(T) * 4 + 255) / 256 * 256; }

}  // namespace

size_t lora_apply_workspace_bytes(int T, int, int r) { return map_bytes(T) + static_cast<size_t>(T) * r * 4; }

cudaError_t lora_apply(const LoraApply &q, void *ws, cudaStream_t s) {
    const LoraProblem &p = q.p;
    int *map = static_cast<int *>(ws);
    float *V = reinterpret_cast<float *>(static_cast<char *>(ws) + map_bytes(p.T));
    cudaError_t e = launch_pdl(row_map_kernel, dim3(1), dim3(1024), 0, s, p, map);
    if (e != cudaSuccess) return e;
    e = launch_pdl(shrink_kernel, dim3(static_cast<unsigned>((static_cast<size_t>(p.T) * p.r + 7) / 8)), dim3(256), 0, s, q,
                   static_cast<const int *>(map), V);
    if (e != cudaSuccess) return e;
    for (int t0 = 0; t0 < p.T; t0 += 65535) {  // grid.y
        if (t0) return cudaErrorNotSupported;
        e = launch_pdl(expand_kernel, dim3((p.N + 255) / 256, std::min(p.T, 65535)), dim3(256), 0, s, q,
                       static_cast<const int *>(map), static_cast<const float *>(V));
        if (e != cudaSuccess) return e;
    }
    return cudaGetLastError();
}

size_t lora_grad_workspace_bytes(int T, int, int, int r, int, int) { return map_bytes(T) + static_cast<size_t>(T) * r * 4; }

cudaError_t lora_grad(const LoraGrad &q, void *ws, cudaStream_t s) {
    const LoraProblem &p = q.p;
    if (p.T > 65535) return cudaErrorNotSupported;
    int *map = static_cast<int *>(ws);
    float *G = reinterpret_cast<float *>(static_cast<char *>(ws) + map_bytes(p.T));
    cudaError_t e = launch_pdl(row_map_kernel, dim3(1), dim3(1024), 0, s, p, map);
    if (e != cudaSuccess) return e;
    const int *m = map;
    const float *g = G;
    e = launch_pdl(grad_shrink_kernel, dim3(static_cast<unsigned>((static_cast<size_t>(p.T) * p.r + 7) / 8)), dim3(256), 0, s, q, m, G);
    if (e == cudaSuccess && q.dX) e = launch_pdl(grad_input_kernel, dim3((p.K + 255) / 256, p.T), dim3(256), 0, s, q, m, g);
    if (e == cudaSuccess && p.na > 0) {
        e = launch_pdl(grad_weight_kernel, dim3((p.K + 127) / 128, p.r, p.na), dim3(128), 0, s, q, m, g, 0);
        if (e == cudaSuccess) e = launch_pdl(grad_weight_kernel, dim3((p.N + 127) / 128, p.r, p.na), dim3(128), 0, s, q, m, g, 1);
    }
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace qg
