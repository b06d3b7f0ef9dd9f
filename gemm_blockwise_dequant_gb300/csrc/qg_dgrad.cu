// qg_dgrad.cu -- dX[M][K] = dY[M][N] . dequant(W)[N][K]: the gradient of the
// activations through a frozen blockwise-quantized weight.
//
// The contraction runs over the weight's rows n, so a block's scale and zero
// point change along the sum and the weight has to be formed before the
// product (in the forward pass they could be applied to a block's partial
// sum).
#include <algorithm>

#include "qg_device.cuh"
#include "qg_internal.h"

namespace qg {
namespace {

// One weight in fp32, exactly as the forward kernels define it.
__device__ float weight_at(const GemmProblem &p, int n, int k) {
    const int nb = p.K / p.bs, b = k / p.bs;
    const size_t bit = static_cast<size_t>(k) * p.bits;
    const uint8_t *row = p.W + static_cast<size_t>(n) * (static_cast<size_t>(p.K) * p.bits / 8);
    unsigned v = row[bit >> 3];
    if ((bit & 7) + p.bits > 8) v |= static_cast<unsigned>(row[(bit >> 3) + 1]) << 8;
    const unsigned q = (v >> (bit & 7)) & ((1u << p.bits) - 1u);
    const size_t pi = static_cast<size_t>(n) * nb + b;
    if (p.kind == WK_CODEBOOK) return __fmul_rn(p.codebook[q], p.absmax[pi]);
    const float z = p.zp_mode == ZP_TENSOR ? h2f(p.zp[pi]) : p.uniform_zp;
    return __fmul_rn(__fsub_rn(static_cast<float>(q), z), h2f(p.scales[pi]));
}

// 64 x 64 tile of dX, 16 weight rows at a time, 4 x 4 outputs a thread.
__global__ void __launch_bounds__(256) dgrad_simple_kernel(const GemmProblem p) {
    __shared__ float dy[16][68], w[16][68];
    const int k0 = blockIdx.x * 64, m0 = blockIdx.y * 64, t = threadIdx.x;
    const int tm = (t >> 4) * 4, tk = (t & 15) * 4;
    float acc[4][4] = {};
    pdl_wait();
    pdl_launch_dependents();
    for (int n0 = 0; n0 < p.N; n0 += 16) {
        for (int i = t; i < 16 * 64; i += 256) {
            const int m = i >> 4, n = i & 15;
            dy[n][m] = m0 + m < p.M && n0 + n < p.N ? load_a_elem(p.A, p.a_dtype, static_cast<size_t>(m0 + m) * p.N + n0 + n) : 0.f;
        }
        for (int i = t; i < 16 * 64; i += 256) {
            const int n = i >> 6, k = i & 63;
            w[n][k] = n0 + n < p.N && k0 + k < p.K ? weight_at(p, n0 + n, k0 + k) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < 16; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(dy[n][tm + i], w[n][tk + j], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j)
            if (m0 + tm + i < p.M && k0 + tk + j < p.K)
                store_y_elem(p.Y, p.y_dtype, static_cast<size_t>(m0 + tm + i) * p.K + k0 + tk + j, acc[i][j]);
}

}  // namespace

size_t dgrad_workspace_bytes(int, int, int, int, int) { return 0; }

cudaError_t dgrad(const GemmProblem &p, void *, cudaStream_t s) {
    const cudaError_t e = launch_pdl(dgrad_simple_kernel, dim3((p.K + 63) / 64, (p.M + 63) / 64), dim3(256), 0, s, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace qg
