// qg_lora_wgrad.cu -- launches of the adapters' own gradients.
#include "qg_lora_wgrad.cuh"

#include <algorithm>

namespace qg {
namespace {

template <int XT, bool NATIVE, int MJ>
cudaError_t launch_one(WgradArgs q, cudaStream_t s) {
    using Kern = WgradKernel<XT, NATIVE, MJ>;
    auto kern = lora_wgrad_kernel<XT, NATIVE, MJ>;
    const LoraProblem &p = q.p;
    for (int w = 0; w < 2; ++w) q.tiles[w] = (q.cols[w] + Kern::COLS - 1) / Kern::COLS;
    const int chunks = (p.r + Kern::RJ - 1) / Kern::RJ;
    // As many CTAs as are resident at once (rank > 16: one an SM, else two), while each still has two row chunks.
    const int slots = device_info().sm_count * (MJ > 1 ? 1 : 2);
    const int64_t ctas = static_cast<int64_t>(q.tiles[0] + q.tiles[1]) * p.na * chunks;
    q.cs = 1;
    while (q.cs < 8 && ctas * q.cs * 2 <= slots && p.T / p.na > 2 * kWgChunk * q.cs) q.cs *= 2;
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e = allow_smem(kern, done, Kern::SMEM);
    if (e != cudaSuccess) return e;
    return launch_cluster(kern, dim3(static_cast<unsigned>(q.tiles[0] + q.tiles[1]) * q.cs, p.na, chunks), dim3(256), Kern::SMEM, s, q.cs, q);
}

template <int XT, bool NATIVE>
cudaError_t launch_rank(const WgradArgs &q, cudaStream_t s) {
    return q.p.r <= 16 ? launch_one<XT, NATIVE, 1>(q, s) : q.p.r <= 32 ? launch_one<XT, NATIVE, 2>(q, s) : launch_one<XT, NATIVE, 4>(q, s);
}

}  // namespace

cudaError_t launch_wgrad(const WgradArgs &q, int x_dtype, cudaStream_t s) {
    if (x_dtype == kBF16) return q.g_dtype == kBF16 ? launch_rank<kBF16, true>(q, s) : launch_rank<kBF16, false>(q, s);
    return x_dtype == kF16 ? launch_rank<kF16, false>(q, s) : launch_rank<kF32, false>(q, s);
}

}  // namespace qg
