// qg_moe_tokens.cu -- a mixture-of-experts layer over a few tokens: the choice of experts from the router's logits, and
// the layer as three launches (both expert products, qg_moe_tokens.cuh, and the weighted sum of each token's experts).
//
//   ids[t] = the k largest of logits[t], the lower index first among equals
//   weights[t][j] = exp(l_j - M) / sum exp(l_i - M)     over the k chosen (renormalize) or over all experts
//   y[t] = sum_j weights[t][j] o[t * k + j]              in the order of the slots
#include "../../include/qgemm.h"
#include "qg_device.cuh"
#include "qg_moe_tokens.h"

namespace qg {
namespace {

using moe::kMaxExperts;

constexpr int kRouteWarps = 4, kPerLane = kMaxExperts / 32;

__device__ __forceinline__ unsigned long long order_key(float x, int index) {
    const uint32_t b = __float_as_uint(x + 0.f);  // one zero
    const uint32_t o = x != x ? 0xFFFFFFFFu : b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
    return static_cast<unsigned long long>(o) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(index));
}

// A warp for each token: bound by the latency of k rounds of a warp-wide maximum.
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(const void *logits, int dtype, int64_t ld, int T, int E, int k, int renormalize,
                                                                 int32_t *ids, float *weights) {
    const int t = blockIdx.x * kRouteWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    pdl_launch_dependents();
    pdl_wait();
    if (t >= T) return;
    float x[kPerLane];
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) x[i] = i * 32 + lane < E ? load_a_elem(logits, dtype, static_cast<size_t>(t * ld + i * 32 + lane)) : -INFINITY;
    unsigned taken = 0;
    float top = -INFINITY, mine = 0.f, chosen = 0.f;  // lane j keeps slot j's logit
    for (int j = 0; j < k; ++j) {
        unsigned long long best = 0;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i)
            if (i * 32 + lane < E && !(taken >> i & 1)) {
                const unsigned long long key = order_key(x[i], i * 32 + lane);
                best = key > best ? key : best;
            }
        for (int o = 16; o >= 1; o >>= 1) {
            const unsigned long long other = __shfl_xor_sync(~0u, best, o);
            best = other > best ? other : best;
        }
        const int e = static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(best));
        const uint32_t o = static_cast<uint32_t>(best >> 32);
        const float v = o == 0xFFFFFFFFu ? __int_as_float(0x7FFFFFFF) : __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
        if (j == 0) top = v;
        if (lane == j) mine = v, ids[static_cast<int64_t>(t) * k + j] = e;
        if ((e & 31) == lane) taken |= 1u << (e >> 5);
    }
    // an expert at -inf has weight 0, also where all are
    const bool none = top == -INFINITY;
    float sum = 0.f;
    if (lane < k && !none) sum = chosen = expf(mine - top);
    if (!renormalize) {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i)
            if (i * 32 + lane < E && !none) sum += expf(x[i] - top);
    }
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    if (lane < k) weights[static_cast<int64_t>(t) * k + lane] = none ? 0.f : chosen / sum;
}

// Four outputs a thread, the slots in their order: two to three microseconds with the launch, bound by latency.
__global__ void __launch_bounds__(128) combine_kernel(const float *__restrict__ o, const int32_t *__restrict__ ids, const float *__restrict__ weights,
                                                      int T, int k, int E, int hidden, void *y, int y_dtype) {
    pdl_launch_dependents();
    pdl_wait();
    const int t = blockIdx.y, n = (blockIdx.x * blockDim.x + threadIdx.x) * 4;
    if (n >= hidden) return;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = 0; j < k; ++j) {
        const int pair = t * k + j, e = ids[pair];
        if (e < 0 || e >= E) continue;
        const float w = weights[pair];
        const float4 v = *reinterpret_cast<const float4 *>(o + static_cast<size_t>(pair) * hidden + n);
        s.x = fmaf(w, v.x, s.x), s.y = fmaf(w, v.y, s.y), s.z = fmaf(w, v.z, s.z), s.w = fmaf(w, v.w, s.w);
    }
    const size_t at = static_cast<size_t>(t) * hidden + n;
    if (y_dtype == QG_F32) *reinterpret_cast<float4 *>(static_cast<float *>(y) + at) = s;
    else if (y_dtype == QG_F16) *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(y) + at) = make_uint2(f2h(s.x) | static_cast<uint32_t>(f2h(s.y)) << 16, f2h(s.z) | static_cast<uint32_t>(f2h(s.w)) << 16);
    else *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(y) + at) = make_uint2(f2bf(s.x) | static_cast<uint32_t>(f2bf(s.y)) << 16, f2bf(s.z) | static_cast<uint32_t>(f2bf(s.w)) << 16);
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

cudaError_t route_topk(const void *logits, int dtype, int64_t ld, int T, int E, int k, int renormalize, int32_t *ids, float *weights, cudaStream_t s) {
    const cudaError_t e = launch_pdl(route_kernel, dim3((T + kRouteWarps - 1) / kRouteWarps), dim3(kRouteWarps * 32), 0, s, logits, dtype, ld, T, E, k,
                                     renormalize, ids, weights);
    return e != cudaSuccess ? e : cudaGetLastError();
}

size_t moe_tokens_workspace_bytes(int T, int k, int hidden, int inter) {
    const size_t P = static_cast<size_t>(T) * k;
    return up256(P * inter * sizeof(float)) + P * hidden * sizeof(float);
}

cudaError_t moe_tokens(const MoeTokens &q, void *ws, cudaStream_t s) {
    const int P = q.T * q.k;
    float *h = static_cast<float *>(ws), *o = reinterpret_cast<float *>(static_cast<char *>(ws) + up256(static_cast<size_t>(P) * q.inter * sizeof(float)));
    const auto experts = q.bits == 2 ? moe::launch_experts<2> : q.bits == 4 ? moe::launch_experts<4> : moe::launch_experts<8>;
    const auto fit = q.bits == 2 ? moe::experts_fit<2> : q.bits == 4 ? moe::experts_fit<4> : moe::experts_fit<8>;
    if (!fit(q.hidden, q.bs, q.fc1_zp != nullptr) || !fit(q.inter, q.bs, q.fc2_zp != nullptr)) return cudaErrorNotSupported;
    moe::Args a{};
    a.ids = q.ids;
    a.P = P;
    a.k = q.k;
    a.E = q.E;
    a.bs = q.bs;
    a.most_rows = q.T;
    a.status = q.status;
    a.terms = 1;
    a.fc = 1;
    a.src = q.x;
    a.src_dtype = q.x_dtype;
    a.w = q.fc1_w;
    a.scales = q.fc1_scales;
    a.zp = q.fc1_zp;
    a.bias = q.fc1_bias;
    a.N = 2 * q.inter;
    a.K = q.hidden;
    a.interleaved = q.interleaved;
    a.out = h;
    cudaError_t e = experts(a, s);
    if (e != cudaSuccess) return e;
    a.fc = 2;
    a.src = h;
    a.src_dtype = QG_F32;
    a.w = q.fc2_w;
    a.scales = q.fc2_scales;
    a.zp = q.fc2_zp;
    a.bias = q.fc2_bias;
    a.N = q.hidden;
    a.K = q.inter;
    a.out = o;
    a.status = nullptr;
    // h is fp32: one fp16 of it is off by as much as the rounding of an fp16 y, which two are not; beside that of a bf16 y it is
    // little (1.666e-3 instead of 1.656e-3 from fp64; two terms take 64 tokens from 460 to 478 us)
    a.terms = q.y_dtype == QG_BF16 ? 1 : 2;
    e = experts(a, s);
    if (e != cudaSuccess) return e;
    e = launch_pdl(combine_kernel, dim3((q.hidden / 4 + 127) / 128, q.T), dim3(128), 0, s, static_cast<const float *>(o), q.ids, q.weights, q.T, q.k, q.E,
                   q.hidden, q.y, q.y_dtype);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace qg
