// qg_token_api.cu -- the C ABI of the entry points around a few tokens' logits and experts (include/qgemm.h): argument
// checks and dispatch.  Everything is refused or accepted on the host before anything is enqueued.
#include <cmath>
#include <initializer_list>

#include "../../include/qgemm.h"
#include "qg_internal.h"

namespace {

bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool valid_dtype(int d) { return d == QG_F32 || d == QG_F16 || d == QG_BF16; }
size_t esize(int d) { return d == QG_F32 ? 4 : 2; }

constexpr int kMaxRows = 1 << 20, kMaxVocab = 1 << 28, kMaxTop = 64;
constexpr float kMaxInvTemperature = 2.3e38f;  // times log2(e) it is finite
// Every CTA of the expert products groups all pairs by expert before it begins: more of them are a ragged GEMM's work.
constexpr int kMaxSlots = 16, kMaxPairs = 1024, kMaxExperts = 512;

int finish(cudaError_t e) {
    if (e == cudaErrorNotSupported) return QG_ERR_UNSUPPORTED;
    return e == cudaSuccess ? QG_OK : QG_ERR_CUDA;
}

int check_logits(const void *X, int x_dtype, int64_t ldx, const int64_t *targets, int rows, int vocab, float inv_t) {
    if (!valid_dtype(x_dtype) || rows < 0 || vocab < 1 || ldx < vocab) return QG_ERR_INVALID_ARG;
    if (!(inv_t > 0.f && inv_t < INFINITY)) return QG_ERR_INVALID_ARG;  // NaN too
    if (rows > kMaxRows || vocab > kMaxVocab) return QG_ERR_UNSUPPORTED;
    if (!aligned(targets, 8)) return QG_ERR_INVALID_ARG;
    if (rows > 0 && (!X || !aligned(X, esize(x_dtype)))) return QG_ERR_INVALID_ARG;
    return QG_OK;
}

}  // namespace

extern "C" {

int qg_token_logprobs(const void *X, int x_dtype, int64_t ldx, const int64_t *targets, int rows, int vocab,
                      float inv_temperature, float *logprob, float *entropy, float *lse, int top_k, int64_t *top_ids,
                      float *top_logprobs, int *status_dev, qg_stream_t stream) {
    (void)cudaGetLastError();  // do not report an earlier, unrelated failure as ours
    const int st = check_logits(X, x_dtype, ldx, targets, rows, vocab, inv_temperature);
    if (st != QG_OK) return st;
    if (top_k < 0 || top_k > vocab) return QG_ERR_INVALID_ARG;
    if (top_k > kMaxTop || inv_temperature > kMaxInvTemperature) return QG_ERR_UNSUPPORTED;
    if (!aligned(logprob, 4) || !aligned(entropy, 4) || !aligned(lse, 4) || !aligned(top_ids, 8) || !aligned(top_logprobs, 4) || !aligned(status_dev, 4))
        return QG_ERR_INVALID_ARG;
    if (rows == 0) return QG_OK;
    if (top_k > 0 && (!top_ids || !top_logprobs)) return QG_ERR_INVALID_ARG;
    const qg::TokenLogprobs q{X, x_dtype, ldx, targets, rows, vocab, top_k, inv_temperature, logprob, entropy, lse, top_ids, top_logprobs, status_dev};
    return finish(qg::token_logprobs(q, reinterpret_cast<cudaStream_t>(stream)));
}

int qg_token_logprobs_grad(const void *X, int x_dtype, int64_t ldx, const int64_t *targets, const float *lse,
                           const float *entropy, const float *d_logprob, const float *d_entropy, float inv_temperature,
                           void *dX, int64_t lddx, int rows, int vocab, qg_stream_t stream) {
    (void)cudaGetLastError();
    const int st = check_logits(X, x_dtype, ldx, targets, rows, vocab, inv_temperature);
    if (st != QG_OK) return st;
    if (lddx < vocab || (dX == X && lddx != ldx)) return QG_ERR_INVALID_ARG;
    if (!aligned(lse, 4) || !aligned(entropy, 4) || !aligned(d_logprob, 4) || !aligned(d_entropy, 4) || !aligned(dX, esize(x_dtype))) return QG_ERR_INVALID_ARG;
    if (rows == 0) return QG_OK;
    if (!lse || !d_logprob || !dX || (d_entropy && !entropy)) return QG_ERR_INVALID_ARG;
    const qg::TokenLogprobsGrad q{X, x_dtype, ldx, targets, lse, entropy, d_logprob, d_entropy, dX, lddx, rows, vocab, inv_temperature};
    return finish(qg::token_logprobs_grad(q, reinterpret_cast<cudaStream_t>(stream)));
}

int qmoe_route_topk(const void *logits, int dtype, int64_t ld, int tokens, int num_experts, int k, int renormalize,
                    int32_t *expert_ids, float *expert_weights, qg_stream_t stream) {
    (void)cudaGetLastError();
    if (!valid_dtype(dtype) || tokens < 0 || num_experts < 1 || k < 1 || k > num_experts || ld < num_experts) return QG_ERR_INVALID_ARG;
    if (renormalize != 0 && renormalize != 1) return QG_ERR_INVALID_ARG;
    if (tokens > kMaxRows || num_experts > kMaxExperts || k > kMaxSlots) return QG_ERR_UNSUPPORTED;
    if (tokens == 0) return QG_OK;
    if (!logits || !expert_ids || !expert_weights) return QG_ERR_INVALID_ARG;
    if (!aligned(logits, esize(dtype)) || !aligned(expert_ids, 4) || !aligned(expert_weights, 4)) return QG_ERR_INVALID_ARG;
    return finish(qg::route_topk(logits, dtype, ld, tokens, num_experts, k, renormalize, expert_ids, expert_weights, reinterpret_cast<cudaStream_t>(stream)));
}

size_t qmoe_tokens_workspace_bytes(int tokens, int k, int hidden, int inter) {
    if (tokens <= 0 || k <= 0 || hidden <= 0 || inter <= 0) return 0;
    return qg::moe_tokens_workspace_bytes(tokens, k, hidden, inter);
}

int qmoe_tokens_fused(const void *x, int x_dtype, const int32_t *expert_ids, const float *expert_weights, int tokens, int k,
                      int num_experts, const uint8_t *fc1_w, const uint16_t *fc1_scales, const uint16_t *fc1_zp,
                      const uint16_t *fc1_bias, const uint8_t *fc2_w, const uint16_t *fc2_scales, const uint16_t *fc2_zp,
                      const uint16_t *fc2_bias, int hidden, int inter, int bits, int block_size, int swiglu_interleaved,
                      void *y, int y_dtype, int *status_dev, void *workspace, size_t workspace_bytes, qg_stream_t stream) {
    (void)cudaGetLastError();
    if (!valid_dtype(x_dtype) || !valid_dtype(y_dtype) || tokens < 0 || k < 1 || num_experts < 1) return QG_ERR_INVALID_ARG;
    if (hidden <= 0 || inter <= 0 || (swiglu_interleaved != 0 && swiglu_interleaved != 1)) return QG_ERR_INVALID_ARG;
    if (x_dtype == QG_F32 || (bits != 2 && bits != 4 && bits != 8)) return QG_ERR_UNSUPPORTED;
    if (block_size != 32 && block_size != 64 && block_size != 128 && block_size != 256) return QG_ERR_UNSUPPORTED;
    if (hidden % block_size || inter % block_size) return QG_ERR_INVALID_ARG;
    if (k > kMaxSlots || num_experts > kMaxExperts || tokens > kMaxPairs / k || hidden > (1 << 20) || inter > (1 << 20)) return QG_ERR_UNSUPPORTED;
    if (tokens == 0) return QG_OK;
    if (!x || !expert_ids || !expert_weights || !fc1_w || !fc1_scales || !fc2_w || !fc2_scales || !y) return QG_ERR_INVALID_ARG;
    for (const void *p : {x, static_cast<const void *>(fc1_w), static_cast<const void *>(fc1_scales), static_cast<const void *>(fc1_zp), static_cast<const void *>(fc2_w),
                          static_cast<const void *>(fc2_scales), static_cast<const void *>(fc2_zp), static_cast<const void *>(y)})
        if (!aligned(p, 16)) return QG_ERR_INVALID_ARG;
    if (!aligned(expert_ids, 4) || !aligned(expert_weights, 4) || !aligned(status_dev, 4) || !aligned(fc1_bias, 2) || !aligned(fc2_bias, 2)) return QG_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < qg::moe_tokens_workspace_bytes(tokens, k, hidden, inter)) return QG_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned(workspace, 16)) return QG_ERR_INVALID_ARG;
    const qg::MoeTokens q{x, x_dtype, expert_ids, expert_weights, tokens, k, num_experts, fc1_w, fc1_scales, fc1_zp, fc1_bias, fc2_w, fc2_scales, fc2_zp,
                          fc2_bias, hidden, inter, bits, block_size, swiglu_interleaved, y, y_dtype, status_dev};
    return finish(qg::moe_tokens(q, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
