// qg_token_api.cu -- the C ABI of the entry points around a few tokens' logits and experts (include/qgemm.h): argument
// checks and dispatch.  Everything is refused or accepted on the host before anything is enqueued.
#include <cmath>

#include "../../include/qgemm.h"
#include "qg_internal.h"

namespace {

bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool valid_dtype(int d) { return d == QG_F32 || d == QG_F16 || d == QG_BF16; }
size_t esize(int d) { return d == QG_F32 ? 4 : 2; }

constexpr int kMaxRows = 1 << 20, kMaxVocab = 1 << 28, kMaxTop = 64;

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
    if (top_k > kMaxTop) return QG_ERR_UNSUPPORTED;
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

}  // extern "C"
