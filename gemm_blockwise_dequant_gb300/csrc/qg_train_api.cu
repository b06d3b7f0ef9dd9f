// qg_train_api.cu -- the C ABI of the adapter and fine-tuning entry points
// (include/qgemm.h): argument checks and dispatch.  Everything is refused or
// accepted on the host before anything is enqueued.
#include <climits>

#include "../../include/qgemm.h"
#include "qg_internal.h"

namespace {

bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool valid_dtype(int d) { return d == QG_F32 || d == QG_F16 || d == QG_BF16; }
int64_t esize(int d) { return d == QG_F32 ? 4 : 2; }

// as the GEMM entry points: larger sizes are not implemented (32-bit row and column indexes)
constexpr int kMaxRows = 1 << 20, kMaxN = 1 << 28, kMaxK = 1 << 24;
// Every CTA looks its rows up in the whole list of requests: more of them would take longer to find than to serve.
constexpr int kMaxSegments = 1 << 16, kMaxAdapters = 65535, kMaxRank = 128;

int finish(cudaError_t e) {
    if (e == cudaErrorNotSupported) return QG_ERR_UNSUPPORTED;
    return e == cudaSuccess ? QG_OK : QG_ERR_CUDA;
}

// What qg_lora_apply and qg_lora_grad check alike.
int check_lora(const int64_t *offs, const int32_t *ids, int S, int x_dtype, int w_dtype, const float *scaling, int na,
               int r, int T, int N, int K, const int *status) {
    if (!valid_dtype(x_dtype) || !valid_dtype(w_dtype)) return QG_ERR_INVALID_ARG;
    if (T < 0 || N < 0 || K <= 0 || S < 0 || na < 0 || r <= 0) return QG_ERR_INVALID_ARG;
    if (x_dtype != QG_F32 && w_dtype != x_dtype) return QG_ERR_UNSUPPORTED;
    if (r > kMaxRank || r % 8 || K % 8) return QG_ERR_UNSUPPORTED;
    if (T > kMaxRows || N > kMaxN || K > kMaxK || S > kMaxSegments || na > kMaxAdapters) return QG_ERR_UNSUPPORTED;
    if (!offs || !aligned(offs, 8) || (S > 0 && (!ids || !aligned(ids, 4)))) return QG_ERR_INVALID_ARG;
    if ((scaling && !aligned(scaling, 4)) || (status && !aligned(status, 4))) return QG_ERR_INVALID_ARG;
    return QG_OK;
}

int check_workspace(const void *ws, size_t have, size_t need) {
    if (need == 0) return QG_OK;
    if (!ws || have < need) return QG_ERR_WORKSPACE_TOO_SMALL;
    return aligned(ws, 16) ? QG_OK : QG_ERR_INVALID_ARG;
}

int dgrad_common(const void *dY, int dy_dtype, const uint8_t *W, const void *params, const uint16_t *zp, void *dX,
                 int dx_dtype, int M, int N, int K, int bits, int bs, void *ws, size_t ws_bytes, qg::GemmProblem &p,
                 qg_stream_t stream) {
    if (!valid_dtype(dy_dtype) || !valid_dtype(dx_dtype)) return QG_ERR_INVALID_ARG;
    if (M < 0 || N < 0 || K < 0) return QG_ERR_INVALID_ARG;
    if (bits != 2 && bits != 3 && bits != 4 && bits != 8) return QG_ERR_UNSUPPORTED;
    if (bs != 32 && bs != 64 && bs != 128 && bs != 256) return QG_ERR_UNSUPPORTED;
    if (K % bs) return QG_ERR_INVALID_ARG;
    if (M > kMaxRows || N > kMaxN || K > kMaxK) return QG_ERR_UNSUPPORTED;
    if (M == 0 || K == 0) return QG_OK;
    if (!dX || !aligned(dX, 16)) return QG_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (N == 0)
        return cudaMemsetAsync(dX, 0, static_cast<size_t>(M) * K * esize(dx_dtype), s) == cudaSuccess ? QG_OK : QG_ERR_CUDA;
    if (!dY || !W || !params) return QG_ERR_INVALID_ARG;
    if (!aligned(dY, 16) || !aligned(W, 16) || !aligned(params, 16) || (zp && !aligned(zp, 16))) return QG_ERR_INVALID_ARG;
    const int st = check_workspace(ws, ws_bytes, qg::dgrad_workspace_bytes(dy_dtype, M, N, K, bits));
    if (st != QG_OK) return st;
    p.A = dY;
    p.a_dtype = dy_dtype;
    p.W = W;
    p.Y = dX;
    p.y_dtype = dx_dtype;
    p.M = M;
    p.N = N;
    p.K = K;
    p.bits = bits;
    p.bs = bs;
    return finish(qg::dgrad(p, ws, s));
}

}  // namespace

extern "C" {

size_t qg_lora_apply_workspace_bytes(int rows, int num_segments, int rank, int N, int K) {
    if (rows <= 0 || num_segments < 0 || rank <= 0 || N <= 0 || K <= 0) return 0;
    return qg::lora_apply_workspace_bytes(rows, num_segments, rank, N, K);
}

int qg_lora_apply(const void *X, int x_dtype, int64_t ldx, const int64_t *seg_offsets, const int32_t *seg_adapter,
                  int num_segments, const void *A, const void *B, int w_dtype, const float *scaling, int num_adapters,
                  int rank, const void *Y_in, int y_in_dtype, int64_t ldy_in, void *Y, int y_dtype, int64_t ldy,
                  float *V_out, int rows, int N, int K, int *status_dev, void *workspace, size_t workspace_bytes,
                  qg_stream_t stream) {
    (void)cudaGetLastError();  // do not report an earlier, unrelated failure as ours
    int st = check_lora(seg_offsets, seg_adapter, num_segments, x_dtype, w_dtype, scaling, num_adapters, rank, rows, N, K,
                        status_dev);
    if (st != QG_OK) return st;
    if (!valid_dtype(y_dtype) || (Y_in && !valid_dtype(y_in_dtype))) return QG_ERR_INVALID_ARG;
    if (Y_in && y_in_dtype != QG_F32 && y_in_dtype != y_dtype) return QG_ERR_UNSUPPORTED;
    if (ldx < K || ldy < N || (Y_in && ldy_in < N)) return QG_ERR_INVALID_ARG;
    if (Y_in == Y && Y_in && (y_in_dtype != y_dtype || ldy_in != ldy)) return QG_ERR_INVALID_ARG;
    if (rows == 0 || N == 0 || num_segments == 0) return QG_OK;
    if (!X || !Y || (num_adapters > 0 && (!A || !B))) return QG_ERR_INVALID_ARG;
    if (!aligned(X, 16) || (ldx * esize(x_dtype)) % 16 || !aligned(A, 16) || !aligned(B, 16)) return QG_ERR_INVALID_ARG;
    if (!aligned(Y, esize(y_dtype)) || (Y_in && !aligned(Y_in, esize(y_in_dtype))) || !aligned(V_out, 16))
        return QG_ERR_INVALID_ARG;
    st = check_workspace(workspace, workspace_bytes, qg::lora_apply_workspace_bytes(rows, num_segments, rank, N, K));
    if (st != QG_OK) return st;
    qg::LoraApply q{};
    q.p = {seg_offsets, seg_adapter, num_segments, A, B, w_dtype, scaling, num_adapters, rank, rows, N, K, status_dev};
    q.X = X;
    q.x_dtype = x_dtype;
    q.ldx = ldx;
    q.Yin = Y_in;
    q.yin_dtype = y_in_dtype;
    q.ldyin = ldy_in;
    q.Y = Y;
    q.y_dtype = y_dtype;
    q.ldy = ldy;
    q.V = V_out;
    return finish(qg::lora_apply(q, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

size_t qg_lora_grad_workspace_bytes(int rows, int num_segments, int num_adapters, int rank, int N, int K) {
    if (rows <= 0 || num_segments < 0 || num_adapters < 0 || rank <= 0 || N < 0 || K <= 0) return 0;
    return qg::lora_grad_workspace_bytes(rows, num_segments, num_adapters, rank, N, K);
}

int qg_lora_grad(const void *dY, int x_dtype, int64_t lddy, const void *X, int64_t ldx, const float *V,
                 const int64_t *seg_offsets, const int32_t *seg_adapter, int num_segments, const void *A,
                 const void *B, int w_dtype, const float *scaling, int num_adapters, int rank, const void *dX_in,
                 void *dX, int64_t lddx, void *dA, void *dB, int g_dtype, int accumulate, int rows, int N, int K,
                 int *status_dev, void *workspace, size_t workspace_bytes, qg_stream_t stream) {
    (void)cudaGetLastError();
    int st = check_lora(seg_offsets, seg_adapter, num_segments, x_dtype, w_dtype, scaling, num_adapters, rank, rows, N, K,
                        status_dev);
    if (st != QG_OK) return st;
    if (!valid_dtype(g_dtype) || (accumulate != 0 && accumulate != 1)) return QG_ERR_INVALID_ARG;
    if (g_dtype != w_dtype && g_dtype != QG_F32) return QG_ERR_UNSUPPORTED;
    if (lddy < N || ldx < K || (dX && lddx < K) || (dX_in && !dX)) return QG_ERR_INVALID_ARG;
    if (num_adapters > 0 && (!A || !dA || (N > 0 && (!B || !dB)))) return QG_ERR_INVALID_ARG;
    if (!aligned(A, 16) || !aligned(B, 16) || !aligned(dA, 16) || !aligned(dB, 16)) return QG_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (rows == 0 || num_segments == 0) {  // no row of any adapter: the gradients are zeros
        if (accumulate || num_adapters == 0) return QG_OK;
        const size_t per = static_cast<size_t>(num_adapters) * rank * esize(g_dtype);
        if (cudaMemsetAsync(dA, 0, per * K, s) != cudaSuccess) return QG_ERR_CUDA;
        if (N > 0 && cudaMemsetAsync(dB, 0, per * N, s) != cudaSuccess) return QG_ERR_CUDA;
        return QG_OK;
    }
    // N == 0 goes on: its sums are empty, and dX is dX_in
    if ((N > 0 && !dY) || !X || !V || !aligned(dY, esize(x_dtype)) || !aligned(X, 16) || !aligned(V, 16)) return QG_ERR_INVALID_ARG;
    if ((ldx * esize(x_dtype)) % 16 || (dX && (lddx * esize(x_dtype)) % 16)) return QG_ERR_INVALID_ARG;
    if (!aligned(dX, 16) || !aligned(dX_in, 16)) return QG_ERR_INVALID_ARG;
    st = check_workspace(workspace, workspace_bytes,
                         qg::lora_grad_workspace_bytes(rows, num_segments, num_adapters, rank, N, K));
    if (st != QG_OK) return st;
    qg::LoraGrad q{};
    q.p = {seg_offsets, seg_adapter, num_segments, A, B, w_dtype, scaling, num_adapters, rank, rows, N, K, status_dev};
    q.dY = dY;
    q.X = X;
    q.x_dtype = x_dtype;
    q.lddy = lddy;
    q.ldx = ldx;
    q.V = V;
    q.dXin = dX_in;
    q.dX = dX;
    q.lddx = lddx;
    q.dA = dA;
    q.dB = dB;
    q.g_dtype = g_dtype;
    q.accumulate = accumulate;
    return finish(qg::lora_grad(q, workspace, s));
}

size_t qgemm_dgrad_workspace_bytes(int dy_dtype, int M, int N, int K, int bits) {
    if (M <= 0 || N <= 0 || K <= 0 || !valid_dtype(dy_dtype)) return 0;
    return qg::dgrad_workspace_bytes(dy_dtype, M, N, K, bits);
}

int qgemm_nbits_dgrad(const void *dY, int dy_dtype, const uint8_t *W, const uint16_t *scales_f16,
                      const uint16_t *zero_points_f16, void *dX, int dx_dtype, int M, int N, int K, int bits,
                      int block_size, void *workspace, size_t workspace_bytes, qg_stream_t stream) {
    (void)cudaGetLastError();
    qg::GemmProblem p{};
    p.kind = qg::WK_NBITS;
    p.scales = scales_f16;
    p.zp = zero_points_f16;
    p.zp_mode = zero_points_f16 ? qg::ZP_TENSOR : qg::ZP_NONE;
    if (bits >= 1 && bits <= 8) p.uniform_zp = static_cast<float>(1 << (bits - 1));
    return dgrad_common(dY, dy_dtype, W, scales_f16, zero_points_f16, dX, dx_dtype, M, N, K, bits, block_size, workspace,
                        workspace_bytes, p, stream);
}

int qgemm_nbits_uniform_zp_dgrad(const void *dY, int dy_dtype, const uint8_t *W, const uint16_t *scales_f16,
                                 float uniform_zp, void *dX, int dx_dtype, int M, int N, int K, int bits,
                                 int block_size, void *workspace, size_t workspace_bytes, qg_stream_t stream) {
    (void)cudaGetLastError();
    if (!(uniform_zp >= -65504.f && uniform_zp <= 65504.f)) return QG_ERR_INVALID_ARG;  // not a finite fp16 value
    qg::GemmProblem p{};
    p.kind = qg::WK_NBITS;
    p.scales = scales_f16;
    p.zp_mode = qg::ZP_UNIFORM;
    p.uniform_zp = uniform_zp;
    return dgrad_common(dY, dy_dtype, W, scales_f16, nullptr, dX, dx_dtype, M, N, K, bits, block_size, workspace,
                        workspace_bytes, p, stream);
}

int qgemm_codebook4_dgrad(const void *dY, int dy_dtype, const uint8_t *W, const float *codebook16,
                          const float *absmax, void *dX, int dx_dtype, int M, int N, int K, int block_size,
                          void *workspace, size_t workspace_bytes, qg_stream_t stream) {
    (void)cudaGetLastError();
    if (M > 0 && N > 0 && K > 0 && (!codebook16 || !aligned(codebook16, 4))) return QG_ERR_INVALID_ARG;
    qg::GemmProblem p{};
    p.kind = qg::WK_CODEBOOK;
    p.codebook = codebook16;
    p.absmax = absmax;
    return dgrad_common(dY, dy_dtype, W, absmax, nullptr, dX, dx_dtype, M, N, K, 4, block_size, workspace,
                        workspace_bytes, p, stream);
}

int qg_grad_list_init(qg_grad_tensor *tensors_host, int count, int64_t *chunks) {
    if (count < 0 || !chunks || (count > 0 && !tensors_host)) return QG_ERR_INVALID_ARG;
    int64_t at = 0;
    for (int i = 0; i < count; ++i) {
        qg_grad_tensor &t = tensors_host[i];
        if (t.numel < 0 || !valid_dtype(t.dtype)) return QG_ERR_INVALID_ARG;
        if (!t.out) t.out = const_cast<void *>(t.grad);
        if (t.numel > 0 && !t.grad) return QG_ERR_INVALID_ARG;
        if (!aligned(t.grad, esize(t.dtype)) || !aligned(t.out, esize(t.dtype))) return QG_ERR_INVALID_ARG;
        t.first_chunk = at;
        t.reserved = 0;
        at += qg::clip_chunks(t.grad, t.numel, static_cast<int>(esize(t.dtype)));
        if (at > INT_MAX) return QG_ERR_UNSUPPORTED;
    }
    *chunks = at;
    return QG_OK;
}

size_t qg_clip_grad_norm_workspace_bytes(int64_t chunks) { return qg::clip_workspace_bytes(chunks < 0 ? 0 : chunks); }

int qg_clip_grad_norm(const qg_grad_tensor *tensors_dev, int count, int64_t chunks, float max_norm, float eps,
                      float *norm_dev, void *workspace, size_t workspace_bytes, qg_stream_t stream) {
    (void)cudaGetLastError();
    if (count < 0 || chunks < 0 || chunks > INT_MAX || (count == 0 && chunks > 0)) return QG_ERR_INVALID_ARG;
    if (!(max_norm >= 0.f) || !(eps >= 0.f)) return QG_ERR_INVALID_ARG;  // NaN too
    if (!norm_dev || !aligned(norm_dev, 4) || (count > 0 && (!tensors_dev || !aligned(tensors_dev, 8)))) return QG_ERR_INVALID_ARG;
    const int st = check_workspace(workspace, workspace_bytes, qg::clip_workspace_bytes(chunks));
    if (st != QG_OK) return st;
    return finish(qg::clip_grad_norm(tensors_dev, count, chunks, max_norm, eps, norm_dev, workspace,
                                     reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
