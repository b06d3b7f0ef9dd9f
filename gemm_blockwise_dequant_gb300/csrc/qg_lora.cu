// qg_lora.cu -- low-rank adapters of many requests beside a shared projection:
// planning of the forward pass (apply) and the backward pass (grad).
#include <algorithm>

#include "qg_lora_rows.cuh"
#include "qg_lora_tc.h"
#include "qg_lora_wgrad.cuh"

namespace qg {

template <> cudaError_t launch_rows<kBF16, kBF16>(const RowsArgs &, bool, const RowsPlan &, cudaStream_t);
template <> cudaError_t launch_rows<kF16, kF16>(const RowsArgs &, bool, const RowsPlan &, cudaStream_t);
template <> cudaError_t launch_rows<kF32, kF32>(const RowsArgs &, bool, const RowsPlan &, cudaStream_t);
template <> cudaError_t launch_rows<kF32, kF16>(const RowsArgs &, bool, const RowsPlan &, cudaStream_t);
template <> cudaError_t launch_rows<kF32, kBF16>(const RowsArgs &, bool, const RowsPlan &, cudaStream_t);
cudaError_t launch_wgrad(const WgradArgs &q, int x_dtype, cudaStream_t s);

namespace {

// Rows of 16-bit activations from which on the tensor cores (tcgen05) make dA and
// dB faster: 24.6 against 26.1 us at 128 x (4096, 1024), rank 16, 38 against 59 at
// rank 64.
constexpr int kTcGradRows = 128;

// The products over rows in two launches, the first one on the tensor cores,
// instead of one: 38.0 against 40.5 us at 2048 x (4096 -> 14336), rank 16, 35.7
// against 36.9 at 4096 x (5120 -> 5120), 32.7 against 36.8 at half the rows and rank
// 64; but 23.8 against 22.1 there at rank 16, and 20.2 against 18.1 at 4096 x (4096
// -> 1024).
bool two_launches(int T, int N, int K, int r) {
    return T >= 1024 && static_cast<double>(T) * (static_cast<double>(N) + K) * (r + 16) >= 1.2e9;
}

size_t esize(int d) { return d == kF32 ? 4 : 2; }

bool rows_at(unsigned bytes, const void *p, int64_t ld, int dtype) {  // all rows at such boundaries
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && (ld * static_cast<int64_t>(esize(dtype))) % bytes == 0;
}
bool rows16(const void *p, int64_t ld, int dtype) { return rows_at(16, p, ld, dtype); }

// The cluster of a tile is as wide as leaves all CTAs resident at once, two an SM,
// while each has at least 256 values of a row to contract: 64 requests of one row
// at 4096 -> 14336, rank 16, take 37.2 / 23.8 / 15.9 / 20.6 us with 1 / 2 / 4 / 8
// CTAs a tile, one row 36 / 21.6 / 13.9 / 9.9 / 8.2 (16).  Clusters of 16 are few
// at a time (256 rows: 15.2 us with them, 9.3 with 8).  In the backward pass of
// 16-bit rows clusters of 8 pay only while a CTA has an SM to itself: 512 rows with
// dA and dB take 24.7 us with 4 and 27.9 with 8 (fp32: 51.0 and 43.2; forward 11.3
// and 10.5).
RowsPlan make_plan(int T, int S, int c1, bool bwd16) {
    RowsPlan plan{};
    const int sms = device_info().sm_count;
    plan.tiles = (T + kRowsTile - 1) / kRowsTile + S;  // the most that any offsets can need
    const int real = std::max(T / kRowsTile, std::min(S, T));
    plan.cs = 1;
    while (plan.cs < 16 && real * plan.cs * 2 <= (plan.cs < (bwd16 ? 4 : 8) ? 2 * sms : sms) && c1 >= 512 * plan.cs) plan.cs *= 2;
    return plan;
}

// The second product alone: 64-row tiles, whose columns as many CTAs share as
// keep two on every SM.
RowsPlan expand_plan(int T, int S, int c2) {
    RowsPlan plan{};
    plan.tiles = (T + 63) / 64 + S;
    plan.cs = 1;
    while (plan.cs < 64 && (T / 64) * plan.cs * 2 <= 2 * device_info().sm_count && c2 >= 512 * plan.cs) plan.cs *= 2;
    return plan;
}

// 16-bit activations at 16-byte boundaries, not cut into small requests, and adapters
// with outputs to read (copies of an empty tensor cannot be set up; the row kernel needs none).
bool tensor_cores(const LoraProblem &p, int x_dtype, bool aligned) {
    return x_dtype != kF32 && aligned && p.T / 128 >= p.S && p.na > 0 && p.N > 0 && lora_tc_available();
}

// CTAs that share a tile's contraction: enough for two an SM, of eight steps or more.
int shrink_splits(int T, int S, int c1) {
    const int tiles = std::max(T / 128, std::min(S, T));
    int cs = 1;
    while (cs < 8 && tiles * cs * 2 <= 2 * device_info().sm_count && c1 >= 1024 * cs) cs *= 2;
    return cs;
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

cudaError_t rows(const RowsArgs &args, int x_dtype, bool bwd, cudaStream_t s) {
    RowsArgs q = args;
    const RowsPlan plan = q.given ? expand_plan(q.p.T, q.p.S, q.c2) : make_plan(q.p.T, q.p.S, std::max(q.c1, q.c2), bwd && x_dtype != kF32);
    q.cs = plan.cs;
    if (x_dtype == kBF16) return launch_rows<kBF16, kBF16>(q, bwd, plan, s);
    if (x_dtype == kF16) return launch_rows<kF16, kF16>(q, bwd, plan, s);
    if (q.p.w_dtype == kF32) return launch_rows<kF32, kF32>(q, bwd, plan, s);
    return q.p.w_dtype == kF16 ? launch_rows<kF32, kF16>(q, bwd, plan, s) : launch_rows<kF32, kBF16>(q, bwd, plan, s);
}

}  // namespace

// V between the two products of many rows
size_t lora_apply_workspace_bytes(int T, int, int r, int N, int K) { return two_launches(T, N, K, r) ? static_cast<size_t>(T) * r * 4 : 0; }

cudaError_t lora_apply(const LoraApply &a, void *ws, cudaStream_t s) {
    RowsArgs q{};
    q.p = a.p;
    q.in = a.X;
    q.ld_in = a.ldx;
    q.c1 = a.p.K;
    q.c2 = a.p.N;
    q.w1 = a.p.A;
    q.w2 = a.p.B;
    q.base = a.Yin;
    q.base_dtype = a.yin_dtype;
    q.ld_base = a.ldyin;
    q.out = a.Y;
    q.out_dtype = a.y_dtype;
    q.ld_out = a.ldy;
    q.sums = a.V;
    q.in_vec = rows16(a.X, a.ldx, a.x_dtype);
    q.in_words = rows_at(4, a.X, a.ldx, a.x_dtype);
    q.out_vec = rows16(a.Y, a.ldy, a.y_dtype) && (!a.Yin || rows16(a.Yin, a.ldyin, a.yin_dtype));
    if (two_launches(a.p.T, a.p.N, a.p.K, a.p.r) && tensor_cores(a.p, a.x_dtype, q.in_vec)) {
        ShrinkTc t{};
        t.p = a.p;
        t.sums = a.V ? a.V : static_cast<float *>(ws);
        t.bf16 = a.x_dtype == kBF16;
        t.cs = shrink_splits(a.p.T, a.p.S, a.p.K);
        const cudaError_t e = launch_shrink_tc(t, a.X, a.ldx, a.p.A, s);
        if (e != cudaSuccess) return e;
        q.given = t.sums;
        q.sums = nullptr;
    }
    const cudaError_t e = rows(q, a.x_dtype, false, s);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// CTAs, or tiles, that write down their rows' largest values: of shrink (clusters of up to 8) or of the row kernel.
static int grad_parts(int T, int S) { return std::max(shrink_tc_tiles(T, S) * 8, (T + kRowsTile - 1) / kRowsTile + S); }

// G, the rows' gradients inside the adapter; for the tensor cores also the largest
// values and the adapters of the tiles, and the 16-bit terms of G and V
size_t lora_grad_workspace_bytes(int T, int S, int, int r, int, int) {
    const size_t sums = align256(static_cast<size_t>(T) * r * 4);
    return T < kTcGradRows ? sums : sums + align256(static_cast<size_t>(grad_parts(T, S)) * 12) + wgrad_tc_terms_bytes(T, r);
}

cudaError_t lora_grad(const LoraGrad &a, void *ws, cudaStream_t s) {
    RowsArgs q{};
    q.p = a.p;
    q.in = a.dY;
    q.ld_in = a.lddy;
    q.c1 = a.p.N;
    q.c2 = a.p.K;
    q.w1 = a.p.B;
    q.w2 = a.p.A;
    q.base = a.dXin;
    q.base_dtype = a.x_dtype;
    q.ld_base = a.lddx;
    q.out = a.dX;
    q.out_dtype = a.x_dtype;
    q.ld_out = a.lddx;
    q.sums = static_cast<float *>(ws);
    q.in_vec = rows16(a.dY, a.lddy, a.x_dtype);
    q.in_words = rows_at(4, a.dY, a.lddy, a.x_dtype);
    q.out_vec = 1;
    const bool tc = a.p.T >= kTcGradRows && tensor_cores(a.p, a.x_dtype, q.in_vec),
               two = tc && two_launches(a.p.T, a.p.N, a.p.K, a.p.r);
    int parts = 0;
    int *tile_adapter = nullptr;
    float *tile_max = nullptr, *G = q.sums;
    uint16_t *terms = nullptr;
    const bool bf16 = a.x_dtype == kBF16;
    if (tc) {
        const int cs = two ? shrink_splits(a.p.T, a.p.S, a.p.N) : 1;
        parts = two ? shrink_tc_tiles(a.p.T, a.p.S) * cs : (a.p.T + kRowsTile - 1) / kRowsTile + a.p.S;
        tile_adapter = reinterpret_cast<int *>(static_cast<char *>(ws) + align256(static_cast<size_t>(a.p.T) * a.p.r * 4));
        tile_max = reinterpret_cast<float *>(tile_adapter + parts);
        terms = reinterpret_cast<uint16_t *>(reinterpret_cast<char *>(tile_adapter) + align256(static_cast<size_t>(grad_parts(a.p.T, a.p.S)) * 12));
        q.V = a.V;
        if (bf16) {
            q.terms = {terms, wgrad_tc_terms(true, a.g_dtype), static_cast<size_t>(a.p.T) * a.p.r};
        } else {
            q.tile_adapter = tile_adapter;
            q.tile_max = tile_max;
        }
    }
    cudaError_t e = cudaSuccess;
    if (two) {
        ShrinkTc t{};
        t.p = a.p;
        t.sums = G;
        t.V = a.V;
        t.bwd = 1;
        t.bf16 = bf16;
        t.cs = shrink_splits(a.p.T, a.p.S, a.p.N);
        t.tile_adapter = q.tile_adapter;
        t.tile_max = q.tile_max;
        t.terms = q.terms;
        e = launch_shrink_tc(t, a.dY, a.lddy, a.p.B, s);
        q.given = G;
        q.sums = nullptr;
    }
    if (e == cudaSuccess && (!two || a.dX)) e = rows(q, a.x_dtype, true, s);
    if (e != cudaSuccess) return e;
    if (a.p.na == 0) return cudaGetLastError();
    if (tc) {
        WgradTc w{};
        w.p = a.p;
        w.out[0] = a.dA;
        w.out[1] = a.dB;
        w.g_dtype = a.g_dtype;
        w.accumulate = a.accumulate;
        w.tile_max = tile_max;
        w.tile_adapter = tile_adapter;
        w.parts = parts;
        e = launch_wgrad_tc(w, G, a.V, terms, a.X, a.ldx, a.dY, a.lddy, bf16, s);
        return e != cudaSuccess ? e : cudaGetLastError();
    }
    WgradArgs w{};
    w.p = a.p;
    w.wide[0] = a.X;
    w.wide[1] = a.dY;
    w.ld[0] = a.ldx;
    w.ld[1] = a.lddy;
    w.cols[0] = a.p.K;
    w.cols[1] = a.p.N;
    w.vec[0] = 1;
    w.vec[1] = q.in_vec;
    w.words[0] = 1;
    w.words[1] = q.in_words;
    w.skinny[0] = static_cast<const float *>(ws);
    w.skinny[1] = a.V;
    w.out[0] = a.dA;
    w.out[1] = a.dB;
    w.g_dtype = a.g_dtype;
    w.accumulate = a.accumulate;
    e = launch_wgrad(w, a.x_dtype, s);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace qg
