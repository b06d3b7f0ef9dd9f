// qg_lora_wgrad.cuh -- the adapters' own gradients, dA and dB in one launch:
//
//   dA[a][j][k] = sum_t G[t][j] X[t][k],   dB[a][n][j] = scaling[a] sum_t V[t][j] dY[t][n]
//
// over the rows t of adapter a: a wide matrix (X or dY), read once, against a
// skinny one (G or V).  A CTA owns 8 warps' columns of one adapter; a lane takes
// 16 contiguous bytes of four rows, which are the column operands of as many
// MMAs as the bytes hold values, and the skinny rows come through shared memory,
// split in two operand terms once per CTA.  A cluster shares the rows of the
// columns; its sums meet through distributed shared memory in rank order.
//
// bf16 gradients of bf16 activations use bf16 MMAs (the skinny factor keeps 16
// bits); everything else uses TF32 (22 bits): fp16's range would have to be
// scaled per row, which a sum over rows cannot undo.
#pragma once

#include "qg_lora_common.cuh"

namespace qg {

struct WgradArgs {
    LoraProblem p;
    const void *wide[2];     // X, dY
    int64_t ld[2];
    int cols[2], tiles[2];   // K, N and their column tiles
    int vec[2];              // rows at 16-byte boundaries
    int words[2];            // at 4-byte boundaries
    const float *skinny[2];  // G, V
    void *out[2];            // dA, dB
    int g_dtype, accumulate, cs;
};

constexpr int kWgChunk = 64;  // rows staged at a time

// XT: type of the wide matrix; NATIVE: bf16 MMAs; MJ: 16-row groups of the rank
template <int XT, bool NATIVE, int MJ>
struct WgradKernel {
    static constexpr int CPL = NATIVE && MJ == 1 ? 8 : 4;            // columns of a lane
    static constexpr int WCOLS = 8 * CPL, COLS = 8 * WCOLS;      // of a warp, of a CTA
    static constexpr int RJ = 16 * MJ;
    static constexpr int QBYTES = RJ * kWgChunk * (NATIVE ? 2 : 4);    // one term of the staged factor, [j][t]
    static constexpr int OS = COLS + 4;                                // row stride of the sums
    static constexpr int PB = CPL * (XT == kF32 ? 4 : 2);              // bytes of a lane's piece of a row: 16 or 8
    static constexpr int STAGES = XT == kF32 && MJ == 1 ? 2 : 3;       // two CTAs an SM at rank 16
    static constexpr int WIDE_BYTES = 8 * STAGES * 8 * 32 * PB;        // the lanes' queues: 8 rows a step
    static constexpr int SMEM = (4 * QBYTES + WIDE_BYTES > RJ * OS * 4) ? 4 * QBYTES + WIDE_BYTES : RJ * OS * 4;
    static constexpr int QPT = kWgChunk * RJ / 256;                    // staged values of a thread

    // Place of the staged value (j, t): the row's four-value pieces are permuted by
    // j, so that neither the lanes that write 16 values j of one t nor those that
    // read pieces of 4 to 8 rows j meet in a bank.
    static __device__ __forceinline__ int place(int j, int t) {
        const int f = NATIVE ? ((j & 3) << 2) | ((j >> 2) & 3) : ((j & 1) << 2) | ((j >> 1) & 3);
        return j * kWgChunk + (((t >> 2) ^ f) << 2) + (t & 3);
    }

    // Walks the 64-row chunks of the adapter's requests.
    struct Walk {
        int s, mask_base;
        unsigned mask;
        int64_t t, end;
        int left;  // chunks until the next one of this CTA
    };
    static __device__ __forceinline__ bool advance(const LoraProblem &p, int a, int cs, Walk &w, int &t0, int &rows) {
        for (;;) {
            if (w.t < w.end) {
                const int64_t n = (w.end - w.t + kWgChunk - 1) / kWgChunk;  // chunks left in this request
                if (w.left < n) {
                    const int64_t at = w.t + static_cast<int64_t>(w.left) * kWgChunk;
                    t0 = static_cast<int>(at);
                    rows = static_cast<int>(w.end - at < kWgChunk ? w.end - at : kWgChunk);
                    w.t = at + kWgChunk;
                    w.left = cs - 1;
                    return true;
                }
                w.left -= static_cast<int>(n);
                w.t = w.end;
            }
            while (!w.mask) {
                if (w.s >= p.S) return false;
                const int i = w.s + (threadIdx.x & 31);
                w.mask = __ballot_sync(0xffffffffu, i < p.S && __ldg(p.ids + (i < p.S ? i : 0)) == a);
                w.mask_base = w.s;
                w.s += 32;
            }
            const int seg = w.mask_base + __ffs(w.mask) - 1;
            w.mask &= w.mask - 1;
            w.t = __ldg(p.offs + seg);
            w.end = __ldg(p.offs + seg + 1);
        }
    }

    // Puts CPL values of a row into the lane's queue, zeros outside.
    static __device__ __forceinline__ void queue_wide(const WgradArgs &q, int which, unsigned char *dst, int t, bool in, int col) {
        const size_t at = static_cast<size_t>(t) * q.ld[which] + col;
        const int cols = q.cols[which];
        if (!in || col >= cols || (q.vec[which] && col + CPL <= cols)) {
            in = in && col < cols;
            queue_copy<PB>(dst, static_cast<const char *>(q.wide[which]) + (in ? at * (XT == kF32 ? 4 : 2) : 0), in);
            return;
        }
        if (q.words[which] && (XT == kF32 || col + CPL <= cols || !(cols & 1))) {  // no word holds a value from past the end
            constexpr int VW = XT == kF32 ? 1 : 2;
#pragma unroll
            for (int i = 0; i < CPL; i += VW) {
                const bool win = col + i < cols;
                queue_copy<4>(dst + i * (4 / VW), static_cast<const char *>(q.wide[which]) + (win ? (at + i) * (4 / VW) : 0), win);
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < CPL; ++i) {
            if constexpr (XT == kF32) reinterpret_cast<uint32_t *>(dst)[i] = col + i < cols ? __ldg(static_cast<const unsigned int *>(q.wide[which]) + at + i) : 0u;
            else reinterpret_cast<uint16_t *>(dst)[i] = col + i < cols ? __ldg(static_cast<const unsigned short *>(q.wide[which]) + at + i) : uint16_t(0);
        }
    }

    static __device__ void run(const WgradArgs &q) {
        extern __shared__ __align__(16) unsigned char sm[];
        constexpr int W = XT == kF32 ? 4 : CPL / 2;
        const LoraProblem &p = q.p;
        const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
        const int rank = blockIdx.x % q.cs;
        int tile = blockIdx.x / q.cs;
        const int which = tile >= q.tiles[0];
        if (which) tile -= q.tiles[0];
        const int a = blockIdx.y, j0 = blockIdx.z * RJ, rj = min(RJ, p.r - j0);
        const int col0 = tile * COLS, col = col0 + warp * WCOLS + g * CPL;
        const float *skinny = q.skinny[which];
        pdl_launch_dependents();
        pdl_wait();
        int bad = 0;
        for (int s = tid; s < p.S; s += 256) {
            const int64_t lo = __ldg(p.offs + s), hi = __ldg(p.offs + s + 1);
            bad |= hi < lo || lo < 0 || hi > p.T || (s == 0 && lo != 0);
        }
        if (__syncthreads_or(bad)) return;  // the whole cluster

        // The MMAs add into `acc` with truncation; a chunk's sums are then added to
        // `total` with rounding, so the error does not grow with the rows.
        float acc[MJ][CPL][4], total[MJ][CPL][4] = {};
        float stage[QPT];
        auto fetch = [&](int t0, int rows) {
#pragma unroll
            for (int i = 0; i < QPT; ++i) {
                const int e = tid + i * 256, t = e / RJ, j = e % RJ;
                stage[i] = t < rows && j < rj ? __ldg(skinny + static_cast<size_t>(t0 + t) * p.r + j0 + j) : 0.f;
            }
        };
        auto put = [&](int b) {
            unsigned char *hi = sm + 2 * b * QBYTES, *lo = hi + QBYTES;
#pragma unroll
            for (int i = 0; i < QPT; ++i) {
                const int e = tid + i * 256, at = place(e % RJ, e / RJ);
                if constexpr (NATIVE) {
                    uint16_t h, l;
                    split16<kBF16>(stage[i], h, l);
                    reinterpret_cast<uint16_t *>(hi)[at] = h;
                    reinterpret_cast<uint16_t *>(lo)[at] = l;
                } else {
                    split_tf32(stage[i], reinterpret_cast<uint32_t *>(hi)[at], reinterpret_cast<uint32_t *>(lo)[at]);
                }
            }
        };
        // Two walks over the same 32-row steps: one loads, STAGES - 1 steps ahead of the one that multiplies.
        Walk w{0, 0, 0u, 0, 0, rank}, wl = w;
        unsigned char *queue = sm + 4 * QBYTES + (warp * STAGES * 8 * 32 + lane) * PB;
        int lt = 0, lrows = 0, lst = kWgChunk;
        bool lmore = true;
        auto ahead = [&](int slot) {
            if (lmore && (lst >= kWgChunk || lst >= lrows)) {
                lmore = advance(p, a, q.cs, wl, lt, lrows);
                lst = 0;
            }
            if (lmore) {
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int t = lst + s * 16 + c * 4 + e;
                        queue_wide(q, which, queue + (slot * 8 + s * 4 + e) * 32 * PB, lt + t, t < lrows, col);
                    }
                lst += 32;
            }
            queue_commit();
        };
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i) ahead(i);
        int slot = 0, t0 = 0, rows = 0;
        bool more = advance(p, a, q.cs, w, t0, rows);
        if (more) fetch(t0, rows);
        for (int b = 0; more; b ^= 1) {
            put(b);
            __syncthreads();
            const int cr = rows;
            more = advance(p, a, q.cs, w, t0, rows);
            if (more) fetch(t0, rows);
            const unsigned char *hi = sm + 2 * b * QBYTES, *lo = hi + QBYTES;
#pragma unroll
            for (int m = 0; m < MJ; ++m)
#pragma unroll
                for (int i = 0; i < CPL; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[m][i][e] = 0.f;
#pragma unroll 1
            for (int st = 0; st < kWgChunk && st < cr; st += 32) {
                ahead(slot == 0 ? STAGES - 1 : slot - 1);
                queue_wait<STAGES - 1>();
                uint32_t x[2][4][W];
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const unsigned char *from = queue + (slot * 8 + s * 4 + e) * 32 * PB;
                        if constexpr (W == 4) {
                            const uint4 v = *reinterpret_cast<const uint4 *>(from);
                            x[s][e][0] = v.x, x[s][e][1] = v.y, x[s][e][2] = v.z, x[s][e][3] = v.w;
                        } else {
                            const uint2 v = *reinterpret_cast<const uint2 *>(from);
                            x[s][e][0] = v.x, x[s][e][1] = v.y;
                        }
                    }
                slot = slot == STAGES - 1 ? 0 : slot + 1;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const int tt = st + s * 16 + c * 4;
                    if constexpr (NATIVE) {
                        uint2 fh[MJ][2], fl[MJ][2];
#pragma unroll
                        for (int m = 0; m < MJ; ++m)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int at = place(m * 16 + h * 8 + g, tt);
                                fh[m][h] = *reinterpret_cast<const uint2 *>(reinterpret_cast<const uint16_t *>(hi) + at);
                                fl[m][h] = *reinterpret_cast<const uint2 *>(reinterpret_cast<const uint16_t *>(lo) + at);
                            }
#pragma unroll
                        for (int i = 0; i < CPL; ++i) {
                            const uint32_t sel = (i & 1) ? 0x7632u : 0x5410u;
                            const uint32_t b0 = __byte_perm(x[s][0][i >> 1], x[s][1][i >> 1], sel);
                            const uint32_t b1 = __byte_perm(x[s][2][i >> 1], x[s][3][i >> 1], sel);
#pragma unroll
                            for (int m = 0; m < MJ; ++m) {
                                mma16<kBF16>(acc[m][i], fl[m][0].x, fl[m][1].x, fl[m][0].y, fl[m][1].y, b0, b1);
                                mma16<kBF16>(acc[m][i], fh[m][0].x, fh[m][1].x, fh[m][0].y, fh[m][1].y, b0, b1);
                            }
                        }
                    } else {
                        // two columns' operands, split once, against every row group of the rank
#pragma unroll
                        for (int i0 = 0; i0 < CPL; i0 += 2) {
                            uint32_t v[2][4], vl[2][4];
#pragma unroll
                            for (int i = 0; i < 2; ++i)
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    if constexpr (XT == kF32) {
                                        split_tf32(__uint_as_float(x[s][e][i0 + i]), v[i][e], vl[i][e]);
                                    } else {
                                        const uint32_t z = x[s][e][i0 >> 1];
                                        v[i][e] = __float_as_uint(to_float<XT>(static_cast<uint16_t>(i ? z >> 16 : z & 0xFFFFu)));
                                    }
                                }
#pragma unroll
                            for (int m = 0; m < MJ; ++m) {
                                uint4 fh[2], fl[2];
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    const int at = place(m * 16 + h * 8 + g, tt);
                                    fh[h] = *reinterpret_cast<const uint4 *>(reinterpret_cast<const uint32_t *>(hi) + at);
                                    fl[h] = *reinterpret_cast<const uint4 *>(reinterpret_cast<const uint32_t *>(lo) + at);
                                }
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    float (&d)[4] = acc[m][i0 + i];
                                    if constexpr (XT == kF32) {
                                        mma8(d, fh[0].x, fh[1].x, fh[0].y, fh[1].y, vl[i][0], vl[i][1]);
                                        mma8(d, fh[0].z, fh[1].z, fh[0].w, fh[1].w, vl[i][2], vl[i][3]);
                                    }
                                    mma8(d, fl[0].x, fl[1].x, fl[0].y, fl[1].y, v[i][0], v[i][1]);
                                    mma8(d, fl[0].z, fl[1].z, fl[0].w, fl[1].w, v[i][2], v[i][3]);
                                    mma8(d, fh[0].x, fh[1].x, fh[0].y, fh[1].y, v[i][0], v[i][1]);
                                    mma8(d, fh[0].z, fh[1].z, fh[0].w, fh[1].w, v[i][2], v[i][3]);
                                }
                            }
                        }
                    }
                }
            }
#pragma unroll
            for (int m = 0; m < MJ; ++m)
#pragma unroll
                for (int i = 0; i < CPL; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) total[m][i][e] += acc[m][i][e];
        }
        // ------------------------------------------------------------------ sums of the cluster, and out
        queue_wait<0>();
        __syncthreads();
        float *sums = reinterpret_cast<float *>(sm);
#pragma unroll
        for (int m = 0; m < MJ; ++m)
#pragma unroll
            for (int i = 0; i < CPL; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    sums[(m * 16 + (e >> 1) * 8 + g) * OS + warp * WCOLS + (2 * c + (e & 1)) * CPL + i] = total[m][i][e];
        __syncthreads();
        if (q.cs > 1) {
            cluster_arrive();
            cluster_wait();
        }
        const int ncol = min(COLS, q.cols[which] - col0), width = COLS / q.cs;
        const float scale = which && p.scaling ? __ldg(p.scaling + a) : 1.f;
        for (int e = tid; e < rj * width; e += 256) {
            const int j = which ? e % rj : e / width, cc = rank * width + (which ? e / rj : e % width);
            if (cc >= ncol) continue;
            float s = 0.f;
            if (q.cs > 1)
                for (int k = 0; k < q.cs; ++k) s += peer_float(sums + j * OS + cc, k);
            else
                s = sums[j * OS + cc];
            s *= scale;
            const size_t at = which ? (static_cast<size_t>(a) * p.N + col0 + cc) * p.r + j0 + j
                                    : (static_cast<size_t>(a) * p.r + j0 + j) * p.K + col0 + cc;
            if (q.accumulate) s += load_elem(q.out[which], q.g_dtype, at);
            store_y_elem(q.out[which], q.g_dtype, at, s);
        }
        if (q.cs > 1) {  // the peers have read this CTA's sums
            __syncwarp();
            cluster_arrive();
            cluster_wait();
        }
    }
};

template <int XT, bool NATIVE, int MJ>
__global__ void __launch_bounds__(256, MJ > 1 ? 1 : 2) lora_wgrad_kernel(const WgradArgs q) {
    WgradKernel<XT, NATIVE, MJ>::run(q);
}

}  // namespace qg
