// qg_lora_rows.cuh -- the two thin products over rows, in one kernel:
//
//   forward   V = X A^T,          Y  = Y_in  + scaling V B^T
//   backward  G = scaling dY B,   dX = dX_in + G A
//
// Both read a wide row (contraction over `c1` values) into `rank` sums and
// spread them over `c2` outputs.  A cluster of CTAs owns a tile of rows of one
// request: each CTA contracts its share of the row, the partial sums meet
// through distributed shared memory (added in rank order), and each CTA then
// writes its share of the outputs.  One launch, no workspace between the
// products, and the row's own width supplies the parallelism when there are
// few rows; with many rows the cluster is one CTA and several of them on an SM
// overlap each other's phases.  Bound by memory: the wide rows in and out.
//
// The adapter's tensor is read by every tile of its rows, from L2.  In the
// forward pass its contiguous axis is the contraction (fragments load as they
// are); in the backward pass it is the other one, and a byte permute pairs two
// rows' values (NATIVE) where TF32 fragments take single values.
#pragma once

#include "qg_lora_common.cuh"

namespace qg {

struct RowsArgs {
    LoraProblem p;
    const void *in;      // X or dY
    int64_t ld_in;
    int c1, c2;          // contraction and output widths (forward K, N; backward N, K)
    const void *w1, *w2; // forward A, B; backward B, A
    const void *base;    // Y_in / dX_in or null
    int base_dtype;
    int64_t ld_base;
    void *out;           // Y / dX or null (no second product)
    int out_dtype;
    int64_t ld_out;
    float *sums;         // V_out / G or null, [T][rank]
    float *tile_max;     // backward: [2][tiles] largest finite |G| and |V| of a tile's rows, and its adapter; or null
    int *tile_adapter;
    const float *V;
    TermsOut terms;      // bf16, backward: the terms of G and V for dA and dB
    const float *given;  // the first product's sums where they are known, or null
    int cs;              // CTAs that share a tile: a cluster, unless the sums are given
    int in_vec, out_vec; // rows at 16-byte boundaries: vector accesses
    int in_words;        // input rows at 4-byte boundaries: four words instead of a vector
                         // (2000 rows of 5002 values, rank 16, gradients: bf16 78 -> 57 us,
                         // fp32 127 -> 92; 42 and 83 at 5008; bf16 rows of 5001, two bytes at a time, 82)
};

// GIVEN: the sums of the first product are known (another launch made them).
template <int XT, int WT, bool BWD, int MT, int RG, int NT, bool GIVEN>
struct RowsKernel {
    static constexpr bool NATIVE = XT != kF32;
    static constexpr int KG = 8 / RG;              // warps sharing the rows of a group
    static constexpr int R = 16 * MT * RG;         // rows of a tile
    static constexpr int EL = NATIVE ? 8 : 4;      // contraction values of a lane's 16 bytes
    static constexpr int CH = 4 * EL;              // of a warp's chunk
    static constexpr int BLK = 2 * CH;             // two chunks: 128 bytes of a row
    static constexpr int UW = NATIVE ? 16 : 8;     // rank values of one MMA of the second product
    static constexpr int EU = UW / 4;
    static constexpr int RC = 8 * NT;              // rank values of one pass of the first product
    static constexpr int PS = RC + 4;              // row stride of the partial sums (bank spread)

    static constexpr int PIECES = 4 * MT;          // 16-byte pieces of a lane and block: chunk, row group, row half
    static constexpr int STAGES = 3;

    // Puts 16 bytes of a row (EL values from k on) into the lane's queue, zeros past the end.
    static __device__ __forceinline__ void queue_in(const RowsArgs &q, uint4 *dst, const char *row, int k, bool row_in) {
        if (q.in_vec) {  // the last piece of a row that ends inside it is left to the loads below
            if (!row_in || k >= q.c1 || k + EL <= q.c1) {
                const bool in = row_in && k < q.c1;
                queue_copy<16>(dst, row + (in ? static_cast<size_t>(k) * (NATIVE ? 2 : 4) : 0), in);
                return;
            }
        } else if (q.in_words && (!NATIVE || k + EL <= q.c1 || !(q.c1 & 1))) {  // no word holds a value from past the end
            copy_words(dst, row, k, NATIVE ? 2 : 1, row_in ? q.c1 : 0);
            return;
        }
        uint32_t w[4] = {0, 0, 0, 0};
        if (row_in) {
            if constexpr (NATIVE) {
                const unsigned short *x = reinterpret_cast<const unsigned short *>(row);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (k + e < q.c1) w[e >> 1] |= static_cast<uint32_t>(__ldg(x + k + e)) << (16 * (e & 1));
            } else {
                const unsigned int *x = reinterpret_cast<const unsigned int *>(row);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (k + e < q.c1) w[e] = __ldg(x + k + e);
            }
        }
        *dst = make_uint4(w[0], w[1], w[2], w[3]);
    }

    // The adapter's values of a lane's chunk.  Forward: A[a][j][k ..], the lane
    // column g of tile i is j = j0 + 8 i + g; w.v[i] is what tile i's MMAs take.
    // Backward: B[a][k + e][j], j = j0 + g NT + i, NT contiguous values of EL rows.
    // Tiles i0 .. i0 + NH - 1 at a time.
    static constexpr int NH = NT < 4 ? NT : 4;
    struct W1 {
        uint32_t v[BWD ? EL : NH][BWD ? (WT == kF32 ? NH : NH / 2) : 4];
    };

    static __device__ __forceinline__ void load_w1(const RowsArgs &q, int a, int j0, int i0, int k, int g, W1 &w) {
        const int r = q.p.r;
        if constexpr (!BWD) {
#pragma unroll
            for (int i = 0; i < NH; ++i) {
                w.v[i][0] = w.v[i][1] = w.v[i][2] = w.v[i][3] = 0;
                if (j0 + 8 * (i0 + i) >= r || k >= q.c1) continue;  // the rank is a multiple of 8
                const size_t at = (static_cast<size_t>(a) * r + j0 + 8 * (i0 + i) + g) * q.c1 + k;
                if constexpr (WT == kF32 || NATIVE) {
                    const uint4 v = __ldg(reinterpret_cast<const uint4 *>(static_cast<const char *>(q.w1) + at * (NATIVE ? 2 : 4)));
                    w.v[i][0] = v.x, w.v[i][1] = v.y, w.v[i][2] = v.z, w.v[i][3] = v.w;
                } else {
                    const uint2 v = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(q.w1) + at));
                    widen(v.x, w.v[i][0], w.v[i][1]);
                    widen(v.y, w.v[i][2], w.v[i][3]);
                }
            }
        } else {
            constexpr int WORDS = WT == kF32 ? NH : NH / 2;
            const bool jin = j0 + g * NT < r;  // a multiple of 8: the NT values are in or out
            const char *src = static_cast<const char *>(q.w1) + ((static_cast<size_t>(a) * q.c1 + k) * r + j0 + g * NT + i0) * (WT == kF32 ? 4 : 2);
#pragma unroll
            for (int e = 0; e < EL; ++e) {
                const bool in = jin && k + e < q.c1;
                const char *x = src + static_cast<size_t>(e) * r * (WT == kF32 ? 4 : 2);
#pragma unroll
                for (int o = 0; o < WORDS; ++o) w.v[e][o] = 0;
                if (!in) continue;
                if constexpr (WORDS % 4 == 0) {
#pragma unroll
                    for (int o = 0; o < WORDS; o += 4) {
                        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(x) + o / 4);
                        w.v[e][o] = v.x, w.v[e][o + 1] = v.y, w.v[e][o + 2] = v.z, w.v[e][o + 3] = v.w;
                    }
                } else if constexpr (WORDS == 2) {
                    const uint2 v = __ldg(reinterpret_cast<const uint2 *>(x));
                    w.v[e][0] = v.x, w.v[e][1] = v.y;
                } else {
                    w.v[e][0] = __ldg(reinterpret_cast<const unsigned int *>(x));
                }
            }
        }
    }

    // What tile i's MMAs take: NATIVE word x = values 2x, 2x + 1 of the
    // contraction; TF32 value x.
    static __device__ __forceinline__ uint32_t w1_word(const W1 &w, int i, int x) {
        if constexpr (!BWD) return w.v[i][x];
        else if constexpr (NATIVE) return __byte_perm(w.v[2 * x][i / 2], w.v[2 * x + 1][i / 2], (i & 1) ? 0x7632u : 0x5410u);
        else if constexpr (WT == kF32) return w.v[x][i];
        else return __float_as_uint(to_float<WT>(static_cast<uint16_t>((i & 1) ? w.v[x][i / 2] >> 16 : w.v[x][i / 2] & 0xFFFFu)));
    }

    static __device__ __forceinline__ void widen(uint32_t v, uint32_t &a, uint32_t &b) {  // two 16-bit values to fp32 bits
        a = __float_as_uint(to_float<WT>(static_cast<uint16_t>(v & 0xFFFFu)));
        b = __float_as_uint(to_float<WT>(static_cast<uint16_t>(v >> 16)));
    }

    // TF32 product of x (fp32, two terms) and w (fp32 bits; two terms when the adapter is fp32)
    static __device__ __forceinline__ void mma_tf32(float (&d)[4], const float (&x)[4], uint32_t w0, uint32_t w1) {
        uint32_t h[4], l[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) split_tf32(x[i], h[i], l[i]);
        mma_tf32_split(d, h, l, w0, w1);
    }
    static __device__ __forceinline__ void mma_tf32_split(float (&d)[4], const uint32_t (&h)[4], const uint32_t (&l)[4], uint32_t w0, uint32_t w1) {
        if constexpr (WT == kF32) {
            uint32_t h0, l0, h1, l1;
            split_tf32(__uint_as_float(w0), h0, l0);
            split_tf32(__uint_as_float(w1), h1, l1);
            mma8(d, l[0], l[1], l[2], l[3], h0, h1);
            mma8(d, h[0], h[1], h[2], h[3], l0, l1);
            mma8(d, h[0], h[1], h[2], h[3], h0, h1);
        } else {
            mma8(d, l[0], l[1], l[2], l[3], w0, w1);
            mma8(d, h[0], h[1], h[2], h[3], w0, w1);
        }
    }

    // The adapter's values of the second product for unit u and the 4 tiles of a
    // 32-column group: b[i][0..1].  Column (tile i, lane column q) is
    // n0 + 8 (q / 2) + 2 i + q % 2, so that a lane ends with 8 contiguous outputs.
    static __device__ __forceinline__ void load_w2(const RowsArgs &q, int a, int u, int n0, int g, int c, uint32_t (&b)[4][2]) {
        const int r = q.p.r, j = u * UW + c * EU;
        const bool jin = j < r;
        if constexpr (!BWD) {  // B[a][n][j ..]
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int n = n0 + (g >> 1) * 8 + 2 * i + (g & 1);
                b[i][0] = b[i][1] = 0;
                if (!jin || n >= q.c2) continue;
                const size_t at = (static_cast<size_t>(a) * q.c2 + n) * r + j;
                if constexpr (NATIVE || WT == kF32) {
                    const uint2 v = __ldg(reinterpret_cast<const uint2 *>(static_cast<const char *>(q.w2) + at * (NATIVE ? 2 : 4)));
                    b[i][0] = v.x, b[i][1] = v.y;
                } else {
                    widen(__ldg(reinterpret_cast<const unsigned int *>(static_cast<const uint16_t *>(q.w2) + at)), b[i][0], b[i][1]);
                }
            }
        } else {  // A[a][j + e][k ..]: 8 contiguous columns of each row, of which this lane's are every other one
            const int k = n0 + (g >> 1) * 8;
            const bool in = jin && k < q.c2;
            const size_t at = (static_cast<size_t>(a) * r + j) * q.c2 + k;
            if constexpr (NATIVE) {
                uint4 row[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    row[e] = in ? __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(q.w2) + at + static_cast<size_t>(e) * q.c2))
                                : make_uint4(0, 0, 0, 0);
                const uint32_t sel = (g & 1) ? 0x7632u : 0x5410u;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    b[i][0] = __byte_perm(word(row[0], i), word(row[1], i), sel);
                    b[i][1] = __byte_perm(word(row[2], i), word(row[3], i), sel);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const size_t o = at + static_cast<size_t>(e) * q.c2;
                    if constexpr (WT == kF32) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint2 v = in ? __ldg(reinterpret_cast<const uint2 *>(static_cast<const float *>(q.w2) + o + 2 * i)) : make_uint2(0, 0);
                            b[i][e] = (g & 1) ? v.y : v.x;
                        }
                    } else {
                        const uint4 v = in ? __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(q.w2) + o)) : make_uint4(0, 0, 0, 0);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t x = word(v, i);
                            b[i][e] = __float_as_uint(to_float<WT>(static_cast<uint16_t>((g & 1) ? x >> 16 : x & 0xFFFFu)));
                        }
                    }
                }
            }
        }
    }

    static __device__ __forceinline__ uint32_t word(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

    // Shared memory.  First product: the lanes' queues.  Then: the CTA's sums
    // (read by the cluster), the rows' whole sums and their scales, and behind
    // them the warps' partial sums, later the operand fragments of the second
    // product and the queues of its base rows.
    static __host__ __device__ int rank_pad(int r) { return (r + UW - 1) / UW * UW; }
    static __host__ __device__ int sums_bytes(int r) { return (GIVEN ? 1 : 2) * R * rank_pad(r) * 4 + R * 4; }
    static __host__ __device__ int frag_bytes(int r) { return (R / 16) * (rank_pad(r) / UW) * 2 * 512; }
    static constexpr int PART_BYTES = KG * R * PS * 4;
    static constexpr int IN_BYTES = 8 * STAGES * PIECES * 512;
    static constexpr int BW = NATIVE ? 1 : 2;       // 16-byte pieces of 8 base values in the activations' type
    static constexpr int BASE_PIECES = 2 * MT * BW;  // of a lane and group
    static constexpr bool PAIRS = GIVEN && BWD && NATIVE;         // 64 columns at a time (pair_groups)
    // Each of the 8 warps keeps its base rows in a region of its own, whichever loop it is at: warps go from one
    // loop to the next without waiting for each other.
    static constexpr int PAIR_PIECES = 4 * MT;      // of a lane and pair of groups, two stages
    static constexpr int QUEUE_PIECES = PAIRS && 2 * PAIR_PIECES > STAGES * BASE_PIECES ? 2 * PAIR_PIECES : STAGES * BASE_PIECES;
    static constexpr int BASE_BYTES = 8 * QUEUE_PIECES * 512;
    static __device__ __forceinline__ uint4 *base_queue(uint4 *frag, int r, int warp, int lane) {
        return frag + frag_bytes(r) / 16 + warp * (QUEUE_PIECES * 32) + lane;
    }
    static __host__ __device__ int queue_offset(int r) { return r > RC ? sums_bytes(r) : 0; }  // several passes: their sums stay
    static __host__ __device__ int smem_bytes(int r) {
        if (GIVEN) return sums_bytes(r) + frag_bytes(r) + BASE_BYTES;
        const int later = PART_BYTES > frag_bytes(r) + BASE_BYTES ? PART_BYTES : frag_bytes(r) + BASE_BYTES;
        return sums_bytes(r) + later > queue_offset(r) + IN_BYTES ? sums_bytes(r) + later : queue_offset(r) + IN_BYTES;
    }

    static __device__ void run(const RowsArgs &q) {
        extern __shared__ __align__(16) unsigned char sm[];
        const LoraProblem &p = q.p;
        const int r = p.r, rp = rank_pad(r);
        float *mine = reinterpret_cast<float *>(sm);
        float *whole = GIVEN ? mine : mine + R * rp;
        float *rscale = whole + R * rp;
        float *part = rscale + R;
        uint4 *frag = reinterpret_cast<uint4 *>(part);
        const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
        const int rg = warp / KG, kg = warp % KG;
        const int rank = blockIdx.x % q.cs, tile = blockIdx.x / q.cs;
        pdl_launch_dependents();
        pdl_wait();
        RowTile t;
        const bool fine = find_tile(p, tile, R, blockIdx.x == 0, t);
        if (!fine || t.rows == 0 || t.adapter < 0)
            if (BWD && !GIVEN && q.tile_adapter && rank == 0 && tid == 0) q.tile_adapter[tile] = -1;
        if (!fine || t.rows == 0) return;  // the same for the whole cluster
        const float scale = t.adapter >= 0 && p.scaling ? __ldg(p.scaling + t.adapter) : 1.f;

        const int ngrp = (q.c2 + 31) / 32;  // 32-column groups of the second product, and this CTA's
        const int n_lo = static_cast<int>(static_cast<int64_t>(ngrp) * rank / q.cs), n_hi = static_cast<int>(static_cast<int64_t>(ngrp) * (rank + 1) / q.cs);

        if (GIVEN && t.adapter >= 0) {
            for (int e = tid; e < R * rp; e += 256) {
                const int row = e / rp, j = e - row * rp;
                whole[e] = row < t.rows && j < r ? __ldg(q.given + static_cast<size_t>(t.t0 + row) * r + j) : 0.f;
            }
            __syncthreads();
        }
        if constexpr (!GIVEN) {
            if (t.adapter >= 0) {
                // ---------------------------------------------------------- first product
                const int nblk = (q.c1 + BLK - 1) / BLK;
                const int b0 = static_cast<int>(static_cast<int64_t>(nblk) * rank / q.cs), b1 = static_cast<int>(static_cast<int64_t>(nblk) * (rank + 1) / q.cs);
                const int row0 = rg * 16 * MT;
                const char *rowp[MT][2];
                bool rin[MT][2];
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int row = row0 + m * 16 + h * 8 + g;
                        rin[m][h] = row < t.rows;
                        rowp[m][h] = static_cast<const char *>(q.in) + static_cast<size_t>(t.t0 + (rin[m][h] ? row : 0)) * q.ld_in * (NATIVE ? 2 : 4);
                    }
                for (int j0 = 0; j0 < r; j0 += RC) {
                    float acc[MT][NT][4] = {};
                    uint4 *queue = reinterpret_cast<uint4 *>(sm + queue_offset(r)) + warp * (STAGES * PIECES * 32) + lane;
                    auto ahead = [&](int b, int slot) {
                        if (b < b1) {
#pragma unroll
                            for (int s = 0; s < 2; ++s)
#pragma unroll
                                for (int m = 0; m < MT; ++m)
#pragma unroll
                                    for (int h = 0; h < 2; ++h)
                                        queue_in(q, queue + (slot * PIECES + (s * MT + m) * 2 + h) * 32, rowp[m][h], b * BLK + s * CH + c * EL, rin[m][h]);
                        }
                        queue_commit();
                    };
                    if (j0) __syncthreads();  // the queues lie over the partial sums of the previous pass
#pragma unroll
                    for (int i = 0; i < STAGES - 1; ++i) ahead(b0 + kg + i * KG, i);
                    int slot = 0;
                    for (int b = b0 + kg; b < b1; b += KG) {
                        ahead(b + (STAGES - 1) * KG, slot == 0 ? STAGES - 1 : slot - 1);
                        constexpr bool TOGETHER = NT <= 4;  // both chunks' adapter values, under the wait for the row
                        W1 wb[TOGETHER ? 2 : 1];
                        if (TOGETHER) {
                            load_w1(q, t.adapter, j0, 0, b * BLK + c * EL, g, wb[0]);
                            load_w1(q, t.adapter, j0, 0, b * BLK + CH + c * EL, g, wb[TOGETHER ? 1 : 0]);
                        }
                        queue_wait<STAGES - 1>();
                        const uint4 *x = queue + slot * PIECES * 32;
                        float part_acc[MT][NT][4] = {};
#pragma unroll
                        for (int s = 0; s < 2; ++s)
#pragma unroll
                            for (int i0 = 0; i0 < NT; i0 += NH) {
                                if (!TOGETHER) load_w1(q, t.adapter, j0, i0, b * BLK + s * CH + c * EL, g, wb[0]);
                                const W1 &w = wb[TOGETHER ? s : 0];
#pragma unroll
                                for (int m = 0; m < MT; ++m) {
                                    const uint4 x0 = x[((s * MT + m) * 2) * 32], x1 = x[((s * MT + m) * 2 + 1) * 32];
                                    if constexpr (NATIVE) {
#pragma unroll
                                        for (int i = 0; i < NH; ++i) {
                                            mma16<XT>(part_acc[m][i0 + i], x0.x, x1.x, x0.y, x1.y, w1_word(w, i, 0), w1_word(w, i, 1));
                                            mma16<XT>(part_acc[m][i0 + i], x0.z, x1.z, x0.w, x1.w, w1_word(w, i, 2), w1_word(w, i, 3));
                                        }
                                    } else {
#pragma unroll
                                        for (int half = 0; half < 2; ++half) {
                                            uint32_t hi[4], lo[4];
                                            split_tf32(__uint_as_float(half ? x0.z : x0.x), hi[0], lo[0]);
                                            split_tf32(__uint_as_float(half ? x1.z : x1.x), hi[1], lo[1]);
                                            split_tf32(__uint_as_float(half ? x0.w : x0.y), hi[2], lo[2]);
                                            split_tf32(__uint_as_float(half ? x1.w : x1.y), hi[3], lo[3]);
#pragma unroll
                                            for (int i = 0; i < NH; ++i)
                                                mma_tf32_split(part_acc[m][i0 + i], hi, lo, w1_word(w, i, 2 * half), w1_word(w, i, 2 * half + 1));
                                        }
                                    }
                                }
                            }
                        // The MMAs add with truncation: a block's sums are added to the row's with
                        // rounding, so the error does not grow with the row.
#pragma unroll
                        for (int m = 0; m < MT; ++m)
#pragma unroll
                            for (int i = 0; i < NT; ++i)
#pragma unroll
                                for (int e = 0; e < 4; ++e) acc[m][i][e] += part_acc[m][i][e];
                        slot = slot == STAGES - 1 ? 0 : slot + 1;
                    }
                    queue_wait<0>();
                    __syncthreads();  // every lane is done with its queue
                    const int jn = min(RC, r - j0);
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int i = 0; i < NT; ++i)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int col = 2 * c + (e & 1), row = row0 + m * 16 + (e >> 1) * 8 + g;
                                part[(kg * R + row) * PS + (BWD ? col * NT + i : i * 8 + col)] = acc[m][i][e];
                            }
                    __syncthreads();
                    for (int e = tid; e < R * jn; e += 256) {
                        const int row = e / jn, j = e - row * jn;
                        float s = 0.f;
#pragma unroll
                        for (int w = 0; w < KG; ++w) s += part[(w * R + row) * PS + j];
                        mine[row * rp + j0 + j] = s;
                    }
                }
                // ---------------------------------------------------------- the cluster's sums
                if (q.cs > 1) {
                    __syncwarp();
                    cluster_arrive();
                    cluster_wait();
                } else {
                    __syncthreads();
                }
                const bool maxima = BWD && q.tile_adapter && rank == 0;
                float mx = 0.f, mv = 0.f;
                for (int e = tid; e < R * rp; e += 256) {
                    const int row = e / rp, j = e - row * rp;
                    float s = 0.f;
                    if (j < r) {
                        if (q.cs > 1)
                            for (int w = 0; w < q.cs; ++w) s += peer_float(mine + e, w);
                        else
                            s = mine[e];
                        if (BWD) s *= scale;
                        if (q.sums && rank == 0 && row < t.rows) {
                            const size_t at = static_cast<size_t>(t.t0 + row) * r + j;
                            q.sums[at] = s;
                            if (BWD && XT == kBF16 && q.terms.at) {
                                put_terms(q.terms, 0, at, s);
                                put_terms(q.terms, 1, at, __ldg(q.V + at));
                            }
                        }
                    }
                    whole[e] = s;
                    if (maxima) {
                        mx = fmaxf(mx, finite_abs(s));
                        if (j < r && row < t.rows) mv = fmaxf(mv, finite_abs(__ldg(q.V + static_cast<size_t>(t.t0 + row) * r + j)));
                    }
                }
                if (maxima) {  // at the place of the partial sums, which have been read
                    unsigned *top = reinterpret_cast<unsigned *>(part);
                    if (tid < 2) top[tid] = 0;
                    __syncthreads();
                    atomicMax(top, __float_as_uint(mx));  // of values that are not negative: the order does not matter
                    atomicMax(top + 1, __float_as_uint(mv));
                    __syncthreads();
                    if (tid == 0) {
                        q.tile_adapter[tile] = t.adapter;
                        q.tile_max[tile] = __uint_as_float(top[0]);
                        q.tile_max[gridDim.x / q.cs + tile] = __uint_as_float(top[1]);
                    }
                }
                __syncthreads();
                if (q.cs > 1) cluster_arrive();  // done with the peers' memory; awaited before leaving
            } else if (!BWD && q.sums && rank == 0) {
                for (int e = tid; e < t.rows * r; e += 256) q.sums[static_cast<size_t>(t.t0) * r + e] = 0.f;
            }
        }
        if (t.adapter >= 0) {
            // ---------------------------------------------------------- operand fragments of the sums
            if (q.out) {
                if constexpr (XT == kF16) {  // bf16 has fp32's range
                    constexpr int TPR = 256 / R;  // threads of a row: neighbours in a warp
                    float mx = 0.f;
                    for (int j = tid % TPR; j < r; j += TPR) mx = fmaxf(mx, fabsf(whole[(tid / TPR) * rp + j]));
#pragma unroll
                    for (int o = TPR / 2; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                    const int ef = static_cast<int>((__float_as_uint(mx) >> 23) & 0xFFu);
                    if (tid % TPR == 0) rscale[tid / TPR] = exp2i(ef == 255 || mx == 0.f ? 0 : min(max(ef - 127, -126), 126));
                    __syncthreads();
                }
                const int units = rp / UW;
                for (int f = tid; f < (R / 16) * units * 32; f += 256) {
                    const int l = f & 31, u = (f >> 5) % units, m = (f >> 5) / units;
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {  // fragment word x: row g (+8 for odd x), the first or second part of the lane's values
                        const int row = m * 16 + (l >> 2) + (x & 1) * 8;
                        const float *v = whole + row * rp + u * UW + (l & 3) * EU + (x >> 1) * (EU / 2);
                        if constexpr (NATIVE) {
                            const float inv = XT == kF16 ? 1.f / rscale[row] : 1.f;
                            uint16_t h0, l0, h1, l1;
                            split16<XT>(v[0] * inv, h0, l0);
                            split16<XT>(v[1] * inv, h1, l1);
                            hi[x] = pack2(h0, h1), lo[x] = pack2(l0, l1);
                        } else {
                            split_tf32(v[0], hi[x], lo[x]);
                        }
                    }
                    frag[((m * units + u) * 2) * 32 + l] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    frag[((m * units + u) * 2 + 1) * 32 + l] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                __syncthreads();
            }
        }

        // -------------------------------------------------------------- second product
        if (q.out) {
            const int units = rp / UW;
            const int row0 = rg * 16 * MT;
            float mul[MT][2];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    mul[m][h] = BWD ? 1.f : scale;
                    if (XT == kF16 && t.adapter >= 0) mul[m][h] *= rscale[row0 + m * 16 + h * 8 + g];
                }
            uint4 *queue = base_queue(frag, r, warp, lane);
            int first = n_lo + kg;
            if (t.adapter >= 0 && q.out_vec && q.out_dtype == XT && (!q.base || q.base_dtype == XT) && units <= UM)
            {
                if constexpr (PAIRS) first = pair_groups(q, t, n_lo, n_hi, kg, row0, rg, g, c, lane, units, mul, frag, queue);
                first = whole_groups(q, t, first, n_hi, row0, rg, g, c, lane, units, mul, frag, queue);
            }
            if constexpr (!BWD)
                if (!q.out_vec) first = odd_groups(q, t, first, n_hi, row0, rg, g, c, lane, units, mul, frag, reinterpret_cast<float *>(queue - lane));
            // What is left: the columns that do not fill a group, other types.
            // The base rows ahead of their sums, when they have the activations' type.
            const bool queued = q.base && q.out_vec && q.base_dtype == XT;
            auto ahead = [&](int b, int slot) {
                const int n = b * 32 + c * 8;
                if (queued && b < n_hi && n + 8 <= q.c2) {
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int row = row0 + m * 16 + h * 8 + g;
                            const bool in = row < t.rows;
                            const char *src = static_cast<const char *>(q.base) + (in ? (static_cast<size_t>(t.t0 + row) * q.ld_base + n) * (NATIVE ? 2 : 4) : 0);
#pragma unroll
                            for (int o = 0; o < BW; ++o) queue_copy<16>(queue + (slot * BASE_PIECES + (m * 2 + h) * BW + o) * 32, src + 16 * o, in);
                        }
                }
                queue_commit();
            };
#pragma unroll
            for (int i = 0; i < STAGES - 1; ++i) ahead(first + i * KG, i);
            int slot = 0;
            for (int b = first; b < n_hi; b += KG) {
                ahead(b + (STAGES - 1) * KG, slot == 0 ? STAGES - 1 : slot - 1);
                const int n0 = b * 32, n = n0 + c * 8;
                const bool vec = q.out_vec && n + 8 <= q.c2;
                float acc[MT][4][4] = {};
                if (t.adapter >= 0)
                    for (int u = 0; u < units; ++u) {
                        uint32_t w[4][2];
                        load_w2(q, t.adapter, u, n0, g, c, w);
                        multiply(acc, frag, u, units, rg, lane, w);
                    }
                queue_wait<STAGES - 1>();
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int row = row0 + m * 16 + h * 8 + g;
                        if (row >= t.rows) continue;
                        float y[8];
                        if (queued && vec) take_base(queue + (slot * BASE_PIECES + (m * 2 + h) * BW) * 32, y);
                        else load_base(q, t.t0 + row, n, vec, y);
                        if (t.adapter >= 0) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) y[e] = fmaf(acc[m][e >> 1][h * 2 + (e & 1)], mul[m][h], y[e]);
                        }
                        store_out(q, t.t0 + row, n, vec, y);
                    }
                slot = slot == STAGES - 1 ? 0 : slot + 1;
            }
        }
        if (!GIVEN && q.cs > 1 && t.adapter >= 0) {
            __syncwarp();
            cluster_wait();
        }
    }

    static constexpr int UM = NT * 8 / UW;  // most units of a rank up to RC

    static __device__ __forceinline__ void multiply(float (&acc)[MT][4][4], const uint4 *frag, int u, int units, int rg, int lane, const uint32_t (&w)[4][2]) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int mt = rg * MT + m;
            const uint4 h = frag[((mt * units + u) * 2) * 32 + lane], l = frag[((mt * units + u) * 2 + 1) * 32 + lane];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (NATIVE) {
                    mma16<XT>(acc[m][i], l.x, l.y, l.z, l.w, w[i][0], w[i][1]);
                    mma16<XT>(acc[m][i], h.x, h.y, h.z, h.w, w[i][0], w[i][1]);
                } else {
                    const uint32_t hh[4] = {h.x, h.y, h.z, h.w}, ll[4] = {l.x, l.y, l.z, l.w};
                    mma_tf32_split(acc[m][i], hh, ll, w[i][0], w[i][1]);
                }
            }
        }
    }

    // The second product over whole 32-column groups, base and outputs in the
    // activations' type at 16-byte boundaries: addresses are steps from pointers
    // set up once (computed anew for every group they were two thirds of the
    // instructions).  Returns the first group that it leaves.
    static __device__ __forceinline__ int whole_groups(const RowsArgs &q, const RowTile &t, int first, int n_hi, int row0, int rg, int g, int c, int lane,
                                                       int units, const float (&mul)[MT][2], const uint4 *frag, uint4 *queue) {
        constexpr int XS = NATIVE ? 2 : 4, WS = WT == kF32 ? 4 : 2;
        const int end = min(n_hi, q.c2 / 32), r = q.p.r;
        if (first >= end) return first;
        const size_t row = static_cast<size_t>(t.t0 + row0 + g);
        const int64_t base_step = q.ld_base * (8 * XS), out_step = q.ld_out * (8 * XS);  // eight rows
        const char *base = static_cast<const char *>(q.base) + (row * q.ld_base + first * 32 + c * 8) * XS;
        char *out = static_cast<char *>(q.out) + (row * q.ld_out + first * 32 + c * 8) * XS;
        bool in[MT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) in[m][h] = row0 + m * 16 + h * 8 + g < t.rows;
        // the lane's adapter values: forward rows n (r values each), backward rows j (c2 values each)
        const char *w2 = static_cast<const char *>(q.w2) +
                         (BWD ? (static_cast<size_t>(t.adapter) * r + c * EU) * q.c2 + first * 32 + (g >> 1) * 8
                              : (static_cast<size_t>(t.adapter) * q.c2 + first * 32 + (g >> 1) * 8 + (g & 1)) * r + c * EU) * WS;
        const int64_t w_row = static_cast<int64_t>(BWD ? q.c2 : 2 * r) * WS, w_unit = static_cast<int64_t>(BWD ? static_cast<int64_t>(UW) * q.c2 : UW) * WS;
        const int w_group = KG * 32 * (BWD ? 1 : r) * WS;
        // The adapter's values come DEPTH groups of this warp ahead of their use (one
        // 16-row tile takes 1 KB of them a group at rank 16: 64 requests of one row
        // took 15.2 us with one group ahead).
        constexpr int DEPTH = MT > 1 || UM > 2 ? 1 : UM == 2 ? 2 : 4;
        uint32_t ring[DEPTH][UM][4][2];
        auto load = [&](const char *p, uint32_t (&w)[UM][4][2]) {
#pragma unroll
            for (int u = 0; u < UM; ++u) {
                const bool jin = u * UW + c * EU < r;
                const char *pu = p + u * w_unit;
#pragma unroll
                for (int i = 0; i < 4; ++i) w[u][i][0] = w[u][i][1] = 0;
                if (!jin) continue;
                if constexpr (!BWD) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (NATIVE || WT == kF32) {
                            const uint2 v = __ldg(reinterpret_cast<const uint2 *>(pu + i * w_row));
                            w[u][i][0] = v.x, w[u][i][1] = v.y;
                        } else {
                            widen(__ldg(reinterpret_cast<const unsigned int *>(pu + i * w_row)), w[u][i][0], w[u][i][1]);
                        }
                    }
                } else if constexpr (NATIVE) {
                    uint4 x[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = __ldg(reinterpret_cast<const uint4 *>(pu + e * w_row));
                    const uint32_t sel = (g & 1) ? 0x7632u : 0x5410u;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        w[u][i][0] = __byte_perm(word(x[0], i), word(x[1], i), sel);
                        w[u][i][1] = __byte_perm(word(x[2], i), word(x[3], i), sel);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if constexpr (WT == kF32) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) w[u][i][e] = __ldg(reinterpret_cast<const unsigned int *>(pu + e * w_row) + 2 * i + (g & 1));
                        } else {
                            const uint4 x = __ldg(reinterpret_cast<const uint4 *>(pu + e * w_row));
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                w[u][i][e] = __float_as_uint(to_float<WT>(static_cast<uint16_t>((g & 1) ? word(x, i) >> 16 : word(x, i) & 0xFFFFu)));
                        }
                    }
                }
            }
        };
        auto ahead = [&](int slot) {  // the base rows at `base`, which moves on
            if (q.base) {
                const char *p = base;
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
#pragma unroll
                        for (int o = 0; o < BW; ++o)
                            queue_copy<16>(queue + (slot * BASE_PIECES + (m * 2 + h) * BW + o) * 32, in[m][h] ? p + 16 * o : static_cast<const char *>(q.base), in[m][h]);
                        p += base_step;
                    }
                base += KG * 32 * XS;
            }
            queue_commit();
        };
        int loaded = first;
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i, loaded += KG) {
            if (loaded < end) ahead(i);
            else queue_commit();
        }
        constexpr bool EARLY = UM <= 4;  // else a group's values are loaded where they are used
        if (EARLY) {
#pragma unroll
            for (int d = 0; d < DEPTH; ++d)
                if (first + d * KG < end) load(w2 + d * w_group, ring[d]);
        }
        int slot = 0, b = first;
        while (b < end) {
#pragma unroll
            for (int d = 0; d < DEPTH; ++d) {
                if (b >= end) break;
                if (loaded < end) ahead(slot == 0 ? STAGES - 1 : slot - 1);
                else queue_commit();
                uint32_t (&w)[UM][4][2] = ring[d];
                if (!EARLY) load(w2, w);
                float acc[MT][4][4] = {};
#pragma unroll
                for (int u = 0; u < UM; ++u)
                    if (u < units) multiply(acc, frag, u, units, rg, lane, w[u]);
                if (EARLY && b + DEPTH * KG < end) load(w2 + DEPTH * w_group, w);
                w2 += w_group;
                queue_wait<STAGES - 1>();
                char *o = out;
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h, o += out_step) {
                        float y[8];
                        if (q.base) {
                            take_base(queue + (slot * BASE_PIECES + (m * 2 + h) * BW) * 32, y);
#pragma unroll
                            for (int e = 0; e < 8; ++e) y[e] = fmaf(acc[m][e >> 1][h * 2 + (e & 1)], mul[m][h], y[e]);
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e) y[e] = acc[m][e >> 1][h * 2 + (e & 1)] * mul[m][h];
                        }
                        if (in[m][h]) store_row(o, y);
                    }
                out += KG * 32 * XS;
                slot = slot == STAGES - 1 ? 0 : slot + 1;
                b += KG, loaded += KG;
            }
        }
        queue_wait<0>();
        return b;
    }

    // The same over pairs of groups, in the backward pass: a lane takes 8 columns of
    // each adapter row in one load and uses them all, and a row tile's fragments
    // are read once for 64 columns.  Column (tile i, lane column q) is n0 + 8 q + i;
    // a lane ends with 16 contiguous outputs.  Returns the first group left to this warp.
    static __device__ __forceinline__ int pair_groups(const RowsArgs &q, const RowTile &t, int n_lo, int n_hi, int kg, int row0, int rg, int g, int c,
                                                      int lane, int units, const float (&mul)[MT][2], const uint4 *frag, uint4 *queue) {
        const int pairs = (min(n_hi, q.c2 / 32) - n_lo) / 2, r = q.p.r;
        if (pairs <= 0) return n_lo + kg;
        const size_t row = static_cast<size_t>(t.t0 + row0 + g);
        const int col = (n_lo + 2 * kg) * 32;
        const int64_t base_step = q.ld_base * 16, out_step = q.ld_out * 16;  // eight rows
        const char *base = static_cast<const char *>(q.base) + (row * q.ld_base + col + c * 16) * 2;
        char *out = static_cast<char *>(q.out) + (row * q.ld_out + col + c * 16) * 2;
        const char *w2 = static_cast<const char *>(q.w2) + ((static_cast<size_t>(t.adapter) * r + c * EU) * q.c2 + col + g * 8) * 2;
        const int64_t w_row = static_cast<int64_t>(q.c2) * 2;
        bool in[MT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) in[m][h] = row0 + m * 16 + h * 8 + g < t.rows;
        auto ahead = [&](int slot) {
            if (q.base) {
                const char *p = base;
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h, p += base_step)
#pragma unroll
                        for (int o = 0; o < 2; ++o)
                            queue_copy<16>(queue + (slot * PAIR_PIECES + (m * 2 + h) * 2 + o) * 32, in[m][h] ? p + 16 * o : static_cast<const char *>(q.base), in[m][h]);
                base += KG * 64 * 2;
            }
            queue_commit();
        };
        if (kg < pairs) ahead(0);
        int slot = 0;
        for (int b = kg; b < pairs; b += KG, slot ^= 1) {
            if (b + KG < pairs) ahead(slot ^ 1);
            else queue_commit();
            float acc[MT][8][4] = {};
            for (int u = 0; u < units; ++u) {
                uint4 x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[e] = u * UW + c * EU < r ? __ldg(reinterpret_cast<const uint4 *>(w2 + (static_cast<int64_t>(u) * UW + e) * w_row)) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const int mt = rg * MT + m;
                    const uint4 h = frag[((mt * units + u) * 2) * 32 + lane], l = frag[((mt * units + u) * 2 + 1) * 32 + lane];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t sel = (i & 1) ? 0x7632u : 0x5410u;
                        const uint32_t b0 = __byte_perm(word(x[0], i >> 1), word(x[1], i >> 1), sel), b1 = __byte_perm(word(x[2], i >> 1), word(x[3], i >> 1), sel);
                        mma16<XT>(acc[m][i], l.x, l.y, l.z, l.w, b0, b1);
                        mma16<XT>(acc[m][i], h.x, h.y, h.z, h.w, b0, b1);
                    }
                }
            }
            w2 += KG * 64 * 2;
            queue_wait<1>();
            char *o = out;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h, o += out_step)
#pragma unroll
                    for (int part = 0; part < 2; ++part) {  // columns 16 c + 8 part ..
                        float y[8];
                        if (q.base) {
                            take_base(queue + (slot * PAIR_PIECES + (m * 2 + h) * 2 + part) * 32, y);
#pragma unroll
                            for (int e = 0; e < 8; ++e) y[e] = fmaf(acc[m][e][h * 2 + part], mul[m][h], y[e]);
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e) y[e] = acc[m][e][h * 2 + part] * mul[m][h];
                        }
                        if (in[m][h]) store_row(o + 16 * part, y);
                    }
            out += KG * 64 * 2;
        }
        queue_wait<0>();
        return n_lo + 2 * pairs + kg;
    }

    // The second product where rows begin at odd addresses: a lane's 8 columns go
    // through the warp's part of the queue, so that each access to memory is 32
    // neighbours of one row (element by element from the lanes' own columns an
    // access touched 8 rows: 1858 x (2496 -> 14270), rank 24, 167 -> 97 us in fp32
    // and 168 -> 72 in fp16; at 14272 columns 81 and 39).  Returns the first group that it leaves: none.
    static __device__ __forceinline__ int odd_groups(const RowsArgs &q, const RowTile &t, int first, int n_hi, int row0, int rg, int g, int c, int lane,
                                                     int units, const float (&mul)[MT][2], const uint4 *frag, float *stage) {
        constexpr int LS = 36;  // row stride: no bank conflicts either way
        static_assert(MT * 16 * LS * 4 <= QUEUE_PIECES * 512, "the stage lies in the warp's queue");
        const int rows = t.rows - row0;
        const auto base_at = [&](int n) { return static_cast<size_t>(t.t0 + row0) * q.ld_base + n; };
        // four rows at a time, so that a tile of one row does not pay for sixteen
        const auto four_rows = [&](auto body) {
#pragma unroll
            for (int i0 = 0; i0 < MT * 16; i0 += 4)
                if (i0 < rows) {
#pragma unroll
                    for (int i = i0; i < i0 + 4; ++i) body(i);
                }
        };
        int b = first;
        for (; b < n_hi; b += KG) {
            const int n0 = b * 32;
            const int mine = n0 + lane < q.c2 ? rows : 0;
            uint32_t raw[MT * 16];
            if (q.base && q.base_dtype == kF32) {
                const uint32_t *p = static_cast<const uint32_t *>(q.base) + base_at(n0 + lane);
                four_rows([&](int i) { raw[i] = i < mine ? p[i * q.ld_base] : 0u; });
            } else if (q.base) {
                const uint16_t *p = static_cast<const uint16_t *>(q.base) + base_at(n0 + lane);
                four_rows([&](int i) { raw[i] = i < mine ? p[i * q.ld_base] : 0u; });
            }
            float acc[MT][4][4] = {};
            if (t.adapter >= 0)
                for (int u = 0; u < units; ++u) {
                    uint32_t w[4][2];
                    load_w2(q, t.adapter, u, n0, g, c, w);
                    multiply(acc, frag, u, units, rg, lane, w);
                }
            if (q.base) {
                if (q.base_dtype == kF32) four_rows([&](int i) { stage[i * LS + lane] = __uint_as_float(raw[i]); });
                else if (q.base_dtype == kF16) four_rows([&](int i) { stage[i * LS + lane] = h2f(static_cast<uint16_t>(raw[i])); });
                else four_rows([&](int i) { stage[i * LS + lane] = __uint_as_float(raw[i] << 16); });
                __syncwarp();
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int row = m * 16 + h * 8 + g;
                    if (row >= rows) continue;
                    float4 *d = reinterpret_cast<float4 *>(stage + row * LS + c * 8);
#pragma unroll
                    for (int o = 0; o < 2; ++o) {
                        float4 y = q.base ? d[o] : make_float4(0.f, 0.f, 0.f, 0.f);
                        if (t.adapter >= 0) {
                            y.x = fmaf(acc[m][2 * o][h * 2], mul[m][h], y.x);
                            y.y = fmaf(acc[m][2 * o][h * 2 + 1], mul[m][h], y.y);
                            y.z = fmaf(acc[m][2 * o + 1][h * 2], mul[m][h], y.z);
                            y.w = fmaf(acc[m][2 * o + 1][h * 2 + 1], mul[m][h], y.w);
                        }
                        d[o] = y;
                    }
                }
            __syncwarp();
            const size_t at = static_cast<size_t>(t.t0 + row0) * q.ld_out + n0 + lane;
            if (q.out_dtype == kF32) {
                float *p = static_cast<float *>(q.out) + at;
                four_rows([&](int i) { if (i < mine) p[i * q.ld_out] = stage[i * LS + lane]; });
            } else if (q.out_dtype == kF16) {
                uint16_t *p = static_cast<uint16_t *>(q.out) + at;
                four_rows([&](int i) { if (i < mine) p[i * q.ld_out] = f2h(stage[i * LS + lane]); });
            } else {
                uint16_t *p = static_cast<uint16_t *>(q.out) + at;
                four_rows([&](int i) { if (i < mine) p[i * q.ld_out] = f2bf(stage[i * LS + lane]); });
            }
            __syncwarp();
        }
        return b;
    }

    // 8 values of the activations' type at a 16-byte boundary
    static __device__ __forceinline__ void store_row(char *o, const float (&y)[8]) {
        if constexpr (NATIVE) {
            uint32_t v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (XT == kF16) {
                    const __half2 p = __floats2half2_rn(y[2 * e], y[2 * e + 1]);
                    v[e] = *reinterpret_cast<const uint32_t *>(&p);
                } else {
                    const __nv_bfloat162 p = __floats2bfloat162_rn(y[2 * e], y[2 * e + 1]);
                    v[e] = *reinterpret_cast<const uint32_t *>(&p);
                }
            }
            *reinterpret_cast<uint4 *>(o) = make_uint4(v[0], v[1], v[2], v[3]);
        } else {
            reinterpret_cast<float4 *>(o)[0] = make_float4(y[0], y[1], y[2], y[3]);
            reinterpret_cast<float4 *>(o)[1] = make_float4(y[4], y[5], y[6], y[7]);
        }
    }

    // 8 base values of the activations' type from the lane's queue
    static __device__ __forceinline__ void take_base(const uint4 *from, float (&v)[8]) {
        const uint4 a = from[0];
        if constexpr (XT == kF16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t x = word(a, i);
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&x));
                v[2 * i] = f.x, v[2 * i + 1] = f.y;
            }
        } else if constexpr (XT == kBF16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(word(a, i) << 16), v[2 * i + 1] = __uint_as_float(word(a, i) & 0xFFFF0000u);
        } else {
            const uint4 b = from[32];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(word(a, i)), v[4 + i] = __uint_as_float(word(b, i));
        }
    }

    static __device__ __forceinline__ void load_base(const RowsArgs &q, int t, int n, bool vec, float (&v)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.f;
        if (!q.base) return;
        const size_t at = static_cast<size_t>(t) * q.ld_base + n;
        if (vec) {
            if (q.base_dtype == kF32) {
                const float4 a = *reinterpret_cast<const float4 *>(static_cast<const float *>(q.base) + at);
                const float4 b = *reinterpret_cast<const float4 *>(static_cast<const float *>(q.base) + at + 4);
                v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
            } else {
                const uint4 a = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(q.base) + at);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t x = word(a, i);
                    const uint16_t x0 = static_cast<uint16_t>(x & 0xFFFFu), x1 = static_cast<uint16_t>(x >> 16);
                    v[2 * i] = q.base_dtype == kF16 ? h2f(x0) : bf2f(x0);
                    v[2 * i + 1] = q.base_dtype == kF16 ? h2f(x1) : bf2f(x1);
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (n + e < q.c2) v[e] = load_elem(q.base, q.base_dtype, at + e);
        }
    }

    static __device__ __forceinline__ void store_out(const RowsArgs &q, int t, int n, bool vec, const float (&y)[8]) {
        const size_t at = static_cast<size_t>(t) * q.ld_out + n;
        if (vec) {
            if (q.out_dtype == kF32) {
                float4 *d = reinterpret_cast<float4 *>(static_cast<float *>(q.out) + at);
                d[0] = make_float4(y[0], y[1], y[2], y[3]);
                d[1] = make_float4(y[4], y[5], y[6], y[7]);
            } else {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[i] = q.out_dtype == kF16 ? pack2(f2h(y[2 * i]), f2h(y[2 * i + 1])) : pack2(f2bf(y[2 * i]), f2bf(y[2 * i + 1]));
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(q.out) + at) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (n + e < q.c2) store_y_elem(q.out, q.out_dtype, at + e, y[e]);
        }
    }
};

// Both products: tiles of kRowsTile rows, which all eight warps share; the second
// one alone: 64 rows in two groups of 32.  (Tiles of 64 rows for both were slower
// at every size measured, 256 to 4096 rows: 77 against 77 us for 4096 x 5120 x
// 5120 fp32 at rank 16, 245 against 172 at rank 64.)
constexpr int kRowsTile = 16;
struct RowsPlan {
    int cs, tiles;
};

template <int XT, int WT, bool BWD, int MT, int RG, int NT, bool GIVEN>
__global__ void __launch_bounds__(256, 2) lora_rows_kernel(const RowsArgs q) {
    RowsKernel<XT, WT, BWD, MT, RG, NT, GIVEN>::run(q);
}

template <int XT, int WT, bool BWD, int MT, int RG, int NT, bool GIVEN>
cudaError_t launch_rows_one(RowsArgs q, const RowsPlan &plan, cudaStream_t s) {
    auto kern = lora_rows_kernel<XT, WT, BWD, MT, RG, NT, GIVEN>;
    const int smem = RowsKernel<XT, WT, BWD, MT, RG, NT, GIVEN>::smem_bytes(q.p.r);
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e = allow_smem(kern, done, RowsKernel<XT, WT, BWD, MT, RG, NT, GIVEN>::smem_bytes(kMaxRank), true);
    if (e != cudaSuccess) return e;
    if constexpr (!GIVEN) {
        static ClusterFit fit;
        q.cs = fitting_cluster(reinterpret_cast<const void *>(kern), fit, q.cs, 256, RowsKernel<XT, WT, BWD, MT, RG, NT, GIVEN>::smem_bytes(kMaxRank));
    }
    return launch_cluster(kern, dim3(static_cast<unsigned>(plan.tiles) * q.cs), dim3(256), smem, s, GIVEN ? 1 : q.cs, q);
}

template <int XT, int WT, bool BWD, int MT, int RG, bool GIVEN>
cudaError_t launch_rows_rank(const RowsArgs &q, const RowsPlan &plan, cudaStream_t s) {
    const int r = q.p.r;
    return r <= 16 ? launch_rows_one<XT, WT, BWD, MT, RG, 2, GIVEN>(q, plan, s)
                   : r <= 32 ? launch_rows_one<XT, WT, BWD, MT, RG, 4, GIVEN>(q, plan, s) : launch_rows_one<XT, WT, BWD, MT, RG, 8, GIVEN>(q, plan, s);
}

template <int XT, int WT, bool BWD>
cudaError_t launch_rows_shape(const RowsArgs &q, const RowsPlan &plan, cudaStream_t s) {
    if constexpr (XT != kF32)  // many rows of 16-bit activations take their sums from the tensor cores
        if (q.given) return launch_rows_rank<XT, WT, BWD, 2, 2, true>(q, plan, s);
    return launch_rows_rank<XT, WT, BWD, 1, 1, false>(q, plan, s);
}

// Defined once for each pair of types (qg_lora_bf16.cu and its siblings).
template <int XT, int WT>
cudaError_t launch_rows(const RowsArgs &q, bool bwd, const RowsPlan &plan, cudaStream_t s);
#define QG_DEFINE_LAUNCH_ROWS(XT, WT)                                                                                  \
    template <>                                                                                                        \
    cudaError_t launch_rows<XT, WT>(const RowsArgs &q, bool bwd, const RowsPlan &plan, cudaStream_t s) {               \
        return bwd ? launch_rows_shape<XT, WT, true>(q, plan, s) : launch_rows_shape<XT, WT, false>(q, plan, s);       \
    }

}  // namespace qg
