// qg_lora_tc.cu -- the adapters' contractions on the tensor cores (tcgen05 +
// TMA), for 16-bit activations in batches of many rows:
//
//   shrink  V = X A^T  (forward)  or  G = scaling dY B  (backward)
//   wgrad   dA = G^T X  and  dB = scaling V^T dY
//
// Each reads a wide matrix once and is bound by that read; a ring of TMA stages
// keeps about 100 to 200 KB an SM in flight, which loads through registers or
// per-lane queues cannot, and no thread touches the wide operand.
//
// Layouts (128-byte swizzle).  K-major operands have the contraction along
// their rows; MN-major ones come as [64-column block][row] straight from
// row-major memory, so nothing is transposed:
//             MMA operand A (128)          MMA operand B
//   forward   X, K-major, 128 rows         A[a], K-major
//   backward  dY, K-major, 128 rows        B[a], MN-major
//   wgrad     G or V, MN-major, 16-bit     X or dY, MN-major, 256 columns
// (wgrad the other way round, the wide operand as A in two halves and N = the
// rank, kept the tensor pipe busy for 116 cycles an MMA and was bound by it.)
// The thin operand of wgrad is fp32; it comes in two 16-bit terms (three for fp32
// gradients of bf16 activations).  For bf16 whatever makes G writes them, of V
// too; for fp16 a small kernel does, after scaling by the power of two that the
// adapter's largest value gives.  Done by every CTA of wgrad for itself, that
// work took longer than its wide operand (125 us of 8192 x (4096 + 14336) bf16 at
// rank 64).
#include <algorithm>
#include <atomic>

#include "qg_lora_tc.h"
#include "qg_tc_common.cuh"

namespace qg {
namespace {

constexpr int kStep = 64;            // contraction values of a step
constexpr int kTileRows = 128;       // rows of a shrink tile
constexpr int kInBytes = kTileRows * kStep * 2;
constexpr int kBlock = kStep * 128;  // 64 rows of a 64-column block
constexpr int kShrinkThreads = 192;  // TMA, MMA, four warps that read the sums back
constexpr int kBars = 256;           // bytes of barriers and flags
// The MMAs add to their accumulator with truncation (about 1.4e-8 of a sum each
// time, measured), which would grow with the contraction: after this many steps
// of four MMAs or more the accumulator is added, with rounding, to sums in
// registers while the next steps go to a second one.
constexpr int kDrainShrink = 8, kDrainWgrad = 4;

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// MN-major operand: 64-column blocks `block` bytes apart, 8-row groups 1024.
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t saddr, int block = kBlock) {
    uint64_t d = static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(block >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

__device__ __forceinline__ int pow2_cols(int n) { return n <= 32 ? 32 : n <= 64 ? 64 : n <= 128 ? 128 : 256; }

// ------------------------------------------------------------------ shrink
__global__ void __launch_bounds__(kShrinkThreads) lora_shrink_tc_kernel(const __grid_constant__ CUtensorMap in_map,
                                                                        const __grid_constant__ CUtensorMap w_map, const ShrinkTc q) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int stage_bytes = kInBytes + q.w_bytes;
    unsigned char *bars = sm + q.stages * stage_bytes;
    uint64_t *full = reinterpret_cast<uint64_t *>(bars), *empty = full + q.stages;
    uint64_t *accf = empty + q.stages, *drained = accf + 2;  // of two accumulators
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drained + 2);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    unsigned *smax = tmem_slot + 2;  // largest sums and V of this CTA's rows, as bits
    const LoraProblem &p = q.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = p.r;
    const int rank = blockIdx.x % q.cs, tile = blockIdx.x / q.cs;
    pdl_launch_dependents();
    pdl_wait();
    RowTile t;
    const bool fine = find_tile(p, tile, kTileRows, blockIdx.x == 0, t);
    if (!fine || t.rows == 0 || t.adapter < 0) {  // the whole cluster
        if (q.tile_adapter && tid == 0) q.tile_adapter[blockIdx.x] = -1;
        if (fine && t.rows > 0 && rank == 0)
            for (int e = tid; e < t.rows * r; e += kShrinkThreads) q.sums[static_cast<size_t>(t.t0) * r + e] = 0.f;
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < q.stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&accf[i], 1);
            mbar_init(&drained[i], 4);
        }
        *abort_flag = 0;
        smax[0] = smax[1] = 0;
        mbar_fence_init();
    }
    const uint32_t cols = pow2_cols(q.n);  // of one accumulator
    if (warp == 1) tmem_alloc(tmem_slot, 2 * cols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int s0 = static_cast<int>(static_cast<int64_t>(q.steps) * rank / q.cs), ns = static_cast<int>(static_cast<int64_t>(q.steps) * (rank + 1) / q.cs) - s0;

    bool ok = true;
    if (warp == 0) {
        if (lane == 0)
            for (int i = 0; i < ns; ++i) {
                const int s = i % q.stages, k = (s0 + i) * kStep;
                if (!mbar_wait(&empty[s], ((i / q.stages) & 1) ^ 1, abort_flag, q.fault, FAULT_WAIT_TC)) break;
                unsigned char *dst = sm + s * stage_bytes;
                mbar_arrive_expect_tx(&full[s], stage_bytes);
                tma_load_2d(dst, &in_map, k, t.t0, &full[s]);  // rows past the tensor come as zeros, later requests' are ignored
                if (!q.bwd) {
                    tma_load_3d(dst + kInBytes, &w_map, k, 0, t.adapter, &full[s]);
                } else {
                    for (int b = 0; b * kBlock < q.w_bytes; ++b) tma_load_3d(dst + kInBytes + b * kBlock, &w_map, 64 * b, k, t.adapter, &full[s]);
                }
            }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = idesc_f16(128, q.n, q.bf16) | (q.bwd ? 1u << 16 : 0u);
            for (int i = 0; i < ns; ++i) {
                const int s = i % q.stages, blk = i / kDrainShrink, buf = blk & 1;
                const bool fresh = i % kDrainShrink == 0;
                ok = (!fresh || mbar_wait(&drained[buf], ((blk >> 1) & 1) ^ 1, abort_flag, q.fault, FAULT_WAIT_TC)) &&
                     mbar_wait(&full[s], (i / q.stages) & 1, abort_flag, q.fault, FAULT_WAIT_TC);
                if (!ok) break;
                tc_fence_after();
                const uint32_t at = smem_u32(sm + s * stage_bytes);
                const uint64_t ad = sdesc_k128(at), bd = q.bwd ? sdesc_mn(at + kInBytes) : sdesc_k128(at + kInBytes);
#pragma unroll
                for (int k = 0; k < kStep / 16; ++k) umma_f16(tmem + buf * cols, ad + 2 * k, bd + (q.bwd ? 128 : 2) * k, idesc, !fresh || k > 0);
                umma_commit(&empty[s]);
                if (i % kDrainShrink == kDrainShrink - 1 || i == ns - 1) umma_commit(&accf[buf]);
            }
        }
    }
    float sum[4][32];  // of this thread's row
    if (warp >= 2) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i) sum[c][i] = 0.f;
        for (int blk = 0; blk * kDrainShrink < ns; ++blk) {
            const int buf = blk & 1;
            ok = mbar_wait(&accf[buf], (blk >> 1) & 1, abort_flag, q.fault, FAULT_WAIT_TC);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (c * 32 >= q.n) break;
                uint32_t v[32];
                tmem_ld32(tmem + buf * cols + (static_cast<uint32_t>((warp & 3) * 32) << 16) + c * 32, v);
#pragma unroll
                for (int i = 0; i < 32; ++i) sum[c][i] += __uint_as_float(v[i]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&drained[buf]);
        }
    }
    __syncwarp();
    // The CTA's sums to shared memory (over the ring: every stage has been read), then the cluster's.
    float *mine = reinterpret_cast<float *>(sm);
    const int stride = q.n + 4;
    tc_fence_before();
    __syncthreads();
    if (warp >= 2) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            float4 *dst = reinterpret_cast<float4 *>(mine + ((warp & 3) * 32 + lane) * stride + c * 32);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c * 32 + 4 * i < q.n) dst[i] = make_float4(sum[c][4 * i], sum[c][4 * i + 1], sum[c][4 * i + 2], sum[c][4 * i + 3]);
        }
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 2 * cols);
        __syncwarp();
    }
    if (q.cs > 1) {
        cluster_arrive();
        cluster_wait();
    }
    const float scale = q.bwd && p.scaling ? __ldg(p.scaling + t.adapter) : 1.f;
    const int r_lo = kTileRows * rank / q.cs, r_hi = min(kTileRows * (rank + 1) / q.cs, t.rows);
    float mx = 0.f, mv = 0.f;
    for (int e = tid; e < (r_hi - r_lo) * (r / 4); e += kShrinkThreads) {  // four values of a row
        const int row = r_lo + e / (r / 4), j = e % (r / 4) * 4;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        if (q.cs > 1) {
            for (int w = 0; w < q.cs; ++w) {
                const float4 v = peer_float4(mine + row * stride + j, w);
                s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
            }
        } else {
            s = *reinterpret_cast<const float4 *>(mine + row * stride + j);
        }
        s.x *= scale, s.y *= scale, s.z *= scale, s.w *= scale;
        const size_t at = static_cast<size_t>(t.t0 + row) * r + j;
        *reinterpret_cast<float4 *>(q.sums + at) = s;
        if (q.terms.at) {
            const float4 v = __ldg(reinterpret_cast<const float4 *>(q.V + at));
            const float g4[4] = {s.x, s.y, s.z, s.w}, v4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                put_terms(q.terms, 0, at + i, g4[i]);
                put_terms(q.terms, 1, at + i, v4[i]);
            }
        }
        mx = fmaxf(mx, fmaxf(fmaxf(finite_abs(s.x), finite_abs(s.y)), fmaxf(finite_abs(s.z), finite_abs(s.w))));
        if (q.tile_adapter) {
            const float4 v = __ldg(reinterpret_cast<const float4 *>(q.V + at));
            mv = fmaxf(mv, fmaxf(fmaxf(finite_abs(v.x), finite_abs(v.y)), fmaxf(finite_abs(v.z), finite_abs(v.w))));
        }
    }
    if (q.tile_adapter) {
        atomicMax(&smax[0], __float_as_uint(mx));  // of values that are not negative: the order does not matter
        atomicMax(&smax[1], __float_as_uint(mv));
        __syncthreads();
        if (tid == 0) {
            q.tile_adapter[blockIdx.x] = t.adapter;
            q.tile_max[blockIdx.x] = __uint_as_float(smax[0]);
            q.tile_max[gridDim.x + blockIdx.x] = __uint_as_float(smax[1]);
        }
    }
    if (q.cs > 1) {  // the peers have read this CTA's sums
        __syncwarp();
        cluster_arrive();
        cluster_wait();
    }
}

// ------------------------------------------------------------------ wgrad
constexpr int kCols = 256;                       // of a CTA
constexpr int kWideBytes = kStep * kCols * 2;    // a step: four 64-column blocks
constexpr int kWgThreads = 64 + 8 * 32;          // TMA, MMA, eight warps that mask and read the sums back

// ------------------------------------------------------------------ terms
// 2^exponent brings values up to `largest` (as bits) within [2^14, 2^15).
__device__ __forceinline__ int fp16_exponent(unsigned largest) {
    const int ef = static_cast<int>((largest >> 23) & 0xFFu);
    return ef == 0 || ef == 255 ? 0 : min(max(14 - (ef - 127), -100), 100);
}

// The largest finite |value| of an adapter's G (which = 0) or V (1), from the shrink launch; every thread of the block calls it.
__device__ __forceinline__ unsigned largest_of(const float *tile_max, const int *tile_adapter, int parts, int which, int a, unsigned *smax) {
    float mx = 0.f;
    for (int i = threadIdx.x; i < parts; i += blockDim.x)
        if (__ldcg(tile_adapter + i) == a) mx = fmaxf(mx, __ldcg(tile_max + which * parts + i));
    atomicMax(smax, __float_as_uint(mx));  // of values that are not negative: the order does not matter
    __syncthreads();
    return *smax;
}

// G and V of a tile of rows as two fp16 terms each, scaled for the tile's adapter.
__global__ void __launch_bounds__(256) lora_terms_kernel(const TermsTc q) {
    __shared__ unsigned smax[2];
    const LoraProblem &p = q.p;
    pdl_launch_dependents();
    pdl_wait();
    RowTile t;
    if (!find_tile(p, blockIdx.x, kTileRows, false, t) || t.rows == 0 || t.adapter < 0) return;
    const int which = blockIdx.y;
    if (threadIdx.x == 0) smax[which] = 0;
    __syncthreads();
    const float up = exp2i(fp16_exponent(largest_of(q.tile_max, q.tile_adapter, q.parts, which, t.adapter, smax + which)));
    const size_t all = static_cast<size_t>(p.T) * p.r, first = static_cast<size_t>(t.t0) * p.r;
    const float *src = q.skinny[which] + first;
    uint16_t *dst = q.terms + which * 2 * all + first;
    for (int e = threadIdx.x * 4; e < t.rows * p.r; e += 1024) {
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(src + e));
        const float x[4] = {v.x * up, v.y * up, v.z * up, v.w * up};
        uint16_t hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) split16<kF16>(x[k], hi[k], lo[k]);
        *reinterpret_cast<uint2 *>(dst + e) = make_uint2(pack2(hi[0], hi[1]), pack2(hi[2], hi[3]));
        *reinterpret_cast<uint2 *>(dst + all + e) = make_uint2(pack2(lo[0], lo[1]), pack2(lo[2], lo[3]));
    }
}

// The 64-row steps of an adapter's requests that belong to CTA `rank` of `cs`, walked by a whole warp.
struct StepWalk {
    int s = 0, base = 0, left;
    unsigned mask = 0;
    int64_t t = 0, end = 0;
    __device__ explicit StepWalk(int rank) : left(rank) {}
    __device__ bool next(const LoraProblem &p, int a, int cs, int &t0, int &rows) {
        for (;;) {
            if (t < end) {
                const int64_t n = (end - t + kStep - 1) / kStep;
                if (left < n) {
                    const int64_t at = t + static_cast<int64_t>(left) * kStep;
                    t0 = static_cast<int>(at);
                    rows = static_cast<int>(end - at < kStep ? end - at : kStep);
                    t = at + kStep;
                    left = cs - 1;
                    return true;
                }
                left -= static_cast<int>(n);
                t = end;
            }
            while (!mask) {
                if (s >= p.S) return false;
                const int i = s + (threadIdx.x & 31);
                mask = __ballot_sync(0xffffffffu, i < p.S && __ldg(p.ids + min(i, p.S - 1)) == a);
                base = s;
                s += 32;
            }
            const int seg = base + __ffs(mask) - 1;
            mask &= mask - 1;
            t = __ldg(p.offs + seg);
            end = __ldg(p.offs + seg + 1);
        }
    }
};

// DRAIN: fp32 gradients, and 16-bit ones of very many rows (drained_wgrad).  One CTA an SM then, for two accumulators
// and the registers of the sums.
template <int TERMS, bool BF16, bool DRAIN>
__global__ void __launch_bounds__(kWgThreads, DRAIN ? 1 : 2) lora_wgrad_tc_kernel(const __grid_constant__ CUtensorMap x_map, const __grid_constant__ CUtensorMap dy_map,
                                                                      const __grid_constant__ CUtensorMap thin_map, const WgradTc q) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const LoraProblem &p = q.p;
    const int blocks = q.n > 64 ? 2 : 1;  // 64-column blocks of the thin operand
    const int term_bytes = blocks * kBlock, thin_bytes = TERMS * term_bytes, stage_bytes = kWideBytes + thin_bytes;
    unsigned char *bars = sm + q.stages * stage_bytes;
    uint64_t *full = reinterpret_cast<uint64_t *>(bars), *empty = full + q.stages, *masked = empty + q.stages;
    uint64_t *accf = masked + q.stages, *drained = accf + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drained + 2);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    unsigned *smax = tmem_slot + 2;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = blockIdx.x % q.cs;
    int tile = blockIdx.x / q.cs;
    const int which = tile >= q.tiles[0];
    if (which) tile -= q.tiles[0];
    const int a = blockIdx.y, col0 = tile * kCols, r = p.r;
    pdl_launch_dependents();
    pdl_wait();
    int bad = 0;
    for (int s = tid; s < p.S; s += kWgThreads) {
        const int64_t lo = __ldg(p.offs + s), hi = __ldg(p.offs + s + 1);
        bad |= hi < lo || lo < 0 || hi > p.T || (s == 0 && lo != 0);
    }
    if (tid == 0) {
        for (int i = 0; i < q.stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
            mbar_init(&masked[i], 8);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&accf[i], 1);
            mbar_init(&drained[i], 8);
        }
        *abort_flag = 0;
        *smax = 0;
        mbar_fence_init();
    }
    if (__syncthreads_or(bad)) return;  // the whole cluster
    if (warp == 1) tmem_alloc(tmem_slot, (DRAIN ? 2 : 1) * kCols);
    float down = 1.f;
    if (!BF16) down = exp2i(-fp16_exponent(largest_of(q.tile_max, q.tile_adapter, q.parts, which, a, smax)));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    StepWalk walk(rank);
    int t0, rows, steps = 0;
    bool ok = true;
    if (warp == 0) {
        const CUtensorMap *map = which ? &dy_map : &x_map;
        while (walk.next(p, a, q.cs, t0, rows)) {
            if (lane == 0) {
                const int s = steps % q.stages;
                ok = mbar_wait(&empty[s], ((steps / q.stages) & 1) ^ 1, abort_flag, q.fault, FAULT_WAIT_TC);
                if (ok) {
                    unsigned char *dst = sm + s * stage_bytes;
                    mbar_arrive_expect_tx(&full[s], stage_bytes);
#pragma unroll
                    for (int b = 0; b < kCols / 64; ++b) tma_load_2d(dst + b * kBlock, map, col0 + 64 * b, t0, &full[s]);
                    for (int m = 0; m < TERMS; ++m)
                        for (int b = 0; b < blocks; ++b)
                            tma_load_3d(dst + kWideBytes + m * term_bytes + b * kBlock, &thin_map, 64 * b, t0, which * TERMS + m, &full[s]);
                }
            }
            if (!__shfl_sync(0xffffffffu, ok, 0)) break;
            ++steps;
        }
    } else if (warp == 1) {
        constexpr uint32_t idesc = idesc_f16(128, kCols, BF16) | (1u << 15) | (1u << 16);  // both MN-major
        const int thin_block = blocks == 2 ? kBlock : 0;  // up to rank 64 rows 64 .. 127 repeat the first ones, unread
        while (walk.next(p, a, q.cs, t0, rows)) {
            if (lane == 0) {
                const int s = steps % q.stages, blk = DRAIN ? steps / kDrainWgrad : 0, buf = blk & 1;
                const bool fresh = DRAIN ? steps % kDrainWgrad == 0 : steps == 0;
                ok = (!DRAIN || !fresh || mbar_wait(&drained[buf], ((blk >> 1) & 1) ^ 1, abort_flag, q.fault, FAULT_WAIT_TC)) &&
                     mbar_wait(&full[s], (steps / q.stages) & 1, abort_flag, q.fault, FAULT_WAIT_TC) &&
                     mbar_wait(&masked[s], (steps / q.stages) & 1, abort_flag, q.fault, FAULT_WAIT_TC);
                if (ok) {
                    tc_fence_after();
                    const uint32_t at = smem_u32(sm + s * stage_bytes);
                    const uint64_t ad = sdesc_mn(at + kWideBytes, thin_block), bd = sdesc_mn(at);
#pragma unroll
                    for (int m = TERMS - 1; m >= 0; --m)
#pragma unroll
                        for (int k = 0; k < kStep / 16; ++k)
                            umma_f16(tmem + buf * kCols, ad + m * (term_bytes >> 4) + 128 * k, bd + 128 * k, idesc, !fresh || k > 0 || m < TERMS - 1);
                    umma_commit(&empty[s]);
                    if (DRAIN && steps % kDrainWgrad == kDrainWgrad - 1) umma_commit(&accf[buf]);
                }
            }
            if (!__shfl_sync(0xffffffffu, ok, 0)) break;
            ++steps;
        }
        // what is left in the last accumulator
        if (lane == 0 && (!DRAIN || steps % kDrainWgrad)) umma_commit(&accf[DRAIN ? (steps / kDrainWgrad) & 1 : 0]);
        __syncwarp();
    }
    float sum[DRAIN ? 4 : 1][32];  // DRAIN: value j = the lane's, 128 columns
    if (warp >= 2) {
        const int sub = warp & 3, half = (warp - 2) >> 2;
#pragma unroll
        for (int c = 0; c < (DRAIN ? 4 : 1); ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i) sum[c][i] = 0.f;
        auto drain = [&](int blk) {
            const int buf = blk & 1;
            ok = mbar_wait(&accf[buf], (blk >> 1) & 1, abort_flag, q.fault, FAULT_WAIT_TC);
            if (!__all_sync(0xffffffffu, ok)) return false;
            tc_fence_after();
            if (sub * 32 < r)
#pragma unroll
                for (int c = 0; c < (DRAIN ? 4 : 1); ++c) {
                    uint32_t v[32];
                    tmem_ld32(tmem + buf * kCols + (static_cast<uint32_t>(sub * 32) << 16) + half * 128 + c * 32, v);
#pragma unroll
                    for (int i = 0; i < 32; ++i) sum[c][i] += __uint_as_float(v[i]);
                }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&drained[buf]);
            return true;
        };
        // A request that ends inside a step: the rows behind it become zeros in both operands (either may hold a NaN).
        const int u = tid - 64;
        while (walk.next(p, a, q.cs, t0, rows)) {
            const int s = steps % q.stages;
            ok = mbar_wait(&full[s], (steps / q.stages) & 1, abort_flag, q.fault, FAULT_WAIT_TC);
            if (!__all_sync(0xffffffffu, ok)) break;
            if (rows < kStep) {
                const int gone = kStep - rows, chunks = (kCols / 64 + TERMS * blocks) * 8;
                for (int e = u; e < gone * chunks; e += 256) {
                    const int row = rows + e / chunks, c = e % chunks;
                    *reinterpret_cast<uint4 *>(sm + s * stage_bytes + (c >> 3) * kBlock + row * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_async_smem();
                __syncwarp();
            }
            if (lane == 0) mbar_arrive(&masked[s]);
            ++steps;
            // the accumulator before the one that the MMAs are at
            if (DRAIN && steps % kDrainWgrad == 0 && steps > kDrainWgrad && !drain(steps / kDrainWgrad - 2)) break;
        }
        if constexpr (DRAIN) {
            const int whole = steps / kDrainWgrad;
            if (ok && whole > 0) ok = drain(whole - 1);
            if (ok && steps % kDrainWgrad) ok = drain(whole);
        } else {
            ok = mbar_wait(accf, 0, abort_flag, q.fault, FAULT_WAIT_TC) && ok;
        }
    }
    __syncwarp();
    // The CTA's sums [j][column] to shared memory (over the ring), then the cluster's, and out.
    float *sums = reinterpret_cast<float *>(sm);
    constexpr int OS = kCols + 4;
    __syncthreads();
    if (warp >= 2) {
        tc_fence_after();
        const int sub = warp & 3, half = (warp - 2) >> 2;  // 32 values j; the half of the columns
        if (sub * 32 < r)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t v[32];
                if constexpr (!DRAIN) tmem_ld32(tmem + (static_cast<uint32_t>(sub * 32) << 16) + half * 128 + c * 32, v);
                float4 *dst = reinterpret_cast<float4 *>(sums + (sub * 32 + lane) * OS + half * 128 + c * 32);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                    if constexpr (DRAIN) x = make_float4(sum[c][4 * i], sum[c][4 * i + 1], sum[c][4 * i + 2], sum[c][4 * i + 3]);
                    else if (ok && steps > 0) x = make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]), __uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3]));
                    if (sub * 32 + lane < r) dst[i] = x;
                }
            }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, (DRAIN ? 2 : 1) * kCols);
        __syncwarp();
    }
    if (q.cs > 1) {
        cluster_arrive();
        cluster_wait();
    }
    const int ncol = min(kCols, q.cols[which] - col0), width = kCols / q.cs;
    const float scale = (which && p.scaling ? __ldg(p.scaling + a) : 1.f) * down;
    auto total = [&](int j, int cc) {  // four columns of the cluster's sums
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        if (q.cs == 1) return *reinterpret_cast<const float4 *>(sums + j * OS + cc);
        for (int k = 0; k < q.cs; ++k) {
            const float4 v = peer_float4(sums + j * OS + cc, k);
            s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
        return s;
    };
    auto put = [&](size_t at, float s) {
        s *= scale;
        if (q.accumulate) s += load_elem(q.out[which], q.g_dtype, at);
        store_y_elem(q.out[which], q.g_dtype, at, s);
    };
    for (int e = tid; e < r * (width / 4); e += kWgThreads) {
        // dA: neighbours take neighbouring columns; dB: neighbouring j of four columns
        const int j = which ? e % r : e / (width / 4), cc = rank * width + (which ? e / r : e % (width / 4)) * 4;
        if (cc >= ncol) continue;
        const float4 s = total(j, cc);
        const float v[4] = {s.x, s.y, s.z, s.w};
        if (!which) {
            const size_t at = (static_cast<size_t>(a) * r + j) * p.K + col0 + cc;  // a multiple of four, and so is ncol
            if (!q.accumulate && q.g_dtype == kF32) {
                *reinterpret_cast<float4 *>(static_cast<float *>(q.out[0]) + at) = make_float4(v[0] * scale, v[1] * scale, v[2] * scale, v[3] * scale);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) put(at + i, v[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (cc + i < ncol) put((static_cast<size_t>(a) * p.N + col0 + cc + i) * r + j, v[i]);
        }
    }
    if (q.cs > 1) {
        __syncwarp();
        cluster_arrive();
        cluster_wait();
    }
}

// ------------------------------------------------------------------ host side
bool make_map(CUtensorMap &m, bool bf16, const void *base, int rank, const cuuint64_t *dims, const cuuint64_t *strides, const cuuint32_t *box) {
    const cuuint32_t es[3] = {1, 1, 1};
    return encode_fn()(&m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, static_cast<cuuint32_t>(rank),
                       const_cast<void *>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int thin_cols(int r) { return (r + 15) / 16 * 16; }

}  // namespace

bool lora_tc_available() { return encode_fn() != nullptr; }

int shrink_tc_tiles(int T, int S) { return (T + kTileRows - 1) / kTileRows + S; }

cudaError_t launch_shrink_tc(ShrinkTc q, const void *in, int64_t ld, const void *w, cudaStream_t s) {
    const LoraProblem &p = q.p;
    const int c1 = q.bwd ? p.N : p.K;
    q.n = thin_cols(p.r);
    q.steps = (c1 + kStep - 1) / kStep;
    q.w_bytes = q.bwd ? (p.r > 64 ? 2 : 1) * kBlock : q.n * 128;
    q.stages = 4;
    q.fault = fault_word();
    CUtensorMap in_map, w_map;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(c1), static_cast<cuuint64_t>(p.T)}, strides[1] = {static_cast<cuuint64_t>(ld) * 2};
    const cuuint32_t box[2] = {kStep, kTileRows};
    const cuuint64_t wd[3] = {static_cast<cuuint64_t>(q.bwd ? p.r : p.K), static_cast<cuuint64_t>(q.bwd ? p.N : p.r), static_cast<cuuint64_t>(p.na)};
    const cuuint64_t ws[2] = {wd[0] * 2, wd[0] * wd[1] * 2};
    const cuuint32_t wb[3] = {64, static_cast<cuuint32_t>(q.bwd ? kStep : q.n), 1};
    if (!make_map(in_map, q.bf16, in, 2, dims, strides, box) || !make_map(w_map, q.bf16, w, 3, wd, ws, wb)) return cudaErrorInvalidValue;
    const int ring = q.stages * (kInBytes + q.w_bytes);
    const int smem = 1024 + std::max(ring, kTileRows * (q.n + 4) * 4) + kBars;
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e = allow_smem(lora_shrink_tc_kernel, done, 4 * (kInBytes + 2 * kBlock) + 1024 + kBars);
    if (e != cudaSuccess) return e;
    return launch_cluster(lora_shrink_tc_kernel, dim3(static_cast<unsigned>(shrink_tc_tiles(p.T, p.S)) * q.cs), dim3(kShrinkThreads), smem, s, q.cs, in_map,
                          w_map, q);
}

namespace {

template <int TERMS, bool BF16, bool DRAIN>
cudaError_t launch_wgrad_terms(WgradTc q, const CUtensorMap *maps, cudaStream_t s) {
    const LoraProblem &p = q.p;
    const int stage = kWideBytes + TERMS * (q.n > 64 ? 2 : 1) * kBlock;
    // More CTAs than SMs: two on an SM, with half the ring each, so that one's start and end run under the other's loads.
    constexpr int kOverhead = 1024 + kBars;
    q.stages = std::min(4, (227 * 1024 - kOverhead) / stage);
    const int64_t ctas = static_cast<int64_t>(q.tiles[0] + q.tiles[1]) * q.cs * p.na;
    if (!DRAIN && ctas > device_info().sm_count && 2 * stage + kOverhead <= 111 * 1024) q.stages = 2;
    const int smem = 1024 + std::max(q.stages * stage, q.n * (kCols + 4) * 4) + kBars;
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e = allow_smem(lora_wgrad_tc_kernel<TERMS, BF16, DRAIN>, done, 227 * 1024);
    if (e != cudaSuccess) return e;
    return launch_cluster(lora_wgrad_tc_kernel<TERMS, BF16, DRAIN>, dim3(static_cast<unsigned>(q.tiles[0] + q.tiles[1]) * q.cs, p.na), dim3(kWgThreads), smem, s, q.cs,
                          maps[0], maps[1], maps[2], q);
}

}  // namespace

int wgrad_tc_terms(bool bf16, int g_dtype) { return bf16 && g_dtype == kF32 ? 3 : 2; }

// Where dA and dB leave the truncating accumulator every few steps: fp32 gradients always; 16-bit ones, rounded
// at the end, only where the bias would near that rounding.  Two terms are an MMA for every 8 rows, 1.5e-8 of the
// sum each: 6e-5 at 32768 rows of one accumulator and 4.9e-4 at 262144, an eighth of fp16's and bf16's unit
// roundoff.  (2^20 rows of one sign: 1.8e-3 without.)  It costs the second CTA of an SM: 203 against 225 us for
// 16384 x (4096 + 14336) fp16 at rank 64, 550 against 729 for 131072 x (1024 + 4096) bf16.
static bool drained_wgrad(bool bf16, int g_dtype, int rows) { return g_dtype == kF32 || rows > (bf16 ? 262144 : 32768); }

size_t wgrad_tc_terms_bytes(int T, int r) { return static_cast<size_t>(2) * 3 * T * r * 2; }

cudaError_t launch_wgrad_tc(WgradTc q, const float *G, const float *V, uint16_t *terms, const void *x, int64_t ldx, const void *dy, int64_t lddy, bool bf16,
                            cudaStream_t s) {
    const LoraProblem &p = q.p;
    const int nt = wgrad_tc_terms(bf16, q.g_dtype);
    q.n = thin_cols(p.r);
    q.cols[0] = p.K;
    q.cols[1] = p.N;
    for (int w = 0; w < 2; ++w) q.tiles[w] = (q.cols[w] + kCols - 1) / kCols;
    q.fault = fault_word();
    // All CTAs resident at once (drained: one an SM, else two), while each still has four steps.
    const int64_t ctas = static_cast<int64_t>(q.tiles[0] + q.tiles[1]) * p.na;
    const auto cluster = [&](int per_sm) {
        int cs = 1;
        while (cs < 8 && ctas * cs * 2 <= per_sm * device_info().sm_count && p.T / p.na >= 8 * kStep * cs) cs *= 2;
        return cs;
    };
    q.cs = cluster(2);
    const bool drain = drained_wgrad(bf16, q.g_dtype, p.T / q.cs);
    if (drain) q.cs = cluster(1);
    CUtensorMap maps[3];
    const cuuint32_t box[3] = {64, kStep, 1};
    for (int w = 0; w < 2; ++w) {
        const cuuint64_t dims[2] = {static_cast<cuuint64_t>(q.cols[w]), static_cast<cuuint64_t>(p.T)};
        const cuuint64_t strides[1] = {static_cast<cuuint64_t>(w ? lddy : ldx) * 2};
        if (!make_map(maps[w], bf16, w ? dy : x, 2, dims, strides, box)) return cudaErrorInvalidValue;
    }
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(p.r), static_cast<cuuint64_t>(p.T), static_cast<cuuint64_t>(2 * nt)};
    const cuuint64_t strides[2] = {dims[0] * 2, dims[0] * dims[1] * 2};
    if (!make_map(maps[2], bf16, terms, 3, dims, strides, box)) return cudaErrorInvalidValue;
    if (bf16)
        return nt == 3 ? launch_wgrad_terms<3, true, true>(q, maps, s)
               : drain ? launch_wgrad_terms<2, true, true>(q, maps, s) : launch_wgrad_terms<2, true, false>(q, maps, s);
    TermsTc c{};
    c.p = p;
    c.skinny[0] = G;
    c.skinny[1] = V;
    c.terms = terms;
    c.tile_max = q.tile_max;
    c.tile_adapter = q.tile_adapter;
    c.parts = q.parts;
    const cudaError_t e = launch_pdl(lora_terms_kernel, dim3(static_cast<unsigned>(shrink_tc_tiles(p.T, p.S)), 2), dim3(256), 0, s, c);
    if (e != cudaSuccess) return e;
    return drain ? launch_wgrad_terms<2, false, true>(q, maps, s) : launch_wgrad_terms<2, false, false>(q, maps, s);
}

}  // namespace qg
