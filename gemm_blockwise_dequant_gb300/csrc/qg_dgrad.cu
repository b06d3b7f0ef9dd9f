// qg_dgrad.cu -- dX[M][K] = dY[M][N] . dequant(W)[N][K]: the gradient of the
// activations through a frozen blockwise-quantized weight.
//
// The contraction runs over the weight's rows n, so a block's scale and zero
// point change along the sum and the weight has to be formed before the
// product.  Tensor cores (tcgen05):
//
//  * Operand A is dY (n contiguous: K-major), loaded by TMA with the 128-byte
//    swizzle.  Operand B is the dequantized weight, 64 rows n by 128 columns k
//    a CTA and step.  Its k are contiguous in memory, so it is written MN-major
//    -- [64-column block][8-row group][row][swizzled 16-byte chunk] -- and
//    nothing is transposed: a thread turns 32 codes of one row (which share
//    their block parameters, as blocks are at least 32 wide) into four 16-byte
//    chunks.
//  * PAIR = 2: two CTAs of a cluster share one tile (cta_group::2).  Each holds
//    128 rows of every 256-row half and 128 of the 256 columns, so a weight is
//    dequantized once for 512 rows and the tensor core reads each operand byte
//    from shared memory half as often as with one CTA a tile.  The step's
//    shared-memory traffic (operands read, weights written, dY written) is what
//    a one-CTA tile of the same size is bound by.
//  * The codes and parameters go from global memory straight into registers,
//    one step ahead; only dY needs the TMA.
//  * 16-bit dY: the weight is rounded to dY's type, as the forward pass does, so
//    that a product is one MMA.  That rounding is as large as the result's own:
//    error of the 2-norm 0.0023 in bf16 and 3.0e-4 in fp16, where the weight in
//    fp32 gives 0.0017 and 2.1e-4.  A second term would double the MMAs, which bound
//    the kernel.
//  * fp32 dY: dY and the weight are each split in two fp16 terms and three of
//    their four products are added (TERMS = 2; the product of the second terms,
//    2^-22, is left out).  The MMAs add with truncation (about 1.5e-8 of a sum each
//    time, measured), so every kDrain steps the accumulator is added to fp32 sums,
//    with rounding, while the MMAs go on in a second one.  A row of dY is first
//    scaled by a power of two, and all weights by one that their largest
//    parameters give, so that neither term leaves fp16's range.
//  * Tiles that do not fill a wave are split along n and their fp32 pieces added
//    in a fixed order: with up to 128 rows by the cluster of CTAs that made them,
//    through distributed shared memory (one launch, no workspace); with more, by
//    a second kernel.
#include <algorithm>
#include <atomic>

#include "qg_internal.h"
#include "qg_tc_common.cuh"

namespace qg {
namespace {

// ------------------------------------------------------------------ tensor cores
constexpr int kBK = 64;         // rows n of a step
constexpr int kRows = 128;      // dY rows a CTA holds of each half
constexpr int kCols = 128;      // weight columns a CTA dequantizes
constexpr int kTask = 32;       // weights of one thread's task: one row, one block
constexpr int kGroups = 2;      // the dequantizing warps take the steps in turn
constexpr int kGroupThreads = kBK * kCols / kTask;  // 256
constexpr int kDequantWarps = kGroups * kGroupThreads / 32;
constexpr int kThreads = 64 + 32 * kDequantWarps;  // warp 0 TMA, warp 1 MMA, then dequant + epilogue
constexpr int kABytes = kRows * kBK * 2;
constexpr int kWBytes = kBK * kCols * 2;
constexpr int kBlockBytes = kBK * 128;             // one 64-column block of the B operand
constexpr int kDrain = 4;       // TERMS = 2: steps of one accumulator
constexpr int kSmemFixed = 1024 + 512 + 2048;      // alignment, barriers, codebook table
constexpr int kSmemBudget = 227 * 1024;

struct DgradArgs {
    const uint8_t *W;
    const void *par;         // fp16 scales or fp32 absmax, [N][nb]
    const uint16_t *zp;
    int zp_mode;
    float zpv;
    const float *codebook;
    void *dX;
    int x_dtype;
    float *partial;
    int M, N, K, nb, lbs, steps, mt;
    int full_tiles, splits, split_steps;  // as TcArgs: whole tiles first, then the others split along n
    const float *row_scale;  // TERMS = 2: the power of two that undoes a row's scale, and the parameters' maxima
    const float *maxima;
    unsigned *fault;
};

// B operand, MN-major, 128-byte swizzle: 64-column blocks kBlockBytes apart
// (leading offset), 8-row groups 1024 bytes apart (stride offset).
__device__ __forceinline__ uint64_t sdesc_mn128(uint32_t saddr) {
    uint64_t d = static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(kBlockBytes >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

template <int PAIR>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    if constexpr (PAIR == 1)
        umma_f16(d, a, b, idesc, acc);
    else
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
}

// Arrive on `bar` (of both CTAs of a pair) once every MMA issued so far has finished.
template <int PAIR>
__device__ __forceinline__ void commit(uint64_t *bar) {
    if constexpr (PAIR == 1)
        umma_commit(bar);
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
            "h"(static_cast<uint16_t>(3))
            : "memory");
}

template <int PAIR>
__device__ __forceinline__ void alloc_tmem(uint32_t *slot, uint32_t cols) {
    if constexpr (PAIR == 1) {
        tmem_alloc(slot, cols);
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}

template <int PAIR>
__device__ __forceinline__ void free_tmem(uint32_t addr, uint32_t cols) {
    if constexpr (PAIR == 1)
        tmem_dealloc(addr, cols);
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// One arrival on the same barrier of CTA 0 of the cluster (a pair).
__device__ __forceinline__ void arrive_leader(uint64_t *bar) {
    asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %0, 0;\n mbarrier.arrive.release.cluster.shared::cluster.b64 _, [a];\n}\n" ::"r"(
                     smem_u32(bar))
                 : "memory");
}

// As mbar_wait, acquiring what other CTAs of the cluster released.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t *bar, uint32_t parity, volatile int *abort, unsigned *fault, unsigned code) {
    const unsigned long long t0 = globaltimer_ns();
    for (uint32_t i = 0;; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
        if ((i & 63u) == 63u) {
            if (*abort) return false;
            if (globaltimer_ns() - t0 > kWaitTimeoutNs) {
                if (fault) atomicOr(fault, code);
                *abort = 1;
                return false;
            }
        }
    }
}

// Four floats of CTA `rank`'s shared memory, at the place of `p` in this CTA's.
__device__ __forceinline__ float4 peer_float4(const float *p, int rank) {
    float4 v;
    asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %4, %5;\n ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n}\n"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(smem_u32(p)), "r"(rank)
                 : "memory");
    return v;
}

// Four outputs, `at` a multiple of four.
__device__ __forceinline__ void store4(void *dX, int x_dtype, size_t at, const float4 &s) {
    if (x_dtype == 0) {
        *reinterpret_cast<float4 *>(static_cast<float *>(dX) + at) = s;
    } else {
        const uint16_t a = x_dtype == 1 ? f2h(s.x) : f2bf(s.x), b = x_dtype == 1 ? f2h(s.y) : f2bf(s.y);
        const uint16_t c = x_dtype == 1 ? f2h(s.z) : f2bf(s.z), d = x_dtype == 1 ? f2h(s.w) : f2bf(s.w);
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(dX) + at) = make_uint2(a | static_cast<uint32_t>(b) << 16, c | static_cast<uint32_t>(d) << 16);
    }
}

// Weight buffers: a multiple of kGroups, as a group must meet every phase of its buffers' barriers.
__host__ __device__ constexpr int w_bufs(int terms) { return 4 / terms; }
__host__ __device__ constexpr int a_slots(int h, int terms) {
    const int n = (kSmemBudget - kSmemFixed - w_bufs(terms) * terms * kWBytes) / (h * terms * kABytes);
    return n > 8 ? 8 : n;
}
constexpr int smem_bytes(int h, int terms) {
    return kSmemFixed + w_bufs(terms) * terms * kWBytes + a_slots(h, terms) * h * terms * kABytes;
}

// ------------------------------------------------------------------ fp32 dY: scales and terms
constexpr int kMaxBlocks = 64;  // CTAs that look for the parameters' maxima

// 2^e that brings `largest` to [2^14, 2^15), or as near as 2^126 does.
__device__ __forceinline__ int scale_exponent(float largest) {
    return min(14 - (static_cast<int>((__float_as_uint(largest) >> 23) & 0xFFu) - 127), 126);
}

// CTAs 0 .. M-1 split a row of dY; the others find the largest |scale| (absmax) and |zero point|.  Of finite
// values: one that is not must not decide the scale of the others.
__global__ void __launch_bounds__(256) split_dy_kernel(const GemmProblem p, int ld, __half *__restrict__ hi, __half *__restrict__ lo,
                                                       float *__restrict__ row_scale, float *__restrict__ maxima) {
    __shared__ float red[2][8];
    pdl_launch_dependents();
    pdl_wait();
    float mx = 0.f, mz = 0.f;
    const int tid = threadIdx.x;
    const float *dy = static_cast<const float *>(p.A) + static_cast<size_t>(blockIdx.x) * p.N;
    const bool row = static_cast<int>(blockIdx.x) < p.M;
    if (row) {
        for (int n = tid; n < p.N; n += 256) mx = fmaxf(mx, finite_abs(dy[n]));
    } else {
        const size_t total = static_cast<size_t>(p.N) * (p.K / p.bs);
        const size_t first = static_cast<size_t>(blockIdx.x - p.M) * 256 + tid, stride = kMaxBlocks * 256;
        if (p.kind == WK_CODEBOOK) {
            for (size_t i = first; i < total; i += stride) mx = fmaxf(mx, finite_abs(__ldg(p.absmax + i)));
            if (tid < 16) mz = finite_abs(__ldg(p.codebook + tid));
        } else {
            for (size_t i = first; i < total; i += stride) mx = fmaxf(mx, finite_abs(h2f(__ldg(reinterpret_cast<const unsigned short *>(p.scales) + i))));
            if (p.zp_mode == ZP_TENSOR)
                for (size_t i = first; i < total; i += stride) mz = fmaxf(mz, finite_abs(h2f(__ldg(reinterpret_cast<const unsigned short *>(p.zp) + i))));
        }
    }
    for (int o = 16; o >= 1; o >>= 1) {
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        mz = fmaxf(mz, __shfl_xor_sync(0xffffffffu, mz, o));
    }
    if ((tid & 31) == 0) red[0][tid >> 5] = mx, red[1][tid >> 5] = mz;
    __syncthreads();
    for (int w = 0; w < 8; ++w) mx = fmaxf(mx, red[0][w]), mz = fmaxf(mz, red[1][w]);
    if (!row) {
        if (tid == 0) maxima[blockIdx.x - p.M] = mx, maxima[kMaxBlocks + blockIdx.x - p.M] = mz;
        return;
    }
    const int e = scale_exponent(mx);
    if (tid == 0) row_scale[blockIdx.x] = exp2i(-e);
    const float up = exp2i(e);
    const size_t at = static_cast<size_t>(blockIdx.x) * ld;
    for (int n = tid; n < ld; n += 256) {
        const float x = n < p.N ? dy[n] * up : 0.f;
        const __half h = __float2half_rn(x);
        hi[at + n] = h;
        lo[at + n] = __float2half_rn(x - __half2float(h));
    }
}

// The exponent of all weights' scale, from the maxima (every thread of a warp calls it).
__device__ __forceinline__ int weight_exponent(const float *maxima, bool codebook, int bits, bool zt, float zpv) {
    const int lane = threadIdx.x & 31;
    float mx = fmaxf(maxima[lane], maxima[lane + 32]), mz = fmaxf(maxima[kMaxBlocks + lane], maxima[kMaxBlocks + lane + 32]);
    for (int o = 16; o >= 1; o >>= 1) {
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        mz = fmaxf(mz, __shfl_xor_sync(0xffffffffu, mz, o));
    }
    return scale_exponent(codebook ? mx * mz : mx * (static_cast<float>((1 << bits) - 1) + (zt ? mz : fabsf(zpv))));
}

// Eight weights of a task (chunk q) in fp32, as the definition forms them, with the parameter already scaled.
template <int WK, int BITS>
__device__ __forceinline__ void weights8(const uint32_t (&c)[BITS], int q, float zp, float par, const float *lut_lane, float (&w)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int bit = (q * 8 + i) * BITS;
        const uint32_t code = (c[bit >> 5] >> (bit & 31)) & ((1u << BITS) - 1u);
        w[i] = WK == WK_CODEBOOK ? __fmul_rn(lut_lane[code * 32], par) : __fmul_rn(__fsub_rn(static_cast<float>(code), zp), par);
    }
}

__device__ __forceinline__ uint32_t half_pair(float a, float b, float &ra, float &rb) {  // two fp16 values and what they leave
    const __half2 h = __floats2half2_rn(a, b);
    ra = a - __low2float(h), rb = b - __high2float(h);
    return h2_as_u32(h);
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n .reg .b64 ra, rb, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %5};\n add.rn.f32x2 rd, ra, rb;\n mov.b64 {%0, %1}, rd;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// Eight weights (chunk q of a task) as bf16 pairs.  A code masked in place under
// the exponent of 2^23 is the float 2^23 + code * 2^shift; without the 2^23, one
// fma with s * 2^-shift and -zp * s (exact: 22 bits) gives the rounded
// (code - zp) * s.  21 instructions against 40 by way of fp16 pairs, on the pipe
// whose work the MMAs feel (4096 x 35840 x 5120 u4: 1090 -> 1042 us).
template <int BITS>
__device__ __forceinline__ uint4 bf16_weights8(const uint32_t (&c)[BITS], int q, float s, float minus_zps) {
    constexpr uint32_t MASK = (1u << BITS) - 1u, MAGIC = 0x4B000000u;
    constexpr float kMagic = 8388608.f;
    uint32_t out[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        float2 x, m;
        if constexpr (BITS == 8) {
            const uint32_t w = c[2 * q + (p >> 1)];
            x.x = __uint_as_float(__byte_perm(w, MAGIC, (p & 1) ? 0x7652u : 0x7650u));
            x.y = __uint_as_float(__byte_perm(w, MAGIC, (p & 1) ? 0x7653u : 0x7651u));
            m = make_float2(s, s);
        } else {
            // 16 bits hold 4 or 8 codes in place; the pair's shift inside them
            const uint32_t w = BITS == 2 ? c[q >> 1] >> (16 * (q & 1)) : c[q] >> (16 * (p >> 1));
            const int at = BITS == 2 ? 4 * p : 8 * (p & 1);
            x.x = __uint_as_float((w & (MASK << at)) | MAGIC);
            x.y = __uint_as_float((w & (MASK << (at + BITS))) | MAGIC);
            m = make_float2(s * __uint_as_float((127u - at) << 23), s * __uint_as_float((127u - at - BITS) << 23));
        }
        const float2 w = ffma2(add2(x, make_float2(-kMagic, -kMagic)), m, make_float2(minus_zps, minus_zps));
        const __nv_bfloat162 b = __floats2bfloat162_rn(w.x, w.y);
        out[p] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
}

// The codes and parameters of one task.
template <int BITS>
struct Task {
    uint32_t c[BITS];  // 32 weights of BITS bits
    uint32_t par, zp;
};

template <int WK, int BITS, bool BF16, int PAIR, int H, int TERMS>
__global__ void __launch_bounds__(kThreads, 1) dgrad_kernel(const __grid_constant__ CUtensorMap dy_map, const __grid_constant__ CUtensorMap dy_lo_map, const DgradArgs p) {
    static_assert(TERMS == 1 || (!BF16 && H == 1), "the second term of dY takes the second half's place");
    constexpr int NA = a_slots(H, TERMS), NW = w_bufs(TERMS);
    constexpr int AT = H * TERMS * kABytes, WT = TERMS * kWBytes;  // of a step
    constexpr int BN = PAIR * kCols;
    constexpr uint32_t TMEM_COLS = H * TERMS * BN;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    unsigned char *a_s = smem, *w_s = a_s + NA * AT;
    uint64_t *full = reinterpret_cast<uint64_t *>(w_s + NW * WT);  // dY of a step landed
    uint64_t *aempty = full + NA;    // its MMAs are done
    uint64_t *wfull = aempty + NA;   // weights of a step written (one arrival a warp)
    uint64_t *wempty = wfull + NW;   // their MMAs are done
    uint64_t *pfull = wempty + NW;   // (leader) the other CTA's dY and weights of a step are there
    uint64_t *accf = pfull + NW;     // every MMA of the tile (TERMS = 2: of one of two accumulators) is done
    uint64_t *drained = accf + 2;    // (leader; TERMS = 2) every warp of the pair has taken an accumulator's sums
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drained + 2);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    float *lut = reinterpret_cast<float *>(w_s + NW * WT + 512);  // 16 x 32 (codebook)
    static_assert((2 * NA + 3 * NW + 4) * 8 + 8 <= 512, "barriers fit");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = PAIR == 2 ? static_cast<int>(blockIdx.x & 1) : 0;
    int tile = blockIdx.x / PAIR, s0 = 0, ns = p.steps, piece = -1, part = 0;
    if (PAIR == 1) {  // the CTAs of a cluster share a tile
        part = tile % p.splits;
        tile /= p.splits;
        s0 = part * p.split_steps;
        ns = max(0, min(p.steps, s0 + p.split_steps) - s0);
    } else if (tile >= p.full_tiles) {
        const int q = tile - p.full_tiles;
        tile = p.full_tiles + q / p.splits;
        s0 = (q % p.splits) * p.split_steps;
        ns = max(0, min(p.steps, s0 + p.split_steps) - s0);
        if (p.splits > 1) piece = q;
    }
    const int m0 = (tile % p.mt) * (H * PAIR * kRows), k0 = (tile / p.mt) * BN;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NA; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&aempty[i], 1);
        }
        for (int i = 0; i < NW; ++i) {
            mbar_init(&wfull[i], kGroupThreads / 32);
            mbar_init(&wempty[i], 1);
            mbar_init(&pfull[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&accf[i], 1);
            mbar_init(&drained[i], kDequantWarps * PAIR);
        }
        *abort_flag = 0;
        mbar_fence_init();
    }
    if (warp == 1) alloc_tmem<PAIR>(tmem_slot, TMEM_COLS);
    pdl_launch_dependents();
    pdl_wait();  // nothing of the call is read or written before the preceding kernel is done
    if constexpr (WK == WK_CODEBOOK)
        for (int i = threadIdx.x; i < 16 * 32; i += kThreads) lut[i] = __ldg(p.codebook + (i >> 5));
    tc_fence_before();
    if constexpr (PAIR == 2) cluster_sync();  // the peer's barriers are ready
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // A split tile's sums, [row][column] over the dY ring, which is read by then.
    constexpr int SS = kCols + 4;
    float *sums = reinterpret_cast<float *>(a_s);
    const bool shared_tile = PAIR == 1 && p.splits > 1;
    static_assert(NA * AT + NW * WT >= kRows * SS * 4, "the sums fit");

    bool ok = true;
    if (warp == 0) {
        if (lane == 0)
            for (int i = 0; i < ns; ++i) {
                const int s = i % NA;
                if (!mbar_wait(&aempty[s], ((i / NA) & 1) ^ 1, abort_flag, p.fault, FAULT_WAIT_TC)) break;
                mbar_arrive_expect_tx(&full[s], AT);
#pragma unroll
                for (int h = 0; h < H; ++h)  // rows past M and columns past N come as zeros
                    tma_load_2d(a_s + s * AT + h * kABytes, &dy_map, (s0 + i) * kBK, m0 + (h * PAIR + rank) * kRows, &full[s]);
                if constexpr (TERMS == 2) tma_load_2d(a_s + s * AT + kABytes, &dy_lo_map, (s0 + i) * kBK, m0 + rank * kRows, &full[s]);
            }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_f16(PAIR * kRows, BN, BF16) | (1u << 16);  // B MN-major
            const bool two = H == 2 && m0 + PAIR * kRows < p.M;  // the second half holds rows
            for (int i = 0; i < ns && ok; ++i) {
                const int s = i % NA, b = i % NW;
                ok = mbar_wait(&full[s], (i / NA) & 1, abort_flag, p.fault, FAULT_WAIT_TC) &&
                     mbar_wait(&wfull[b], (i / NW) & 1, abort_flag, p.fault, FAULT_WAIT_TC);
                if (!ok) break;
                if (PAIR == 2 && rank == 1) {  // the other CTA's part: tell the leader
                    arrive_leader(&pfull[b]);
                    continue;
                }
                if (PAIR == 2) ok = mbar_wait_cluster(&pfull[b], (i / NW) & 1, abort_flag, p.fault, FAULT_WAIT_TC);
                const int blk = TERMS == 2 ? i / kDrain : 0, buf = blk & 1;
                const bool fresh = TERMS == 2 ? i % kDrain == 0 : i == 0;
                if (TERMS == 2 && fresh) ok = ok && mbar_wait_cluster(&drained[buf], ((blk >> 1) & 1) ^ 1, abort_flag, p.fault, FAULT_WAIT_TC);
                if (!ok) break;
                tc_fence_after();
                const uint64_t ad = sdesc_k128(smem_u32(a_s + s * AT));
                const uint64_t ad1 = sdesc_k128(smem_u32(a_s + s * AT + AT - kABytes));
                const uint64_t bd = sdesc_mn128(smem_u32(w_s + b * WT));
#pragma unroll
                for (int k = 0; k < kBK / 16; ++k) {  // 16 n: 32 bytes along A's rows, two 8-row groups of B
                    const uint32_t acc = tmem + buf * BN, add = !fresh || k > 0;
                    mma<PAIR>(acc, ad + 2 * k, bd + 128 * k, idesc, add);
                    if constexpr (TERMS == 2) {
                        mma<PAIR>(acc, ad + 2 * k, bd + (kWBytes >> 4) + 128 * k, idesc, 1);
                        mma<PAIR>(acc, ad1 + 2 * k, bd + 128 * k, idesc, 1);
                    } else if (two) {
                        mma<PAIR>(tmem + BN, ad1 + 2 * k, bd + 128 * k, idesc, add);
                    }
                }
                commit<PAIR>(&aempty[s]);
                commit<PAIR>(&wempty[b]);
                if (TERMS == 2 && (i % kDrain == kDrain - 1 || i == ns - 1)) commit<PAIR>(&accf[buf]);
            }
            if (TERMS == 1 && rank == 0) commit<PAIR>(accf);
        }
    } else {
        // ---------------------------------------------------------------- dequant
        const int t = threadIdx.x - 64, group = t / kGroupThreads, u = t % kGroupThreads;
        const int r = u >> 2, j = u & 3;                       // row of the step, 32-column quarter
        const int col = k0 + rank * kCols + j * kTask;
        const bool col_in = col < p.K;
        const size_t row_bytes = static_cast<size_t>(p.K) * BITS / 8;
        const uint8_t *wp = p.W + static_cast<size_t>(col) * BITS / 8;
        const int pb = col >> p.lbs;
        const bool zt = WK == WK_NBITS && p.zp_mode == ZP_TENSOR;
        // The two quarters of a 64-column block's pair of quarters share banks:
        // quarters 2 and 3 write their chunks in the order 2 3 0 1.
        const bool swap = j >= 2;
        uint32_t off[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            off[i] = (j >> 1) * kBlockBytes + (r >> 3) * 1024 + (r & 7) * 128 + ((((j & 1) * 4 + (i ^ (swap ? 2 : 0))) ^ (r & 7)) << 4);
        auto load = [&](int i, Task<BITS> &k) {
            const int n = (s0 + i) * kBK + r;
            const bool in = i < ns && n < p.N && col_in;  // outside: codes with scale 0, weights 0
            k.par = k.zp = 0;
#pragma unroll
            for (int q = 0; q < BITS; ++q) k.c[q] = 0;
            if (!in) return;
            const uint8_t *src = wp + n * row_bytes;
            if constexpr (BITS == 2) {
                const uint2 v = __ldg(reinterpret_cast<const uint2 *>(src));
                k.c[0] = v.x, k.c[1] = v.y;
            } else {
#pragma unroll
                for (int q = 0; q < BITS / 4; ++q) {
                    const uint4 v = __ldg(reinterpret_cast<const uint4 *>(src) + q);
                    k.c[4 * q] = v.x, k.c[4 * q + 1] = v.y, k.c[4 * q + 2] = v.z, k.c[4 * q + 3] = v.w;
                }
            }
            const size_t pi = static_cast<size_t>(n) * p.nb + pb;
            if constexpr (WK == WK_NBITS) {
                k.par = __ldg(static_cast<const unsigned short *>(p.par) + pi);
                if (zt) k.zp = __ldg(reinterpret_cast<const unsigned short *>(p.zp) + pi);
            } else {
                k.par = __ldg(static_cast<const unsigned int *>(p.par) + pi);
            }
        };
        const float *lut_lane = lut + lane;
        const uint32_t zpu = __half_as_ushort(__float2half_rn(p.zpv)) * 0x10001u;
        const int sub = warp & 3, cq = (warp - 2) >> 2;  // tensor-memory sub-partition; share of the columns
        constexpr int CW = H * BN / (kDequantWarps / 4);
        const uint32_t lane_addr = tmem + (static_cast<uint32_t>(sub * 32) << 16);
        float taken[TERMS == 2 ? CW : 1];  // TERMS = 2: the sums so far of this lane's row, CW columns
        int blocks_taken = 0;
        if constexpr (TERMS == 2)
            for (int q = 0; q < CW; ++q) taken[q] = 0.f;
        auto take = [&]() {
            const int buf = blocks_taken & 1;
            const bool here = mbar_wait(&accf[buf], (blocks_taken >> 1) & 1, abort_flag, p.fault, FAULT_WAIT_TC);
            if (!__all_sync(0xffffffffu, here)) return false;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < CW; c += 32) {
                uint32_t v[32];
                tmem_ld32(lane_addr + buf * BN + cq * CW + c, v);
#pragma unroll
                for (int q = 0; q < 32; ++q) taken[TERMS == 2 ? c + q : 0] += __uint_as_float(v[q]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (PAIR == 1) mbar_arrive(&drained[buf]);  // (its cluster is other CTAs of the tile)
                else arrive_leader(&drained[buf]);
            }
            ++blocks_taken;
            return true;
        };
        float wscale = 1.f;
        if constexpr (TERMS == 2) wscale = exp2i(weight_exponent(p.maxima, WK == WK_CODEBOOK, BITS, zt, p.zpv));
        Task<BITS> next;
        load(group, next);
        for (int i = group; i < ns; i += kGroups) {
            if constexpr (TERMS == 2) {
                while (blocks_taken + 2 <= i / kDrain && ok) ok = take();  // the MMAs are at the other accumulator
                if (!ok) break;
            }
            Task<BITS> k = next;
            load(i + kGroups, next);
            const int b = i % NW;
            if (!mbar_wait(&wempty[b], ((i / NW) & 1) ^ 1, abort_flag, p.fault, FAULT_WAIT_TC)) break;
            if (swap) {
#pragma unroll
                for (int q = 0; q < BITS / 2; ++q) {
                    const uint32_t x = k.c[q];
                    k.c[q] = k.c[q + BITS / 2];
                    k.c[q + BITS / 2] = x;
                }
            }
            unsigned char *ws = w_s + b * WT;
            if constexpr (TERMS == 2) {
                const float par = (WK == WK_CODEBOOK ? __uint_as_float(k.par) : h2f(static_cast<uint16_t>(k.par))) * wscale;
                const float zp = zt ? h2f(static_cast<uint16_t>(k.zp)) : p.zpv;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float w[8], l[8];
                    uint32_t h[4];
                    weights8<WK, BITS>(k.c, q, zp, par, lut_lane, w);
#pragma unroll
                    for (int e = 0; e < 4; ++e) h[e] = half_pair(w[2 * e], w[2 * e + 1], l[2 * e], l[2 * e + 1]);
                    *reinterpret_cast<uint4 *>(ws + off[q]) = make_uint4(h[0], h[1], h[2], h[3]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) h[e] = h2_as_u32(__floats2half2_rn(l[2 * e], l[2 * e + 1]));
                    *reinterpret_cast<uint4 *>(ws + kWBytes + off[q]) = make_uint4(h[0], h[1], h[2], h[3]);
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&wfull[b]);
                continue;
            }
            UnitPar up;
            up.lo = false;
            if constexpr (WK == WK_NBITS) {
                if constexpr (BF16) {
                    up.zpf = zt ? h2f(static_cast<uint16_t>(k.zp)) : p.zpv;
                    up.sf = h2f(static_cast<uint16_t>(k.par));
                } else {
                    up.zp2 = u32_as_h2(zt ? k.zp * 0x10001u : zpu);
                    up.s2 = u32_as_h2(k.par * 0x10001u);
                }
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint4 w;
                if constexpr (WK == WK_CODEBOOK)
                    w = dequant8_codebook<BF16>(k.c[q], __uint_as_float(k.par), lut_lane);
                else if constexpr (BF16)
                    w = bf16_weights8<BITS>(k.c, q, up.sf, -__fmul_rn(up.zpf, up.sf));
                else if constexpr (BITS == 2)
                    w = dequant8_nbits<2, BF16>((k.c[q >> 1] >> (16 * (q & 1))) & 0xFFFFu, 0u, up);
                else if constexpr (BITS == 4)
                    w = dequant8_nbits<4, BF16>(k.c[q], 0u, up);
                else
                    w = dequant8_nbits<8, BF16>(k.c[2 * q], k.c[2 * q + 1], up);
                *reinterpret_cast<uint4 *>(ws + off[q]) = w;
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&wfull[b]);
        }
        // ---------------------------------------------------------------- epilogue
        if constexpr (TERMS == 2) {
            while (blocks_taken * kDrain < ns && ok) ok = take();
        } else {
            ok = mbar_wait(accf, 0, abort_flag, p.fault, FAULT_WAIT_TC);
        }
        tc_fence_after();
#pragma unroll 1
        for (int cc = cq * CW; cc < (cq + 1) * CW; cc += 32) {
            uint32_t v[32];
            if constexpr (TERMS == 1) tmem_ld32(lane_addr + cc, v);
            const int h = cc / BN, c0 = cc - h * BN;
            const int row = h * PAIR * kRows + rank * kRows + sub * 32 + lane, m = m0 + row, kc = k0 + c0;
            if (m >= p.M || kc >= p.K) continue;  // K is a multiple of 32: a column group is in or out
            if (!ok || ns == 0) {
                if (!shared_tile) continue;
#pragma unroll
                for (int q = 0; q < 32; ++q) v[q] = 0;
            }
            if constexpr (TERMS == 2) {
                // The row's and the weights' powers of two are undone together, in two equal steps: one of them alone
                // may leave fp32's range where the result does not.
                const int e = static_cast<int>(__float_as_uint(p.row_scale[m]) >> 23) - static_cast<int>(__float_as_uint(wscale) >> 23);
                const float half = exp2i(e / 2), rest = exp2i(e - e / 2);
#pragma unroll
                for (int q = 0; q < 32; ++q) v[q] = __float_as_uint(taken[cc - cq * CW + q] * half * rest);
            }
            if (shared_tile) {
                float4 *dst = reinterpret_cast<float4 *>(sums + row * SS + c0);
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    dst[q] = make_float4(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1]), __uint_as_float(v[4 * q + 2]),
                                         __uint_as_float(v[4 * q + 3]));
            } else if (piece >= 0) {
                float4 *dst = reinterpret_cast<float4 *>(p.partial + (static_cast<size_t>(piece) * (H * PAIR * kRows) + row) * BN + c0);
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    dst[q] = make_float4(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1]), __uint_as_float(v[4 * q + 2]),
                                         __uint_as_float(v[4 * q + 3]));
            } else if (p.x_dtype == 0) {
                float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(p.dX) + static_cast<size_t>(m) * p.K + kc);
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    dst[q] = make_float4(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1]), __uint_as_float(v[4 * q + 2]),
                                         __uint_as_float(v[4 * q + 3]));
            } else {
                uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.dX) + static_cast<size_t>(m) * p.K + kc);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t o[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float lo = __uint_as_float(v[8 * q + 2 * e]), hi = __uint_as_float(v[8 * q + 2 * e + 1]);
                        o[e] = p.x_dtype == 1 ? (static_cast<uint32_t>(f2h(hi)) << 16) | f2h(lo)
                                              : (static_cast<uint32_t>(f2bf(hi)) << 16) | f2bf(lo);
                    }
                    dst[q] = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    if constexpr (PAIR == 2) cluster_sync();  // the peer's MMAs and arrivals are done with this CTA's memory
    else __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        free_tmem<PAIR>(tmem, TMEM_COLS);
        __syncwarp();
    }
    if (shared_tile) {
        cluster_sync();  // every CTA's sums are written
        const int rows = min(kRows, p.M - m0), cols = min(kCols, p.K - k0) / 4;
        const int lo = rows * part / p.splits, hi = rows * (part + 1) / p.splits;
        for (int e = threadIdx.x; e < (hi - lo) * cols; e += kThreads) {
            const int row = lo + e / cols, c = (e % cols) * 4;
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int z = 0; z < p.splits; ++z) {
                const float4 v = peer_float4(sums + row * SS + c, z);
                s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
            }
            store4(p.dX, p.x_dtype, static_cast<size_t>(m0 + row) * p.K + k0 + c, s);
        }
        cluster_sync();  // and read
    }
}

// dX of the split tiles: their pieces in order, four columns a thread.
__global__ void __launch_bounds__(256) dgrad_reduce_kernel(const float *__restrict__ partial, int tiles, int splits, int rows, int bn,
                                                           int first, int mt, int M, int K, void *dX, int x_dtype) {
    pdl_wait();
    pdl_launch_dependents();
    const int per = rows * (bn / 4);
    const int64_t total = static_cast<int64_t>(tiles) * per;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
        const int q = static_cast<int>(i / per), e = static_cast<int>(i - static_cast<int64_t>(q) * per);
        const int row = e / (bn / 4), c = (e - row * (bn / 4)) * 4, tile = first + q;
        const int m = (tile % mt) * rows + row, k = (tile / mt) * bn + c;
        if (m >= M || k >= K) continue;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int z = 0; z < splits; ++z) {
            const float4 v = *reinterpret_cast<const float4 *>(partial + ((static_cast<size_t>(q) * splits + z) * rows + row) * bn + c);
            s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
        store4(dX, x_dtype, static_cast<size_t>(m) * K + k, s);
    }
}

// dY with its rows at 16-byte boundaries (the TMA's rule), for N that is no multiple of 8.
__global__ void __launch_bounds__(256) pad_rows_kernel(const uint16_t *__restrict__ src, int N, int ld, uint16_t *__restrict__ dst) {
    pdl_wait();
    pdl_launch_dependents();
    const size_t row = blockIdx.x;
    for (int n = threadIdx.x; n < ld; n += 256) dst[row * ld + n] = n < N ? src[row * N + n] : 0;
}

// ------------------------------------------------------------------ plain fp32 tiles
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

// ------------------------------------------------------------------ host side
struct Plan {
    int pair, h, terms, rows, bn, mt, kt, steps;
    int full_tiles, tail_tiles, splits, split_steps;
    size_t partial_bytes, copy_bytes, front_bytes;  // pieces; one 16-bit copy of dY; everything before the pieces
    int ld;
};

// Rows decide the tile: up to 128 rows one CTA a tile (128 x 128), up to 256 a
// pair (256 x 256), above that two halves a pair (512 x 256; fp32 dY needs the
// second half's room for its second term).  Of the pairs' tiles whole ones fill
// complete waves and the others are split along n over the SMs, at least four
// steps a piece.
Plan make_plan(int dy_dtype, int M, int N, int K) {
    Plan c{};
    c.terms = dy_dtype == 0 ? 2 : 1;
    c.pair = M <= kRows ? 1 : 2;
    c.h = M <= 2 * kRows || c.terms == 2 ? 1 : 2;
    c.rows = c.pair * c.h * kRows;
    c.bn = c.pair * kCols;
    c.mt = (M + c.rows - 1) / c.rows;
    c.kt = (K + c.bn - 1) / c.bn;
    c.steps = (N + kBK - 1) / kBK;
    const int units = device_info().sm_count / c.pair;
    const int64_t tiles = static_cast<int64_t>(c.mt) * c.kt;
    c.full_tiles = static_cast<int>(tiles / units * units);
    c.tail_tiles = static_cast<int>(tiles - c.full_tiles);
    c.splits = 1;
    c.split_steps = c.steps;
    if (c.pair == 1) {  // every tile is shared by a cluster of as many CTAs as leave each two steps and all of them resident
        c.full_tiles = 0;
        c.tail_tiles = static_cast<int>(tiles);
        while (c.splits < 16 && tiles * c.splits * 2 <= units && c.steps >= 4 * c.splits) c.splits *= 2;
        c.split_steps = (c.steps + c.splits - 1) / c.splits;
    } else if (c.tail_tiles) {
        const int sp = std::max(1, std::min(units / c.tail_tiles, c.steps / 4));
        c.split_steps = (c.steps + sp - 1) / sp;
        c.splits = (c.steps + c.split_steps - 1) / c.split_steps;
    }
    if (c.pair == 2 && c.splits > 1) c.partial_bytes = sizeof(float) * static_cast<size_t>(c.tail_tiles) * c.splits * static_cast<size_t>(c.rows) * c.bn;
    c.ld = (N + 7) / 8 * 8;
    if (c.ld != N || c.terms == 2) c.copy_bytes = (static_cast<size_t>(M) * c.ld * 2 + 255) / 256 * 256;
    c.front_bytes = c.terms * c.copy_bytes;
    if (c.terms == 2) c.front_bytes += (static_cast<size_t>(M) * 4 + 255) / 256 * 256 + 2 * kMaxBlocks * 4;
    return c;
}

// 3-bit codes take the plain kernel.
bool tensor_cores(int bits) { return bits != 3 && encode_fn() != nullptr; }

template <int WK, int BITS, bool BF16, int PAIR, int H, int TERMS = 1>
cudaError_t launch(const CUtensorMap *maps, DgradArgs a, int tiles, cudaStream_t s) {
    auto kern = dgrad_kernel<WK, BITS, BF16, PAIR, H, TERMS>;
    static std::atomic<unsigned long long> configured{0};
    const int slot = device_slot();
    const unsigned long long bit = slot < 0 ? 0 : 1ull << slot;
    if (!(configured.load(std::memory_order_acquire) & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(H, TERMS));
        if (e != cudaSuccess) return e;
        if (PAIR == 1) {
            const cudaError_t e16 = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e16 != cudaSuccess) return e16;
        }
        configured.fetch_or(bit, std::memory_order_acq_rel);
    }
    if (PAIR == 1) {  // fewer CTAs a tile where so many cannot be a cluster
        static ClusterFit fit;
        const int splits = fitting_cluster(reinterpret_cast<const void *>(kern), fit, a.splits, kThreads, smem_bytes(H, TERMS));
        if (splits != a.splits) {
            tiles = tiles / a.splits * splits;
            a.splits = splits;
            a.split_steps = (a.steps + splits - 1) / splits;
        }
    }
    return launch_cluster(kern, dim3(tiles * PAIR), dim3(kThreads), smem_bytes(H, TERMS), s, PAIR == 1 ? a.splits : PAIR, maps[0], maps[1], a);
}

template <int WK, int BITS, bool BF16>
cudaError_t launch_shape(const Plan &c, const CUtensorMap *maps, const DgradArgs &a, cudaStream_t s) {
    const int tiles = c.full_tiles + c.tail_tiles * c.splits;
    if constexpr (!BF16)
        if (c.terms == 2) return c.pair == 1 ? launch<WK, BITS, false, 1, 1, 2>(maps, a, tiles, s) : launch<WK, BITS, false, 2, 1, 2>(maps, a, tiles, s);
    if (c.pair == 1) return launch<WK, BITS, BF16, 1, 1>(maps, a, tiles, s);
    return c.h == 1 ? launch<WK, BITS, BF16, 2, 1>(maps, a, tiles, s) : launch<WK, BITS, BF16, 2, 2>(maps, a, tiles, s);
}

template <bool BF16>
cudaError_t launch_kind(const GemmProblem &p, const Plan &c, const CUtensorMap *maps, const DgradArgs &a, cudaStream_t s) {
    if (p.kind == WK_CODEBOOK) return launch_shape<WK_CODEBOOK, 4, BF16>(c, maps, a, s);
    if (p.bits == 2) return launch_shape<WK_NBITS, 2, BF16>(c, maps, a, s);
    if (p.bits == 4) return launch_shape<WK_NBITS, 4, BF16>(c, maps, a, s);
    return launch_shape<WK_NBITS, 8, BF16>(c, maps, a, s);
}

}  // namespace

size_t dgrad_workspace_bytes(int dy_dtype, int M, int N, int K, int bits) {
    if (!tensor_cores(bits)) return 0;
    const Plan c = make_plan(dy_dtype, M, N, K);
    return c.front_bytes + c.partial_bytes;
}

cudaError_t dgrad(const GemmProblem &p, void *ws, cudaStream_t s) {
    if (!tensor_cores(p.bits)) {
        const cudaError_t e = launch_pdl(dgrad_simple_kernel, dim3((p.K + 63) / 64, (p.M + 63) / 64), dim3(256), 0, s, p);
        return e != cudaSuccess ? e : cudaGetLastError();
    }
    const Plan c = make_plan(p.a_dtype, p.M, p.N, p.K);
    char *w = static_cast<char *>(ws);
    const void *dy[2] = {p.A, p.A};  // the terms that the tensor maps read
    float *row_scale = nullptr, *maxima = nullptr;
    cudaError_t e = cudaSuccess;
    if (c.terms == 2) {
        dy[0] = w;
        dy[1] = w + c.copy_bytes;
        maxima = reinterpret_cast<float *>(w + 2 * c.copy_bytes);
        row_scale = maxima + 2 * kMaxBlocks;
        e = launch_pdl(split_dy_kernel, dim3(p.M + kMaxBlocks), dim3(256), 0, s, p, c.ld, reinterpret_cast<__half *>(w),
                       reinterpret_cast<__half *>(w + c.copy_bytes), row_scale, maxima);
    } else if (c.copy_bytes) {
        dy[0] = dy[1] = w;
        e = launch_pdl(pad_rows_kernel, dim3(p.M), dim3(256), 0, s, static_cast<const uint16_t *>(p.A), p.N, c.ld, static_cast<uint16_t *>(ws));
    }
    if (e != cudaSuccess) return e;
    CUtensorMap maps[2];
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(c.ld), static_cast<cuuint64_t>(p.M)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(c.ld) * 2};
    const cuuint32_t box[2] = {kBK, kRows}, es[2] = {1, 1};
    for (int i = 0; i < 2; ++i)
        if (encode_fn()(&maps[i], p.a_dtype == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                        const_cast<void *>(dy[i]), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    DgradArgs a{};
    a.W = p.W;
    a.par = p.kind == WK_CODEBOOK ? static_cast<const void *>(p.absmax) : static_cast<const void *>(p.scales);
    a.zp = p.zp;
    a.zp_mode = p.zp_mode;
    a.zpv = p.uniform_zp;
    a.codebook = p.codebook;
    a.dX = p.Y;
    a.x_dtype = p.y_dtype;
    a.partial = reinterpret_cast<float *>(w + c.front_bytes);
    a.row_scale = row_scale;
    a.maxima = maxima;
    a.M = p.M;
    a.N = p.N;
    a.K = p.K;
    a.nb = p.K / p.bs;
    a.lbs = 31 - __builtin_clz(static_cast<unsigned>(p.bs));
    a.steps = c.steps;
    a.mt = c.mt;
    a.full_tiles = c.full_tiles;
    a.splits = c.splits;
    a.split_steps = c.split_steps;
    a.fault = fault_word();
    e = p.a_dtype == 2 ? launch_kind<true>(p, c, maps, a, s) : launch_kind<false>(p, c, maps, a, s);
    if (e != cudaSuccess) return e;
    if (c.pair == 2 && c.splits > 1) {
        const int64_t work = static_cast<int64_t>(c.tail_tiles) * c.rows * (c.bn / 4);
        e = launch_pdl(dgrad_reduce_kernel, dim3(static_cast<unsigned>(std::min<int64_t>((work + 255) / 256, device_info().sm_count * 16))),
                       dim3(256), 0, s, static_cast<const float *>(a.partial), c.tail_tiles, c.splits, c.rows, c.bn, c.full_tiles, c.mt, p.M, p.K,
                       p.Y, p.y_dtype);
        if (e != cudaSuccess) return e;
    }
    return cudaGetLastError();
}

}  // namespace qg
