// qg_tc_common.cuh -- what the tensor-core kernels share: tcgen05 / TMA
// primitives, operand descriptors and the tensor-map encoder's address.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "qg_device.cuh"

namespace qg {

// cuTensorMapEncodeTiled of the loaded driver (null: too old); qg_tc.cu
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();

__device__ __forceinline__ void tma_load_2d(void *dst, const CUtensorMap *map, int x, int y, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
}

// 4 bytes global -> shared, asynchronous; src_bytes 0 writes zeros (nothing is read)
__device__ __forceinline__ void cp_async4(void *dst, const void *src, uint32_t src_bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(src_bytes)
                 : "memory");
}

// one arrival on `bar` once every cp.async this thread issued before has landed
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void tmem_alloc(uint32_t *slot, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

__device__ __forceinline__ void umma_f16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(
            d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void umma_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Shared-memory matrix descriptor: K-major operand, 128-byte swizzle, 8-row
// groups 1024 bytes apart (start address, leading / stride byte offsets in
// 16-byte units, descriptor version 1, swizzle mode 2 = 128B).
__device__ __forceinline__ uint64_t sdesc_k128(uint32_t saddr) {
    uint64_t d = static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(1) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

// Instruction descriptor, kind::f16: fp32 accumulator, A/B fp16 or bf16,
// both K-major, N >> 3 at bit 17, M >> 4 at bit 24.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool bf16) {
    return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(M >> 4) << 24);
}

// 128-byte swizzle: 16-byte chunk c of row r (8 rows per 1024-byte atom)
__device__ __forceinline__ uint32_t swz128(int r, int c) {
    return static_cast<uint32_t>((r >> 3) * 1024 + (r & 7) * 128 + ((c ^ (r & 7)) << 4));
}

__device__ __forceinline__ uint32_t h2_as_u32(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ __half2 u32_as_h2(uint32_t u) { return *reinterpret_cast<__half2 *>(&u); }

// Block parameters of one 8-weight unit: fp16 pairs for the fp16 operand,
// fp32 values for the bf16 operand.
struct UnitPar {
    __half2 zp2, s2;  // fp16 operand
    float zpf, sf;    // bf16 operand
    bool lo;          // fp16 operand: the residual part of the weight
};

// One operand pair from two exact integer codes q (an fp16 pair).
//  fp16: (q - zp) * s with packed fp16 arithmetic.  For the integer and
//        half-integer zero points of the workloads q - zp is exact, so the
//        pair is the single fp16 rounding of the exact product.
//  bf16: the fp32 weight fl32(fl32(q - zp) * s) (two fp32 round-to-nearest
//        operations, no contraction), then one round-to-nearest to bf16.  No
//        fp16 intermediate, so products beyond fp16's range or below its
//        normal range keep bf16's.
template <bool BF16>
__device__ __forceinline__ uint32_t operand_pair(__half2 q, const UnitPar &u) {
    if constexpr (BF16) {
        const float2 qf = __half22float2(q);
        const float w0 = __fmul_rn(__fsub_rn(qf.x, u.zpf), u.sf);
        const float w1 = __fmul_rn(__fsub_rn(qf.y, u.zpf), u.sf);
        const __nv_bfloat162 b = __floats2bfloat162_rn(w0, w1);
        return *reinterpret_cast<const uint32_t *>(&b);
    } else {
        if (!u.lo) return h2_as_u32(__hmul2(__hsub2(q, u.zp2), u.s2));
        // the residual: w (exact in fp32) minus its fp16 rounding, rounded to fp16
        const float2 qf = __half22float2(q);
        const float zf = __low2float(u.zp2), sf = __low2float(u.s2);
        const float w0 = __fmul_rn(__fsub_rn(qf.x, zf), sf), w1 = __fmul_rn(__fsub_rn(qf.y, zf), sf);
        const __half2 hi = __floats2half2_rn(w0, w1);
        return h2_as_u32(__floats2half2_rn(w0 - __low2float(hi), w1 - __high2float(hi)));
    }
}

// 8 weights (k = 8c .. 8c+7 of one row) from their packed codes, as four
// operand pairs: the codes are first turned into exact fp16 integers, then
// operand_pair applies the zero point and the scale.
template <int BITS, bool BF16>
__device__ __forceinline__ uint4 dequant8_nbits(uint32_t codes, uint32_t codes_hi, const UnitPar &u) {
    uint32_t out[4];
    if constexpr (BITS == 8) {
        // codes: 8 bytes, one code each; a byte permute puts two codes under the
        // fp16 exponent of 1024 (0x64): (1024 + q0, 1024 + q1), exact for q < 1024
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t wsrc = j < 2 ? codes : codes_hi;
            const uint32_t h = __byte_perm(wsrc, 0x64646464u, (j & 1) ? 0x4342u : 0x4140u);
            const __half2 q = __hsub2(u32_as_h2(h), __floats2half2_rn(1024.f, 1024.f));
            out[j] = operand_pair<BF16>(q, u);
        }
    } else if constexpr (BITS == 2) {
        // codes: 16 bits, 8 codes; byte j holds codes 4j .. 4j+3
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t v = __byte_perm(codes, 0u, 0x4040u | (j * 0x0101u));  // byte j into bytes 0 and 2
            const uint32_t h01 = (v & 0x000C0003u) | 0x64006400u;  // (1024 + q0, 1024 + 4 q1)
            const uint32_t h23 = (v & 0x00C00030u) | 0x64006400u;  // (1024 + 16 q2, 1024 + 64 q3)
            const __half2 q01 = __hfma2(u32_as_h2(h01), __floats2half2_rn(1.f, 0.25f), __floats2half2_rn(-1024.f, -256.f));
            const __half2 q23 = __hfma2(u32_as_h2(h23), __floats2half2_rn(0.0625f, 0.015625f), __floats2half2_rn(-64.f, -16.f));
            out[2 * j] = operand_pair<BF16>(q01, u);
            out[2 * j + 1] = operand_pair<BF16>(q23, u);
        }
    } else {
        // codes: 32 bits, 8 codes; byte j holds codes 2j, 2j+1
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t v = __byte_perm(codes, 0u, 0x4040u | (j * 0x0101u));
            const uint32_t h = (v & 0x00F0000Fu) | 0x64006400u;  // (1024 + q0, 1024 + 16 q1)
            const __half2 q = __hfma2(u32_as_h2(h), __floats2half2_rn(1.f, 0.0625f), __floats2half2_rn(-1024.f, -64.f));
            out[j] = operand_pair<BF16>(q, u);
        }
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
}

// codebook: w = C[q] * absmax (fp32), rounded to the operand type
template <bool BF16>
__device__ __forceinline__ uint4 dequant8_codebook(uint32_t codes, float am, const float *lut_lane) {
    uint32_t out[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float w0 = lut_lane[((codes >> (8 * j)) & 15u) * 32] * am;
        const float w1 = lut_lane[((codes >> (8 * j + 4)) & 15u) * 32] * am;
        if constexpr (BF16) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(w0, w1);
            out[j] = *reinterpret_cast<const uint32_t *>(&b);
        } else {
            out[j] = h2_as_u32(__floats2half2_rn(w0, w1));
        }
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
}

}  // namespace qg
