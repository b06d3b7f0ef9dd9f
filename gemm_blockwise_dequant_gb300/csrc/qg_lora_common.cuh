// qg_lora_common.cuh -- what the adapter kernels share: warp-level MMAs,
// splitting of fp32 values into operand terms, and the tiles of the requests.
//
// Two kinds of products (mma.sync; both accumulate in fp32).  Up to a rank of
// about 32 they wait for memory and latency, not for the tensor cores, and their
// operands come from global memory straight into fragments: the order of a contraction is free as long
// as both operands share it, so a lane takes 16 contiguous bytes where the
// fragment layout asks for scattered pairs.
//  * NATIVE (16-bit activations and adapters of one type): m16n8k16.  An fp32
//    factor (V, G) is split in two 16-bit terms, for fp16 after its row has been
//    scaled to [1, 2) by a power of two: 16 bits of it are kept for bf16, 22 for fp16.
//  * TF32 (fp32 activations, adapters of any type): m16n8k8.  An fp32 value is
//    split in two TF32 terms (22 bits); 16-bit values are TF32 values as they
//    are.  The product of two second terms (2^-22) is left out.
#pragma once

#include <atomic>

#include "qg_device.cuh"
#include "qg_internal.h"

namespace qg {

constexpr int kF32 = 0, kF16 = 1, kBF16 = 2;
constexpr int kMaxRank = 128;

// Raises a kernel's shared-memory limit (and allows clusters of 16) once per device.
template <typename K>
cudaError_t allow_smem(K kern, std::atomic<unsigned long long> &done, int bytes, bool clusters16 = false) {
    const int slot = device_slot();
    const unsigned long long bit = slot < 0 ? 0 : 1ull << slot;
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && clusters16) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_acq_rel);
    return e;
}

template <int T>
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (T == kBF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// x = hi + lo with both terms TF32; an infinity or NaN is its own first term.
__device__ __forceinline__ void split_tf32(float x, uint32_t &hi, uint32_t &lo) {
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi) : "f"(x));
    const float h = __uint_as_float(hi);
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(lo) : "f"(fabsf(h) < __int_as_float(0x7f800000) ? x - h : 0.f));
}

// x = hi + lo with both terms of the 16-bit type.
template <int T>
__device__ __forceinline__ void split16(float x, uint16_t &hi, uint16_t &lo) {
    hi = T == kBF16 ? f2bf(x) : f2h(x);
    const float h = T == kBF16 ? bf2f(hi) : h2f(hi);
    const float rest = fabsf(h) < __int_as_float(0x7f800000) ? x - h : 0.f;
    lo = T == kBF16 ? f2bf(rest) : f2h(rest);
}

template <int T>
__device__ __forceinline__ float to_float(uint16_t v) {
    return T == kBF16 ? bf2f(v) : h2f(v);
}

__device__ __forceinline__ uint32_t pack2(uint32_t lo, uint32_t hi) { return (lo & 0xFFFFu) | (hi << 16); }

__device__ __forceinline__ float load_elem(const void *p, int dtype, size_t i) {  // data that the call may also write
    if (dtype == kF32) return static_cast<const float *>(p)[i];
    const uint16_t v = static_cast<const uint16_t *>(p)[i];
    return dtype == kF16 ? h2f(v) : bf2f(v);
}

// A run of up to `rows` consecutive rows of one request.
struct RowTile {
    int t0, rows, adapter;  // rows 0: no such tile; adapter -1: none
};

// Tile number `tile` when every request is cut into tiles of `size` rows.  Every
// thread of the block calls it; false when the offsets break their rule (every
// block then returns; block `reporter` sets *status).
__device__ __forceinline__ bool find_tile(const LoraProblem &p, int tile, int size, bool reporter, RowTile &out) {
    __shared__ int wsum[32];
    __shared__ RowTile found;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nwarp = blockDim.x >> 5;
    if (tid == 0) found = {0, 0, -1};
    int base = 0, bad = 0, strange = 0;
    for (int s0 = 0; s0 < p.S; s0 += blockDim.x) {
        const int s = s0 + tid;
        int64_t lo = 0, hi = 0;
        int id = -1, cnt = 0;
        if (s < p.S) {
            lo = __ldg(p.offs + s), hi = __ldg(p.offs + s + 1), id = __ldg(p.ids + s);
            bad |= hi < lo || lo < 0 || hi > p.T || (s == 0 && lo != 0);
            strange |= id >= p.na;
            if (!bad) cnt = static_cast<int>((hi - lo + size - 1) / size);
        }
        int inc = cnt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        __syncthreads();  // wsum of the previous chunk is read, found is written
        if (lane == 31) wsum[warp] = inc;
        __syncthreads();
        int total = 0;
        for (int w = 0; w < nwarp; ++w) {
            if (w == warp) inc += total;
            total += wsum[w];
        }
        const int at = tile - base - (inc - cnt);
        if (at >= 0 && at < cnt) {
            const int64_t t0 = lo + static_cast<int64_t>(at) * size;
            found = {static_cast<int>(t0), static_cast<int>(hi - t0 < size ? hi - t0 : size), id < 0 || id >= p.na ? -1 : id};
        }
        base += total;
    }
    bad = __syncthreads_or(bad);
    if (reporter && p.status && (bad || strange)) *p.status = 1;
    out = found;
    return !bad;
}

// Where the 16-bit terms of G and V go: [G, V][terms][T][rank].
struct TermsOut {
    uint16_t *at;  // null: not wanted here
    int terms;
    size_t all;    // T * rank
};

// The bf16 terms of value `e` of G (which = 0) or V (1): 8 bits each; an infinity or NaN is its own first term.
__device__ __forceinline__ void put_terms(const TermsOut &o, int which, size_t e, float x) {
    for (int m = 0; m < o.terms; ++m) {
        const uint16_t h = f2bf(x);
        const float f = bf2f(h);
        x = fabsf(f) < __int_as_float(0x7f800000) ? x - f : 0.f;
        o.at[(static_cast<size_t>(which) * o.terms + m) * o.all + e] = h;
    }
}

// A lane's queue in shared memory.  A lane copies ahead exactly the bytes that it
// will read itself, so nothing but its own cp.async groups has to be waited for,
// and the loads in flight do not occupy registers.  What lies outside is written as zeros.
template <int BYTES>
__device__ __forceinline__ void queue_copy(void *dst, const void *src, bool in) {
    const uint32_t n = in ? BYTES : 0;
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(n), "n"(BYTES) : "memory");
}
// 16 bytes of a row (the values from k on, vw to a word) as four words; from value `end` on zeros.
__device__ __forceinline__ void copy_words(void *dst, const char *row, int k, int vw, int end) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const bool in = k + e * vw < end;
        queue_copy<4>(static_cast<char *>(dst) + 4 * e, row + (in ? static_cast<size_t>(k + e * vw) * (4 / vw) : 0), in);
    }
}
__device__ __forceinline__ void queue_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void queue_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// A float of CTA `rank`'s shared memory, at the place of `p` in this CTA's.
__device__ __forceinline__ float peer_float(const float *p, int rank) {
    float v;
    asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %1, %2;\n ld.shared::cluster.f32 %0, [a];\n}\n"
                 : "=f"(v)
                 : "r"(smem_u32(p)), "r"(rank)
                 : "memory");
    return v;
}

// Four of them.
__device__ __forceinline__ float4 peer_float4(const float *p, int rank) {
    float4 v;
    asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %4, %5;\n ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n}\n"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(smem_u32(p)), "r"(rank)
                 : "memory");
    return v;
}

}  // namespace qg
