/*
 * qgemm.h -- C ABI of the GB300 (sm_103a) blockwise low-bit dequantize +
 * GEMV / small-M GEMM library, and of the fused single-token QMoE decode.
 *
 *     Y[M, N] = A[M, K] . dequant(W)[N, K]^T
 *
 * Sources (web pages, cited by title and section):
 *   [hip-ep #1318]  hip-ep pull request #1318: 2-bit MatMulNBits kernels for
 *                   phi4-14B on gfx1151.
 *   [hip-ep #1328]  hip-ep pull request #1328: fused QMoE decode that picks
 *                   its tiling before computing.
 *   [bnb #1979]     bitsandbytes pull request #1979: "[ROCm] Fused 4-bit SIMT
 *                   GEMM" (NF4/FP4 codebook weights).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Every data pointer is a DEVICE pointer owned by the caller.  The library
 *    never allocates, frees or synchronises (except qg_fp16_uniform_value and
 *    qg_read_device_fault, which return a value to the host), and enqueues
 *    work on `stream` only, on the current device (`stream` must belong to
 *    it).  It keeps no per-call state between calls, so concurrent calls on
 *    different streams with disjoint outputs and workspaces are independent.
 *    One exception is device-wide: the fault word of qg_read_device_fault
 *    (below), which every call's kernels may set and which any caller's read
 *    clears.
 *  - Weight codes are packed along K, least significant bits first: element
 *    k of row n is bits [(k*bits)%8, (k*bits)%8 + bits) of byte
 *    n*(K*bits/8) + (k*bits)/8.  W is row-major [N][K*bits/8] bytes.
 *  - Per-block parameters (fp16 scales, fp16 zero points, fp32 absmax) are
 *    row-major [N][K/block_size].  fp16/bf16 tensors are passed as their
 *    16-bit patterns (uint16_t).
 *  - A is row-major and contiguous, [M][K] (the raw-pointer contract of
 *    [bnb #1979], "Technical details", raw-pointer safety).  Y is row-major
 *    [M][N] and is fully overwritten.
 *  - Alignment: A, W, scales, zero points, absmax and the workspace must be
 *    16-byte aligned; otherwise the call returns QG_ERR_INVALID_ARG.
 *  - Block sizes 32, 64, 128 and 256 are supported, with K % block_size == 0.
 *    Other block sizes (16 in particular, which [hip-ep #1328] "Notes for
 *    reviewers" reports computing every output wrongly) are refused with
 *    QG_ERR_UNSUPPORTED, never computed.
 *  - Arguments are checked on the host before anything is enqueued; a refused
 *    call launches nothing ([hip-ep #1328], "Test plan": arguments the
 *    launchers must refuse).
 *  - On entry the calling thread's pending, non-sticky CUDA error is cleared,
 *    so an earlier unrelated failure is not reported as this call's failure;
 *    after each launch the launch status is checked and returned as
 *    QG_ERR_CUDA ([hip-ep #1328], "What": clear the error state before the
 *    fused decode launches).
 *  - Results are deterministic: every reduction runs in a fixed order that
 *    depends only on the shape, never on timing, so repeated calls on the
 *    same inputs are bit-identical ([hip-ep #1328], "Why" and "Test plan":
 *    129 calls bit-identical).  Nothing is tuned or timed on live calls.
 *  - M == 0 or N == 0 is a no-op.  K == 0 writes zeros.
 *  - Kernels are launched as programmatic dependents of the preceding kernel
 *    on `stream`: their set-up (barriers, tensor memory) overlaps that
 *    kernel's tail, but no buffer of the call -- weights, block parameters,
 *    activations, expert ids, outputs -- is read or written before that kernel
 *    has completed, so stream order holds exactly as for plain launches.
 */
#ifndef QGEMM_H
#define QGEMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t / CUstream; NULL is the legacy default stream. */
typedef struct CUstream_st *qg_stream_t;

/* Status codes returned by every entry point. */
enum {
    QG_OK = 0,
    QG_ERR_INVALID_ARG = 1,          /* null/misaligned pointer, bad size, K % block_size != 0 */
    QG_ERR_UNSUPPORTED = 2,          /* valid request this library does not implement (bits, block size, dtype combination) */
    QG_ERR_CUDA = 3,                 /* a CUDA launch or copy failed; the CUDA error stays readable via cudaGetLastError */
    QG_ERR_WORKSPACE_TOO_SMALL = 4   /* workspace_bytes below what *_workspace_bytes() returned for this shape */
};

/* Element types of A and Y. */
enum { QG_F32 = 0, QG_F16 = 1, QG_BF16 = 2 };

/*
 * qgemm_nbits -- MatMulNBits: per-block fp16 scale and fp16 zero point.
 *   [hip-ep #1318] "What", Commit 1 (u2 GEMV and WMMA kernels templated on
 *   the A/C element types, reading fp32 A and writing fp32 C directly) and
 *   "Performance", Model (block 64, fp16 scales and zero points).
 *
 *   w[n][k] = (q[n][k] - zp[n][k/bs]) * s[n][k/bs], computed exactly in fp32;
 *   Y[m][n] = sum_k A[m][k] * w[n][k], accumulated in fp32 (tensor-core path:
 *   the weight is rounded to A's 16-bit type before the product; fp32
 *   activations on the tensor cores -- M >= 16, fp32 Y -- go in split
 *   precision: A and w each as two fp16 terms, three products) and rounded
 *   once to y_dtype.
 *
 *   A            [M][K], a_dtype (QG_F32, QG_F16 or QG_BF16)
 *   W            [N][K*bits/8] packed codes, bits = 2, 3, 4 or 8 (the u2 / u3 / u4 /
 *                "Wi8" MatMulNBits leaves of the hip-ep #1318 kernel test table;
 *                3-bit codes run on the SIMT path for every M, a code may continue
 *                into the next byte; 8-bit: one code per byte, midpoint 128 by
 *                default); other widths are refused with QG_ERR_UNSUPPORTED
 *   scales_f16   [N][K/block_size] fp16 patterns
 *   zero_points_f16  [N][K/block_size] fp16 patterns, or NULL for the
 *                midpoint 2^(bits-1)
 *   Y            [M][N], y_dtype
 *   workspace    device scratch of at least
 *                qgemm_workspace_bytes(a_dtype, M, N, K, bits, block_size)
 *                bytes (NULL allowed when that is 0); its contents on entry
 *                do not matter and are garbage on return.  For fp32
 *                activations with M >= 16 that size includes room for the
 *                split-precision activations (4 M K bytes); a smaller
 *                workspace that still covers the call's other needs is
 *                accepted and takes a slower path (fp32 row groups).
 *   Returns a QG_* status.
 */
int qgemm_nbits(const void *A, int a_dtype, const uint8_t *W, const uint16_t *scales_f16,
                const uint16_t *zero_points_f16, void *Y, int y_dtype, int M, int N, int K, int bits,
                int block_size, void *workspace, size_t workspace_bytes, qg_stream_t stream);

/*
 * qgemm_nbits_uniform_zp -- as qgemm_nbits, with every zero point equal to
 * the scalar `uniform_zp` ([hip-ep #1318] "What", Commit 1:
 * hip_matmul_nbits_ex(..., float uniform_zp); "Why": fp16 zero points that
 * are all 1.5 cost as many bytes per token as the scales).  The zero-point
 * tensor is never read.  Bit-identical to qgemm_nbits with a full zero-point
 * tensor holding the fp16 value uniform_zp.
 */
int qgemm_nbits_uniform_zp(const void *A, int a_dtype, const uint8_t *W, const uint16_t *scales_f16,
                           float uniform_zp, void *Y, int y_dtype, int M, int N, int K, int bits,
                           int block_size, void *workspace, size_t workspace_bytes, qg_stream_t stream);

/*
 * qgemm_codebook4 -- NF4/FP4-style weights: a 4-bit code selects one of 16
 * fp32 codebook entries, multiplied by the block's fp32 absmax.
 *   [bnb #1979] "Summary" (NF4/FP4 weights decoded inside the GEMM, decoded
 *   values reused across the M rows) and "Technical details" (centroid
 *   lookup).
 *
 *   w[n][k] = codebook16[q[n][k]] * absmax[n][k/bs]   (fp32)
 *   codebook16  16 fp32 entries (device)
 *   absmax      [N][K/block_size] fp32
 *   Other arguments as qgemm_nbits (bits is 4).
 */
int qgemm_codebook4(const void *A, int a_dtype, const uint8_t *W, const float *codebook16, const float *absmax,
                    void *Y, int y_dtype, int M, int N, int K, int block_size, void *workspace,
                    size_t workspace_bytes, qg_stream_t stream);

/* Workspace bytes the two GEMM entry points need for this shape (same value
 * for qgemm_nbits, qgemm_nbits_uniform_zp and, with bits = 4,
 * qgemm_codebook4).  0 means no workspace is needed. */
size_t qgemm_workspace_bytes(int a_dtype, int M, int N, int K, int bits, int block_size);

/*
 * qmoe_decode_fused -- one token through the top-k experts of a quantized
 * MoE layer: fc1 GEMV, SwiGLU, fc2 GEMV, weighted sum over the k slots.
 *   [hip-ep #1328] "Summary" and "What" (hip_qmoe_decode_fused with
 *   num_experts; u4 weights; block 32/64/128; zero points and bias
 *   optional, "Test plan"); [hip-ep #1318] "Why" (the SwiGLU chain gate ->
 *   sigmoid -> multiplies -> up).
 *
 *   For slot j = 0..k-1 in order, e = expert_ids[j]:
 *     g = dequant(fc1[e]) . x + fc1_bias[e]                 (2*inter values)
 *     gate, up = g[0:inter], g[inter:2*inter]  (swiglu_interleaved = 0)
 *              = g[0::2],    g[1::2]           (swiglu_interleaved = 1)
 *     h = silu(gate) * up                                    (kept in fp32)
 *     o = dequant(fc2[e]) . h + fc2_bias[e]                  (hidden values)
 *   y = round_to_fp16( sum_j expert_weights[j] * o_j ), summed in slot order.
 *
 *   x_f16        [hidden] fp16
 *   expert_ids   [k] int32 (device); an id outside [0, num_experts) adds
 *                nothing and sets *status_dev to 1 (status_dev may be NULL)
 *   expert_weights [k] fp32 (device)
 *   fc1_w        [num_experts][2*inter][hidden*bits/8]
 *   fc1_scales   [num_experts][2*inter][hidden/block_size] fp16
 *   fc1_zp       same shape as fc1_scales, or NULL (midpoint 2^(bits-1))
 *   fc1_bias     [num_experts][2*inter] fp16, or NULL
 *   fc2_w        [num_experts][hidden][inter*bits/8]
 *   fc2_scales   [num_experts][hidden][inter/block_size] fp16
 *   fc2_zp       same shape as fc2_scales, or NULL
 *   fc2_bias     [num_experts][hidden] fp16, or NULL
 *   bits         4 (2 is accepted too)
 *   block_size   32, 64, 128 or 256; hidden and inter multiples of it
 *   y_f16        [hidden] fp16 output
 *   status_dev   device int written with 0 (all ids valid) or 1, or NULL
 *   workspace    at least qmoe_decode_workspace_bytes(k, hidden, inter) bytes
 *                of device memory, 16-byte aligned (QG_ERR_INVALID_ARG
 *                otherwise): the fc1 output g [k][2*inter] fp32 first, then,
 *                at the next multiple of 256 bytes, the slot outputs o
 *                [k][hidden] fp32.  Needs no initial contents; the call
 *                overwrites it.
 */
int qmoe_decode_fused(const uint16_t *x_f16, const int32_t *expert_ids, const float *expert_weights, int k,
                      int num_experts, const uint8_t *fc1_w, const uint16_t *fc1_scales, const uint16_t *fc1_zp,
                      const uint16_t *fc1_bias, const uint8_t *fc2_w, const uint16_t *fc2_scales,
                      const uint16_t *fc2_zp, const uint16_t *fc2_bias, int hidden, int inter, int bits,
                      int block_size, int swiglu_interleaved, uint16_t *y_f16, int *status_dev, void *workspace,
                      size_t workspace_bytes, qg_stream_t stream);

size_t qmoe_decode_workspace_bytes(int k, int hidden, int inter);

/*
 * qmoe_decode_fused_dp4a -- the same decode with int8 activations.
 * [hip-ep #1328] "Summary" (a dp4a form of the fused decode exists beside the fp one), "Test
 * plan" (fp and dp4a x block size x zero points x bias).  The pages do not
 * give the activation quantization; this library's reading: each activation
 * vector (x before fc1, h = silu(gate) * up before fc2) is quantized per block
 * of block_size values along the contraction,
 *     a = max |v|,  sx = fl32(a / 127),  q8 = clamp(rint(fl32(v / sx)), -127, 127)
 * (ties to even; an all-zero block gives sx = 0, q8 = 0), and each output is
 *     sum_b s[r][b] * sx[b] * ( sum_{k in b} q8[k] * q[r][k] - zp[r][b] * sum_{k in b} q8[k] )
 * with exact integer sums, plus the bias.  Results therefore differ from
 * qmoe_decode_fused by the activation quantization error (about 1/254 of each
 * block's largest magnitude per element).
 *
 * Arguments, layouts, statuses and the workspace size are those of
 * qmoe_decode_fused; in addition hidden and inter must be at most 65536
 * (QG_ERR_UNSUPPORTED otherwise).  Deterministic: repeated calls are
 * bit-identical.
 */
int qmoe_decode_fused_dp4a(const uint16_t *x_f16, const int32_t *expert_ids, const float *expert_weights, int k,
                           int num_experts, const uint8_t *fc1_w, const uint16_t *fc1_scales, const uint16_t *fc1_zp,
                           const uint16_t *fc1_bias, const uint8_t *fc2_w, const uint16_t *fc2_scales,
                           const uint16_t *fc2_zp, const uint16_t *fc2_bias, int hidden, int inter, int bits,
                           int block_size, int swiglu_interleaved, uint16_t *y_f16, int *status_dev, void *workspace,
                           size_t workspace_bytes, qg_stream_t stream);

/*
 * qmoe_decode_fused_noalloc -- qmoe_decode_fused for callers that cannot
 * allocate device memory (a decode loop inside a runtime that forbids
 * allocation on its hot path, an embedded host that must not allocate after
 * start-up, a C caller without an allocator).  The source pages have no
 * counterpart: this is an addition of this library.
 *
 * Same arguments and results as qmoe_decode_fused, minus the workspace: the
 * scratch is a fixed device array of QG_QMOE_NOALLOC_SCRATCH_BYTES inside the
 * library, held by every GPU that loads it until the process exits.  Shapes
 * needing more, i.e. qmoe_decode_workspace_bytes(k, hidden, inter) >
 * QG_QMOE_NOALLOC_SCRATCH_BYTES, are refused with QG_ERR_UNSUPPORTED before
 * anything is enqueued.  Calls no cudaMalloc, cudaFree or other allocator.
 *  - The first call on a device looks up the array's device address (once
 *    per device, with that device current); make that first call before any
 *    stream capture.  Like every entry point it works on the current device:
 *    `stream` must belong to it.
 *  - All calls on a device share the one array: calls that can overlap on
 *    the GPU (unordered streams) race.  The array keeps the last call's
 *    contents; no call depends on them.
 */
#define QG_QMOE_NOALLOC_SCRATCH_BYTES (1u << 20)
int qmoe_decode_fused_noalloc(const uint16_t *x_f16, const int32_t *expert_ids, const float *expert_weights, int k,
                              int num_experts, const uint8_t *fc1_w, const uint16_t *fc1_scales,
                              const uint16_t *fc1_zp, const uint16_t *fc1_bias, const uint8_t *fc2_w,
                              const uint16_t *fc2_scales, const uint16_t *fc2_zp, const uint16_t *fc2_bias,
                              int hidden, int inter, int bits, int block_size, int swiglu_interleaved,
                              uint16_t *y_f16, int *status_dev, qg_stream_t stream);

/*
 * qg_fp16_uniform_value -- detect an fp16 tensor whose elements all have the
 * same bit pattern ([hip-ep #1318] "What", Commit 1: the runtime detects an
 * all-equal fp16 zero-point tensor once per buffer and then passes it as a
 * scalar).  +0 and -0 differ; a NaN pattern is reported as not uniform; an
 * empty tensor is not uniform.  Enqueues one kernel on `stream`, then
 * synchronises the stream and writes *is_uniform (0/1) and, when uniform,
 * *value (host pointers).  workspace: at least 16 bytes of device memory.
 */
int qg_fp16_uniform_value(const uint16_t *t, size_t n, int *is_uniform, float *value, void *workspace,
                          size_t workspace_bytes, qg_stream_t stream);

/*
 * Dequantize to fp32 [N][K] (device), bit-exact with the definitions above.
 * Used to check unpacking and dequantization in isolation, and as the
 * "dequantize then dense GEMM" building block.
 *   qg_dequant_nbits: zero_points_f16 may be NULL (midpoint).
 */
int qg_dequant_nbits(const uint8_t *W, const uint16_t *scales_f16, const uint16_t *zero_points_f16, float *out,
                     int N, int K, int bits, int block_size, qg_stream_t stream);
int qg_dequant_nbits_uniform_zp(const uint8_t *W, const uint16_t *scales_f16, float uniform_zp, float *out, int N,
                                int K, int bits, int block_size, qg_stream_t stream);
int qg_dequant_codebook4(const uint8_t *W, const float *codebook16, const float *absmax, float *out, int N, int K,
                         int block_size, qg_stream_t stream);

/*
 * qgemm_codebook4_nested -- qgemm_codebook4 with a nested ("double-quantized")
 * absmax.  [bnb #1979] "Testing plan": nested / non-nested absmax; the pages
 * do not give the format, this library's reading:
 *   absmax[i] = fl32( fl32(absmax_table256[absmax_q[i]] * absmax2[i / nested_block]) + absmax_offset )
 * over the flat row-major index i = n * (K/block_size) + b; then exactly as
 * qgemm_codebook4 with that absmax.
 *
 *   absmax_q         [N][K/block_size] uint8 codes (device)
 *   absmax_table256  [256] fp32 (device, 4-byte aligned)
 *   absmax2          [ceil(N*(K/block_size) / nested_block)] fp32 (device, 4-byte aligned)
 *   absmax_offset    fp32 scalar (not NaN); nested_block >= 1 (bitsandbytes uses 256)
 *   Other arguments as qgemm_codebook4.  The expanded absmax is written to the
 *   front of the workspace (at least qgemm_codebook4_nested_workspace_bytes()).
 */
int qgemm_codebook4_nested(const void *A, int a_dtype, const uint8_t *W, const float *codebook16,
                           const uint8_t *absmax_q, const float *absmax_table256, const float *absmax2,
                           float absmax_offset, int nested_block, void *Y, int y_dtype, int M, int N, int K,
                           int block_size, void *workspace, size_t workspace_bytes, qg_stream_t stream);
size_t qgemm_codebook4_nested_workspace_bytes(int a_dtype, int M, int N, int K, int block_size);

/*
 * qgemm_nbits_packed_zp -- qgemm_nbits with unsigned integer zero points
 * packed like the codes.  [hip-ep #1318] "Notes for reviewers", kernel test
 * table (the 2-, 3-, 4- and 8-bit MatMulNBits leaves); the pages' own zero
 * points are fp16 ("What", Commit 1) and they describe no packed form, so the
 * layout is this library's reading: zero point b of row n is the unsigned
 * `bits`-wide field starting at bit b*bits of row n's bit string, least
 * significant bit first (a field may continue into the next byte), each row
 * occupying ceil((K/block_size)*bits/8) bytes.
 *
 *   zero_points_packed  [N][ceil((K/block_size)*bits/8)] uint8 (device, any
 *                alignment; NULL: QG_ERR_INVALID_ARG)
 *   Other arguments as qgemm_nbits; the workspace holds at least
 *   qgemm_nbits_packed_zp_workspace_bytes() bytes, 16-byte aligned.  A request
 *   that qgemm_nbits would serve with its SIMT GEMV kernel stages the packed
 *   bytes beside the codes and widens each field where it is used; any other
 *   (2-bit block-64 tensor-pipe GEMV, tensor cores) first widens the zero
 *   points to fp16 [N][K/block_size] at the front of the workspace with one
 *   small kernel.  Either way the result is bit-identical to qgemm_nbits
 *   given the same integers as fp16 zero points.  Every check of qgemm_nbits
 *   happens before anything is enqueued.
 */
int qgemm_nbits_packed_zp(const void *A, int a_dtype, const uint8_t *W, const uint16_t *scales_f16,
                          const uint8_t *zero_points_packed, void *Y, int y_dtype, int M, int N, int K, int bits,
                          int block_size, void *workspace, size_t workspace_bytes, qg_stream_t stream);
size_t qgemm_nbits_packed_zp_workspace_bytes(int a_dtype, int M, int N, int K, int bits, int block_size);

/*
 * qmoe_ragged_mm -- ragged expert GEMM: the rows of X are grouped by expert
 * and each group is multiplied by its expert's MatMulNBits weight.
 * [hip-ep #1318] kernel test table, qmoe_ragged_mm leaf Xfp16_Wu4_Yfp16; the
 * pages name the op and its types, the layout is this library's reading.
 *
 *   for e in 0 .. num_experts-1, r in [offs[e], offs[e+1]):
 *       Y[r][n] = sum_k X[r][k] * w_e[n][k],  w_e = (q - zp) * s as qgemm_nbits
 *
 *   X                [T][K] of x_dtype (QG_F32 / F16 / BF16), T = offs[num_experts]
 *   expert_offsets   [num_experts + 1] int64, HOST memory: offs[0] = 0, never
 *                    decreasing (an expert may own no row); read before return
 *   W                [num_experts][N][K*bits/8] codes, bits 2, 4 or 8
 *   scales_f16       [num_experts][N][K/block_size] fp16
 *   zero_points_f16  same shape, fp16, or NULL (midpoint 2^(bits-1))
 *   Y                [T][N] of y_dtype
 * X, W, scales and zero points 16-byte aligned; one expert's slice of W and of
 * the scales must be a multiple of 16 bytes (QG_ERR_UNSUPPORTED otherwise).
 * With 16-bit activations the experts with 9 or more rows run in one grouped
 * tensor-core launch (at most 256 experts); the others, and fp32 activations,
 * run as one GEMM per expert on its rows.  Workspace: at least
 * qmoe_ragged_mm_workspace_bytes(...) for the same offsets (0 when every expert
 * takes the grouped launch).
 */
int qmoe_ragged_mm(const void *X, int x_dtype, const int64_t *expert_offsets, int num_experts, const uint8_t *W,
                   const uint16_t *scales_f16, const uint16_t *zero_points_f16, void *Y, int y_dtype, int N, int K,
                   int bits, int block_size, void *workspace, size_t workspace_bytes, qg_stream_t stream);
size_t qmoe_ragged_mm_workspace_bytes(int x_dtype, const int64_t *expert_offsets, int num_experts, int N, int K,
                                      int bits, int block_size);

/*
 * qmoe_ragged_mm_device_offsets -- the ragged expert GEMM above with the
 * expert offsets in DEVICE memory, so that a router on the GPU needs no host
 * round trip: the computation and the reading of the pages are those of
 * qmoe_ragged_mm ([hip-ep #1318] kernel test table, qmoe_ragged_mm leaf;
 * [hip-ep #1328] "Summary": the QMoE op family).
 *
 *   expert_offsets_dev  [num_experts + 1] int64, device, 8-byte aligned,
 *                       read on the device after the preceding work on the
 *                       stream: offs[0] = 0, never decreasing, offs[E] <=
 *                       max_rows.  Offsets breaking that rule make the call
 *                       compute nothing and set *status_dev to 1 (status_dev
 *                       may be NULL; it is never cleared).
 *   max_rows            rows X and Y hold (host int, >= the real T); rows of
 *                       Y at or past offs[E] are left untouched
 *   X                   [max_rows][K] fp16 or bf16 (fp32: QG_ERR_UNSUPPORTED)
 *   W, scales, zero points, Y, N, K, bits, block_size as qmoe_ragged_mm
 *   num_experts         1 .. 256
 *   workspace           not used (may be NULL);
 *                       qmoe_ragged_mm_device_offsets_workspace_bytes(E)
 *                       returns 0
 * Every expert with rows runs in one grouped tensor-core launch (sized for the
 * most tiles offsets within max_rows can need; each CTA numbers the experts'
 * tiles from the offsets itself, and tiles past the real count end at once).
 * Returns QG_OK, QG_ERR_* for refused arguments (before any launch) or
 * QG_ERR_CUDA.
 */
int qmoe_ragged_mm_device_offsets(const void *X, int x_dtype, const int64_t *expert_offsets_dev, int num_experts,
                                  int max_rows, const uint8_t *W, const uint16_t *scales_f16,
                                  const uint16_t *zero_points_f16, void *Y, int y_dtype, int N, int K, int bits,
                                  int block_size, void *workspace, size_t workspace_bytes, int *status_dev,
                                  qg_stream_t stream);
size_t qmoe_ragged_mm_device_offsets_workspace_bytes(int num_experts);

/*
 * qg_gather_block_quantized -- embedding lookup in a block-quantized table.
 * [hip-ep #1318] kernel test table, gather_block_quantized leaves
 * Xi64_Wu4_Yfp16, Xi64_Wu8_Yfp16 and Xi64_Wfp8_Yfp16 ("Summary", Commit 3:
 * embedding lookups through a gather).  The pages name the op and its types;
 * the layout and rule below are this library's reading of them.
 *
 *   Y[i][d] = round_to(y_dtype, w(row_i, d)),  row_i = indices[i], or
 *             indices[i] + vocab when indices[i] < 0
 *   integer formats: w = fl32( fl32(q - zp) * s )  (as qgemm_nbits; zp the
 *                    midpoint 2^(bits-1) when zero_points_f16 is NULL)
 *   QG_WF_E4M3:      w = fl32( e4m3(q) * s )  (OCP E4M3 without infinities;
 *                    no zero point)
 *   with s = scales_f16[row_i][d / block_size], and rounding to nearest-even.
 *
 *   indices      [n_indices] int64 (device, 8-byte aligned).  An index outside
 *                [-vocab, vocab) gives a zero row and sets *status_dev to 1.
 *   W            [vocab][D*bits/8] codes packed LSB-first along D (bits 2, 4
 *                or 8 for QG_WF_U2 / U4 / U8), or [vocab][D] E4M3 bytes
 *   scales_f16   [vocab][D/block_size] fp16
 *   zero_points_f16  same shape, fp16, or NULL; must be NULL for E4M3
 *   block_size   32, 64, 128 or 256; D a multiple of it
 *   Y            [n_indices][D] of y_dtype (QG_F32, QG_F16 or QG_BF16)
 *   status_dev   device int, written with 0 (every index valid) or 1, or NULL
 * W, scales, zero points and Y must be 16-byte aligned.  Results are exact
 * (bit-identical to the definition) whenever w is exact in fp32, e.g. for
 * integer or half-integer zero points and for every E4M3 table.
 */
enum { QG_WF_U2 = 0, QG_WF_U4 = 1, QG_WF_U8 = 2, QG_WF_E4M3 = 3 };
int qg_gather_block_quantized(const int64_t *indices, int64_t n_indices, const uint8_t *W, int w_format,
                              const uint16_t *scales_f16, const uint16_t *zero_points_f16, int64_t vocab, int D,
                              int block_size, void *Y, int y_dtype, int *status_dev, qg_stream_t stream);

/*
 * Low-rank adapters beside a shared projection, served and trained.  The
 * source pages have no counterpart: these are additions of this library (the
 * quantized weight W [N][K] of the entry points above stays frozen; a request
 * brings an adapter of rank r, A [r][K] and B [N][r], of its own).
 *
 * Requests.  The T rows of X are grouped by request: request i owns rows
 * seg_offsets[i] .. seg_offsets[i+1]-1 and uses adapter seg_adapter[i]
 * (negative: none).  Both arrays are DEVICE memory, read after the preceding
 * work on the stream: offs[0] = 0, never decreasing (a request may own no
 * row), offs[num_segments] <= rows.  Offsets breaking that rule make the call
 * compute nothing and set *status_dev to 1; an adapter id at or past
 * num_adapters counts as none and sets it too.  status_dev may be NULL and is
 * never cleared.  Rows at or past offs[num_segments] are left untouched.
 * At most 65536 requests and 65535 adapters a call (QG_ERR_UNSUPPORTED).
 *
 * qg_lora_apply -- for every row t of a request with adapter a
 *   V[t][j] = sum_k X[t][k] * A[a][j][k]                        (fp32)
 *   Y[t][n] = round( Y_in[t][n] + scaling[a] * sum_j V[t][j] * B[a][n][j] )
 * and Y = round(Y_in) for rows of requests without one.
 *
 *   X            [rows] rows of K values, ldx values apart; x_dtype
 *   A, B         [num_adapters][rank][K] and [num_adapters][N][rank]; w_dtype:
 *                x_dtype, or any type beside fp32 activations
 *   scaling      [num_adapters] fp32, or NULL (all 1)
 *   Y_in         [rows] rows of N values, ldy_in apart, y_in_dtype (QG_F32 or
 *                y_dtype), or NULL (zeros); may be Y itself
 *   Y            [rows] rows of N values, ldy apart, y_dtype
 *   V_out        [rows][rank] fp32 or NULL: V, for the backward pass (0 for
 *                rows without an adapter)
 *   rank         8 .. 128, a multiple of 8 (pad smaller or mixed ranks with
 *                zeros); others QG_ERR_UNSUPPORTED
 *   K            a multiple of 8; X, A and B 16-byte aligned, ldx * the
 *                element size a multiple of 16.  N and the strides of Y are free.
 * Sums are fp32.  16-bit operands multiply exactly; an fp32 operand is split in
 * two TF32 terms (22 bits), and V, for the second product with 16-bit adapters of
 * 16-bit activations, in two terms of their type (bf16: 16 bits, fp16: 22).
 * Deterministic.  workspace: at least qg_lora_apply_workspace_bytes(rows,
 * num_segments, rank, N, K) bytes, 16-byte aligned (NULL when that is 0).
 * rows == 0, N == 0 or num_segments == 0 is a no-op: V_out is not written either.
 *
 * qg_lora_grad -- the backward pass, given dY, X and the V of the forward pass:
 *   G[t][j]  = scaling[a] * sum_n dY[t][n] * B[a][n][j]         (fp32)
 *   dX[t][k] = round( dX_in[t][k] + sum_j G[t][j] * A[a][j][k] )
 *   dA[a][j][k] = sum over the rows t of adapter a of G[t][j] * X[t][k]
 *   dB[a][n][j] = scaling[a] * sum over those rows of dY[t][n] * V[t][j]
 *
 *   dY           [rows] rows of N values, lddy apart, x_dtype (any alignment)
 *   X, A, B      as above;  V  [rows][rank] fp32
 *   dX_in, dX    [rows] rows of K values, lddx apart (both), x_dtype; dX may be
 *                NULL (no gradient of the activations is wanted: A is then not
 *                read), dX_in may be NULL (zeros) or dX itself
 *   dA, dB       shapes of A and B; g_dtype: w_dtype or QG_F32; zero for an
 *                adapter without rows.  accumulate = 1 adds to their contents.
 *   workspace    at least qg_lora_grad_workspace_bytes(...) bytes, 16-byte aligned
 * Sums are fp32 with operands as above; G and V enter dA and dB in two bf16 terms (16
 * bits) for bf16 gradients, else in 22 bits or more.
 * Infinities and NaN (both passes): a result is infinite or NaN where one that is enters
 * its sum, and no other result is; as operands go in two terms, a sum that an infinity
 * makes infinite may come out as NaN.
 * rows == 0 or num_segments == 0: dA and dB are zeros (or what they held), dX is
 * not written.  N == 0: empty sums, so dX is dX_in and dA is zero; dY, B and dB
 * may be NULL.
 */
size_t qg_lora_apply_workspace_bytes(int rows, int num_segments, int rank, int N, int K);
int qg_lora_apply(const void *X, int x_dtype, int64_t ldx, const int64_t *seg_offsets, const int32_t *seg_adapter,
                  int num_segments, const void *A, const void *B, int w_dtype, const float *scaling, int num_adapters,
                  int rank, const void *Y_in, int y_in_dtype, int64_t ldy_in, void *Y, int y_dtype, int64_t ldy,
                  float *V_out, int rows, int N, int K, int *status_dev, void *workspace, size_t workspace_bytes,
                  qg_stream_t stream);
size_t qg_lora_grad_workspace_bytes(int rows, int num_segments, int num_adapters, int rank, int N, int K);
int qg_lora_grad(const void *dY, int x_dtype, int64_t lddy, const void *X, int64_t ldx, const float *V,
                 const int64_t *seg_offsets, const int32_t *seg_adapter, int num_segments, const void *A,
                 const void *B, int w_dtype, const float *scaling, int num_adapters, int rank, const void *dX_in,
                 void *dX, int64_t lddx, void *dA, void *dB, int g_dtype, int accumulate, int rows, int N, int K,
                 int *status_dev, void *workspace, size_t workspace_bytes, qg_stream_t stream);

/*
 * qgemm_*_dgrad -- the gradient of the activations through a frozen quantized
 * weight: dX[M][K] = dY[M][N] . dequant(W)[N][K], with W, its parameters, bits
 * and block_size as in qgemm_nbits / qgemm_nbits_uniform_zp / qgemm_codebook4
 * (an addition of this library, like the adapters above).
 *   dY   [M][N] contiguous, dy_dtype;  dX  [M][K] contiguous, dx_dtype; both
 *        16-byte aligned
 *   16-bit dY: the weight is rounded to dY's type before the product, as in
 *   the forward pass; fp32 dY: dY and the weight go in two scaled fp16 terms each
 *   (22 bits).  fp32 accumulation, one rounding to dx_dtype.  3-bit codes run on
 *   a plain fp32 kernel.
 *   An infinite or NaN dY reaches the whole of its row, an infinite or NaN parameter the
 *   columns of its block, and nothing else; with fp32 dY, whose terms are multiplied one
 *   by one, an infinity comes out as NaN.  A uniform_zp that is no finite fp16 value is
 *   QG_ERR_INVALID_ARG, as in qgemm_nbits_uniform_zp.
 *   workspace: at least qgemm_dgrad_workspace_bytes(dy_dtype, M, N, K, bits)
 *   bytes, 16-byte aligned (NULL when that is 0).
 * M == 0 or K == 0 is a no-op; N == 0 writes zeros.
 */
size_t qgemm_dgrad_workspace_bytes(int dy_dtype, int M, int N, int K, int bits);
int qgemm_nbits_dgrad(const void *dY, int dy_dtype, const uint8_t *W, const uint16_t *scales_f16,
                      const uint16_t *zero_points_f16, void *dX, int dx_dtype, int M, int N, int K, int bits,
                      int block_size, void *workspace, size_t workspace_bytes, qg_stream_t stream);
int qgemm_nbits_uniform_zp_dgrad(const void *dY, int dy_dtype, const uint8_t *W, const uint16_t *scales_f16,
                                 float uniform_zp, void *dX, int dx_dtype, int M, int N, int K, int bits,
                                 int block_size, void *workspace, size_t workspace_bytes, qg_stream_t stream);
int qgemm_codebook4_dgrad(const void *dY, int dy_dtype, const uint8_t *W, const float *codebook16,
                          const float *absmax, void *dX, int dx_dtype, int M, int N, int K, int block_size,
                          void *workspace, size_t workspace_bytes, qg_stream_t stream);

/*
 * qg_clip_grad_norm -- the 2-norm over all the values of a list of gradient
 * tensors, and their scaling to at most max_norm:
 *   norm = sqrt( sum over every tensor and value of grad^2 )
 *   out  = round( grad * min(1, max_norm / (norm + eps)) )
 * A norm that is infinite or NaN is written as such and scales by what the
 * formula gives (0 or NaN), so every out shows it.
 *
 *   tensors     the list in DEVICE memory, laid out by qg_grad_list_init from
 *               a host array (copy it to the device once; it holds addresses)
 *   count       tensors in the list;  chunks  what qg_grad_list_init returned
 *   out         may be grad itself; same dtype and element alignment as grad
 *   norm_dev    fp32, device
 *   workspace   at least qg_clip_grad_norm_workspace_bytes(chunks) bytes, 16-byte aligned
 * Squares are added in fp32 within a chunk (in fp64 where they overflow or
 * underflow there) and in fp64 across chunks.  Deterministic.
 *
 * qg_grad_list_init -- checks a host array's grad, out, numel and dtype (a
 * NULL out means grad; numel may be 0) and fills in first_chunk; *chunks
 * receives the number of chunks.  Host only: enqueues nothing.
 */
typedef struct {
    const void *grad;
    void *out;
    int64_t numel;
    int64_t first_chunk; /* filled in by qg_grad_list_init */
    int32_t dtype;       /* QG_F32, QG_F16 or QG_BF16 */
    int32_t reserved;    /* filled in by qg_grad_list_init */
} qg_grad_tensor;
int qg_grad_list_init(qg_grad_tensor *tensors_host, int count, int64_t *chunks);
size_t qg_clip_grad_norm_workspace_bytes(int64_t chunks);
int qg_clip_grad_norm(const qg_grad_tensor *tensors_dev, int count, int64_t chunks, float max_norm, float eps,
                      float *norm_dev, void *workspace, size_t workspace_bytes, qg_stream_t stream);

/*
 * qg_adamw_step -- one AdamW step over a list of tensors, in place (an addition of this library, like what follows):
 *   c  = min(1, max_norm / (norm + norm_eps)),  norm = sqrt( sum over every tensor and value of grad^2 );  g' = c * grad
 *   m' = beta1 m + (1 - beta1) g',   v' = beta2 v + (1 - beta2) g'^2
 *   p' = p (1 - lr weight_decay) - lr (m' / (1 - beta1^step)) / (sqrt(v' / (1 - beta2^step)) + eps)
 * computed in fp32.  p is the fp32 master copy where a tensor has one (param then receives it rounded), else param.
 *
 * States (state of a tensor), m in exp_avg and the second moment in exp_avg_sq:
 *   QG_STATE_F32    m and v in fp32; the scales are not used
 *   QG_STATE_E4M3   e4m3 codes of m and of u = sqrt(v), value = code * scale with one fp32 scale for every
 *                   QG_STATE_BLOCK values of the tensor (the last block may be shorter): exp_avg_scale and
 *                   exp_avg_sq_scale, [ceil(numel / QG_STATE_BLOCK)].  A step stores round(x / scale), scale = the
 *                   block's largest magnitude / 448 (a block below 1e-30 is stored as zeros with scale 0), u above
 *                   zero never as zero; p' uses m' and v' before that rounding.  All zeros is the state to begin with.
 * The moments are evaluated as they stand above, each product, sum and root rounded to fp32 by itself, and so are codes and
 * scales: round(x * (448 * (1 / amax))) and amax * (1 / 448).  An fp32 program of the same operations therefore keeps the same
 * 8-bit states.  One that orders them otherwise parts from these: a unit in the last place moves one value in a million to the
 * next code, which is up to 7% of it, and where that value comes to be the largest of its block, a scale is off by as much.
 * So does a norm whose last bit is another.  A g'^2 past fp32's range is infinity.
 * A block of a QG_STATE_E4M3 state that an infinity or NaN enters holds NaN from then on; values outside the block keep theirs.
 *
 *   tensors     the list in DEVICE memory, laid out by qg_adamw_list_init from a host array (it holds addresses).
 *               Its buffers may not overlap.
 *   count       tensors in the list;  chunks  what qg_adamw_list_init returned
 *   lr          or, where lr_dev is not NULL, one fp32 in device memory
 *   step        1 for the first step; or, where step_dev is not NULL, one int64 in device memory (below 1: 1), so
 *               that a captured call serves every step.  Both are read when the kernels run, neither is changed.
 *   max_norm    the clipping bound; negative: no clipping (norm_dev is not written).  With clipping, a norm that is
 *               infinite or NaN leaves every tensor as it was.
 *   norm_dev    fp32, device: the norm before clipping, or NULL
 *   workspace   at least qg_adamw_step_workspace_bytes(chunks) bytes, 16-byte aligned (with clipping; else NULL will do)
 * Sums of the norm as in qg_clip_grad_norm.  eps is meant to be far above the root of a v' that fp32 has few bits of (2^-126 and less).
 * Deterministic.
 *
 * qg_adamw_list_init -- checks a host array and fills in first_chunk; *chunks receives the number of chunks.  Pointers
 * have their type's alignment (any address for codes); numel may be 0, with NULL pointers.  Host only.
 */
enum { QG_STATE_F32 = 0, QG_STATE_E4M3 = 1 };
#define QG_STATE_BLOCK 256
typedef struct {
    void *param;
    const void *grad;
    float *master;           /* or NULL */
    void *exp_avg, *exp_avg_sq;
    float *exp_avg_scale, *exp_avg_sq_scale; /* QG_STATE_E4M3 */
    int64_t numel;
    int64_t first_chunk;     /* filled in by qg_adamw_list_init */
    float weight_decay;
    int32_t param_dtype, grad_dtype; /* QG_F32, QG_F16 or QG_BF16, each */
    int32_t state;
} qg_adamw_tensor;
int qg_adamw_list_init(qg_adamw_tensor *tensors_host, int count, int64_t *chunks);
size_t qg_adamw_step_workspace_bytes(int64_t chunks);
int qg_adamw_step(const qg_adamw_tensor *tensors_dev, int count, int64_t chunks, double lr, const float *lr_dev, double beta1,
                  double beta2, double eps, int64_t step, const int64_t *step_dev, float max_norm, float norm_eps,
                  float *norm_dev, void *workspace, size_t workspace_bytes, qg_stream_t stream);

/*
 * qg_token_logprobs -- log probabilities of given tokens, from the logits that the last projection of a model wrote:
 *   z = X[t] * inv_temperature,  lse[t] = log sum_v exp(z_v),  logprob[t] = z[targets[t]] - lse[t]
 *   entropy[t] = - sum_v p_v log p_v,  p_v = exp(z_v - lse[t])  (a term with p_v = 0 is 0)
 *   top_ids[t][j], top_logprobs[t][j]: the top_k most probable tokens and their log probabilities, the largest logit
 *   first, the lower index first among equals
 *
 *   X            [rows] rows of vocab values, ldx values apart; x_dtype; any alignment of its type
 *   targets      [rows] int64 (device), or NULL (none).  Negative: no token is given, logprob 0.  At or past vocab:
 *                the same, and *status_dev is set to 1 (it may be NULL and is never cleared).
 *   inv_temperature  finite, above 0 (in qg_token_logprobs at most 2.3e38: QG_ERR_UNSUPPORTED)
 *   logprob, entropy, lse  [rows] fp32, each may be NULL
 *   top_k        0 .. 64 and at most vocab (0: top_ids and top_logprobs may be NULL)
 *   top_ids      [rows][top_k] int64;  top_logprobs  [rows][top_k] fp32
 * Logits of -inf have probability 0.  A row with nothing above -inf: lse and the log probabilities are -inf, the
 * entropy 0.  A row with +inf or NaN among its logits: NaN throughout; its top_ids are in the order of the logits all
 * the same, NaN above +inf.  Sums in fp32.  Deterministic.  No workspace.
 *
 * qg_token_logprobs_grad -- the gradient of the logits:
 *   dX[t][v] = inv_temperature * ( d_logprob[t] ([v = targets[t]] - p_v) - d_entropy[t] p_v (log p_v + entropy[t]) )
 * with the first term left out of rows without a given token (also: a token at or past vocab).
 *   lse, entropy, inv_temperature  as the forward pass left or had them (entropy: only beside d_entropy)
 *   d_logprob    [rows] fp32;  d_entropy  [rows] fp32 or NULL (zeros)
 *   dX           [rows] rows of vocab values, lddx apart, x_dtype; may be X itself (with lddx = ldx)
 * A row whose two gradients are 0, or whose lse is -inf, gets zeros, whatever its logits.
 * p_v is exp(z_v - lse[t]) of the lse that is given, which is fp32: the p of a row are off by one factor of up to exp(2^-24 |lse[t]|), 3% where lse is
 * 800,000 and nothing where it is some hundreds. Rows that far from zero want their largest logit taken off first. A z past fp32's range has no gradient.
 * rows == 0 is a no-op in both; vocab 1 .. 2^28.
 */
int qg_token_logprobs(const void *X, int x_dtype, int64_t ldx, const int64_t *targets, int rows, int vocab,
                      float inv_temperature, float *logprob, float *entropy, float *lse, int top_k, int64_t *top_ids,
                      float *top_logprobs, int *status_dev, qg_stream_t stream);
int qg_token_logprobs_grad(const void *X, int x_dtype, int64_t ldx, const int64_t *targets, const float *lse,
                           const float *entropy, const float *d_logprob, const float *d_entropy, float inv_temperature,
                           void *dX, int64_t lddx, int rows, int vocab, qg_stream_t stream);

/*
 * qmoe_route_topk -- the experts of each token from its router logits (an addition of this library):
 *   expert_ids[t] = the k largest of logits[t], the largest first, the lower index first among equals (NaN above all)
 *   expert_weights[t][j] = exp(l_j - M) / sum exp(l_i - M), M the largest; the sum over the k chosen (renormalize = 1)
 *   or over all experts (0).  An expert at -inf has weight 0, also where all of them are; a NaN or +inf among the
 *   logits that are summed makes the token's weights NaN.
 *   logits  [tokens] rows of num_experts values (1 .. 512), ld values apart, any of the three types;  k  1 .. 16
 *   expert_ids [tokens][k] int32, expert_weights [tokens][k] fp32: as qmoe_tokens_fused and (a token) qmoe_decode_fused take them
 *
 * qmoe_tokens_fused -- the layer of qmoe_decode_fused over a few tokens at once, each with k experts of its own:
 *   y[t] = round( sum_j expert_weights[t][j] * o_tj ),  o_tj as there, from x[t] and expert expert_ids[t][j]
 * Every chosen expert's weights are read once for all its tokens (16 of them at a time, 8 in the second product of an
 * fp16 or fp32 y; fewer where hidden or inter is above some 2,800).  Weights, scales, zero points, biases, block sizes and swiglu_interleaved as qmoe_decode_fused; bits 2, 4 or 8.
 *   x            [tokens][hidden] fp16 or bf16 (fp32: QG_ERR_UNSUPPORTED)
 *   expert_ids, expert_weights  [tokens][k] int32 and fp32 (device), k 1 .. 16, tokens * k at most 1024, num_experts at
 *                most 512; an id outside [0, num_experts) adds nothing and sets *status_dev to 1 (it may be NULL and is
 *                never cleared); one that a token has twice counts twice
 *   y            [tokens][hidden] of y_dtype
 *   workspace    at least qmoe_tokens_workspace_bytes(tokens, k, hidden, inter) bytes, 16-byte aligned
 * Activations enter the products as fp16 scaled by a power of two for each row (11 bits for what is above 2^-29 of the
 * row's largest), h between the products as two such values (22 bits) or, where y is bf16 or inter above some 20,000, as one; codes, scales and zero
 * points are exact; sums in fp32.  A row with an infinity or NaN gives outputs that are not finite, the other rows are not touched by it.
 * Deterministic; the order of a sum depends on the shape and on how many experts were chosen.  A hidden or inter whose
 * rows do not fit the kernel's shared memory (some 30,000 and more) is QG_ERR_UNSUPPORTED.  More tokens: qmoe_ragged_mm.
 */
int qmoe_route_topk(const void *logits, int dtype, int64_t ld, int tokens, int num_experts, int k, int renormalize,
                    int32_t *expert_ids, float *expert_weights, qg_stream_t stream);
size_t qmoe_tokens_workspace_bytes(int tokens, int k, int hidden, int inter);
int qmoe_tokens_fused(const void *x, int x_dtype, const int32_t *expert_ids, const float *expert_weights, int tokens, int k,
                      int num_experts, const uint8_t *fc1_w, const uint16_t *fc1_scales, const uint16_t *fc1_zp,
                      const uint16_t *fc1_bias, const uint8_t *fc2_w, const uint16_t *fc2_scales, const uint16_t *fc2_zp,
                      const uint16_t *fc2_bias, int hidden, int inter, int bits, int block_size, int swiglu_interleaved,
                      void *y, int y_dtype, int *status_dev, void *workspace, size_t workspace_bytes, qg_stream_t stream);

/*
 * qg_read_device_fault -- every wait inside the library's kernels is
 * bounded; a wait that gives up records a bit in a device-side fault word
 * instead of hanging.  This call synchronises the current device, returns
 * the word in *flags (0: no fault since the last read) and clears it.
 * The word is one per device, shared by every call of every stream and
 * thread: a read reports (and clears) the faults of all calls on the device
 * since the previous read, whoever made them.  A caller that needs to know
 * which call gave up must read the word between its own calls, with no other
 * work on the device in between.  (A wait that gives up is a library fault --
 * a kernel that did not get its data within seconds -- not an argument
 * error: arguments are checked before anything is enqueued.)
 */
int qg_read_device_fault(unsigned int *flags);

/* Human-readable name of a QG_* status. */
const char *qg_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* QGEMM_H */
