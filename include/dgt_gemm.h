/*
 * dgt_gemm.h -- C ABI of the MI355X (gfx950) dense GEMM library.
 *
 * Operation (every entry point): the BLAS GEMM form
 *
 *     C <- alpha * op(A) * op(B) + beta * C
 *
 * with C(i,j) = sum_k op(A)(i,k) * op(B)(k,j) (element formula:
 * dilfish.github.io section 5.2; chongfengling.github.io section 1;
 * elainafan.one "稠密矩阵乘法", where alpha and beta let one call both scale
 * and accumulate).  op(X) is X, or X transposed when gemm_ex is asked for it
 * (every other entry point: no transposes).
 *
 * Layout: row-major with leading dimensions, the column index contiguous
 * (chongfengling.github.io section 2.2; elainafan.one "行主序"):
 *     op(A)(i,k) = A[i*lda + k]  trans_a = 0: A stored M x K, lda >= max(1, K)
 *     op(A)(i,k) = A[k*lda + i]  trans_a = 1: A stored K x M, lda >= max(1, M)
 *     op(B)(k,j) = B[k*ldb + j]  trans_b = 0: B stored K x N, ldb >= max(1, N)
 *     op(B)(k,j) = B[j*ldb + k]  trans_b = 1: B stored N x K, ldb >= max(1, K)
 *     C(i,j)     = C[i*ldc + j]  C is M x N,                  ldc >= max(1, N)
 * The transposed forms are the operands of a linear layer stored as in
 * elainafan.one "全连接层" (input X [batch, in], weight W [out, in], output
 * gradient G [batch, out]): the forward pass X*W^T is trans_b = 1, the
 * weight gradient G^T*X is trans_a = 1, the input gradient G*W needs
 * neither.  A column-major caller passes its storage with the flags set.
 *
 * Precision: gemm_f32 takes fp32 A and B; gemm_bf16 takes A and B as raw
 * bf16 bit patterns (uint16_t, the upper half of an fp32 value: 8-bit
 * exponent, 7-bit mantissa); gemm_f16 takes raw IEEE binary16 bit patterns
 * (5-bit exponent, 10-bit mantissa) -- the BF16 and FP16 rows of the
 * dilfish.github.io section 5.5 precision table.  All accumulate in fp32 on
 * the matrix cores and read/write C in fp32.  The
 * summation order is the kernel's own; results agree with an exact
 * reference to fp32 accumulation accuracy, and bit for bit whenever every
 * partial sum is exactly representable (e.g. small-integer inputs).
 *
 * Semantics of the edge cases (the pages leave them open; BLAS readings):
 *   - beta == 0: C is write-only; NaN/Inf already in C never propagate.
 *   - alpha == 0 or K == 0: A and B are not read; C <- beta*C (zeros when
 *     beta == 0 too).
 *   - M == 0 or N == 0: nothing is done; returns GEMM_OK.
 *
 * Memory and ownership: A, B and C are DEVICE pointers owned by the caller;
 * they must stay valid until the work queued on `stream` has finished.  The
 * library allocates nothing, frees nothing, keeps no per-call state and is
 * safe to call from several host threads.  A misaligned pointer or leading
 * dimension is accepted (fp32: 4-byte, bf16/fp16: 2-byte alignment); it only
 * selects a slower load path, never a fault.
 *
 * Ordering: asynchronous.  Work is queued on `stream` (a hipStream_t cast
 * to void*; NULL = the null stream) and the call returns without waiting.
 *
 * Errors: every entry point returns GEMM_OK (0) or a negative status; on an
 * argument error nothing is queued.  The library never aborts or prints.
 * Argument checks run on the host in this order: dtype and transpose flags,
 * dimensions, leading dimensions, variant id, quick return for an empty C,
 * null pointers, overlap of C with A or B, variant support for the shape.
 * gemm_status_string() names a status.
 */
#ifndef DGT_GEMM_H
#define DGT_GEMM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Entry points may be added without a new version; the ones of a version keep
 * their meaning. */
#define DGT_GEMM_ABI_VERSION 9

/* Input formats (the dtype argument of gemm_ex and gemm_select_variant). */
enum gemm_dtype { GEMM_DTYPE_F32 = 0, GEMM_DTYPE_BF16 = 1, GEMM_DTYPE_F16 = 2 };

enum gemm_status {
    GEMM_OK = 0,
    GEMM_ERR_DIM = -1,          /* M, N or K negative; MX4, gated, W4 and
                                   orthogonalisation: past their limits      */
    GEMM_ERR_LD = -2,           /* lda < max(1,K), ldb < max(1,N) or
                                   ldc < max(1,N)                            */
    GEMM_ERR_NULL = -3,         /* NULL A/B (when read) or C with a
                                   non-empty extent                          */
    GEMM_ERR_OVERLAP = -4,      /* the byte range of C overlaps A's, B's or
                                   the bias's, or two problems of a batch
                                   share C elements                          */
    GEMM_ERR_VARIANT = -5,      /* unknown variant, or one that does not
                                   support this shape / size                 */
    GEMM_ERR_LAUNCH = -6,       /* the HIP runtime rejected a kernel launch  */
    GEMM_ERR_ARG = -7,          /* dtype not a gemm_dtype, a transpose flag
                                   other than 0 or 1, an activation or
                                   group that is none, a negative batch,
                                   splits or workspace size, or a stride
                                   outside [0, 2^48)                         */
    GEMM_ERR_WORKSPACE = -8,    /* gemm_splitk, gemm_streamk,
                                   gemm_orthogonalize, gemm_gated_grad:
                                   workspace NULL or smaller than the call's
                                   workspace size                            */
    GEMM_ERR_SCRATCH = -9,      /* gemm_splitk_noalloc: the shape's partials
                                   (gemm_splitk_workspace_size) exceed
                                   DGT_GEMM_NOALLOC_SCRATCH_BYTES            */
    GEMM_ERR_ALIGN = -10        /* MX4 codes or scales, or W4 codes, whose
                                   base or row pitch is not a multiple of 16
                                   bytes, or a gemm_orthogonalize or
                                   gemm_gated_grad workspace whose base is
                                   not                                       */
};

/* Kernel ladder (for measurement and tests; GEMM_VARIANT_AUTO is what
 * gemm_f32 / gemm_bf16 / gemm_f16 use).  Every variant computes the same operation
 * and handles any shape that it accepts, ragged edges included. */
enum gemm_variant {
    GEMM_VARIANT_AUTO = 0,      /* MFMA tiles; skinny path when M <= 64       */
    GEMM_VARIANT_NAIVE = 1,     /* one lane per output, K-loop of two global
                                   loads and an FMA (dilfish.github.io 5.2;
                                   chongfengling.github.io 2.1 and 2.4:
                                   the contiguous column index on the
                                   64-wide lane index)                        */
    GEMM_VARIANT_LDS = 2,       /* LDS-staged 128x128 macro tiles, 128-bit
                                   global loads, double-buffered, padded LDS
                                   rows, 8x8 outputs per lane on the vector
                                   ALU (dilfish.github.io 5.3 and 5.4)        */
    GEMM_VARIANT_MFMA = 3,      /* LDS-staged macro tiles, double-buffered,
                                   per-wavefront MFMA micro-tiles, masked
                                   ragged edges (dilfish.github.io 5.4-5.5;
                                   qwbw.cn section 三); the workgroup tile
                                   (256 x 256 or 128 x 128; 64 x 64 for fp32
                                   launches with at most 128 tiles of 128 x
                                   128) is chosen per launch                  */
    GEMM_VARIANT_SKINNY = 4,    /* M <= 64: streams B once from HBM (copied
                                   straight into LDS when B is stored N x K
                                   with 16-byte aligned rows), A held in
                                   registers per step (up to four 16-row
                                   blocks), K split over waves and reduced
                                   in LDS (dilfish.github.io 5.1 GEMV row and
                                   batching; qwbw.cn section 四)              */
    GEMM_VARIANT_MFMA_T256 = 5, /* the MFMA rung's global->LDS DMA kernel with
                                   a fixed 256 x 256 workgroup tile (one
                                   workgroup per CU): the block-size choice
                                   of dilfish.github.io 5.3-5.4 made
                                   explicit.  Needs 16-byte aligned operand
                                   rows (pitch and base) and pitches below
                                   2^23 (fp32) or 2^24 (16-bit) elements;
                                   GEMM_ERR_VARIANT otherwise                */
    GEMM_VARIANT_MFMA_T128 = 6, /* the same with 128 x 128 tiles, two
                                   workgroups per CU                          */
    GEMM_VARIANT_MFMA_REGS = 7  /* the MFMA rung without the DMA pipeline:
                                   LDS tiles filled through registers by
                                   128-bit loads, double-buffered
                                   (dilfish.github.io 5.4's double buffer),
                                   MFMA micro-tiles, workgroup tiles of
                                   128 x 128 (fp32) or 256 x 256 (16-bit
                                   inputs); any alignment.  GEMM_VARIANT_MFMA
                                   uses this kernel for operands the DMA
                                   kernels do not take (rows not 16-byte
                                   aligned, pitches past their limits) and,
                                   on 64 x 64 tiles, for the small fp32
                                   launches                                   */
};

/* C <- alpha*A*B + beta*C, fp32 inputs, fp32 accumulate/output. */
int gemm_f32(int M, int N, int K, float alpha, const float* A, int lda,
             const float* B, int ldb, float beta, float* C, int ldc,
             void* stream);

/* C <- alpha*A*B + beta*C, bf16 inputs (raw bits), fp32 accumulate/output. */
int gemm_bf16(int M, int N, int K, float alpha, const uint16_t* A, int lda,
              const uint16_t* B, int ldb, float beta, float* C, int ldc,
              void* stream);

/* C <- alpha*A*B + beta*C, fp16 inputs (raw IEEE binary16 bits), fp32
 * accumulate/output: the half-input / fp32-accumulate matrix-unit path of
 * dilfish.github.io 5.5 (WMMA listing) and qwbw.cn Level 2. */
int gemm_f16(int M, int N, int K, float alpha, const uint16_t* A, int lda,
             const uint16_t* B, int ldb, float beta, float* C, int ldc,
             void* stream);

/* Same as gemm_f32 / gemm_bf16 / gemm_f16 with an explicit ladder rung (enum
 * gemm_variant).  GEMM_VARIANT_SKINNY requires M <= 64, and the fixed-tile
 * MFMA rungs 16-byte aligned operand rows, and return GEMM_ERR_VARIANT
 * otherwise (checked on the host before anything is queued; alpha == 0 or
 * K == 0 never reads A or B and so never fails this check). */
int gemm_f32_variant(int variant, int M, int N, int K, float alpha,
                     const float* A, int lda, const float* B, int ldb,
                     float beta, float* C, int ldc, void* stream);
int gemm_bf16_variant(int variant, int M, int N, int K, float alpha,
                      const uint16_t* A, int lda, const uint16_t* B, int ldb,
                      float beta, float* C, int ldc, void* stream);
int gemm_f16_variant(int variant, int M, int N, int K, float alpha,
                     const uint16_t* A, int lda, const uint16_t* B, int ldb,
                     float beta, float* C, int ldc, void* stream);

/* General form: C <- alpha*op(A)*op(B) + beta*C with the input format
 * `dtype` (enum gemm_dtype; A and B point to float for GEMM_DTYPE_F32, to
 * raw uint16_t bits otherwise), transpose flags trans_a / trans_b (0 or 1,
 * storage as in the layout table above) and a ladder rung `variant` (enum
 * gemm_variant; every rung takes every layout).  The untransposed call is
 * the same operation as gemm_f32 / gemm_bf16 / gemm_f16 (_variant), with the
 * same kernels. */
int gemm_ex(int dtype, int trans_a, int trans_b, int variant, int M, int N,
            int K, float alpha, const void* A, int lda, const void* B, int ldb,
            float beta, float* C, int ldc, void* stream);

/* Strided batch with the bias of a linear layer: for z = 0 .. batch-1,
 *
 *   C_z <- alpha * op(A_z) * op(B_z) + beta * C_z + 1 * bias_z^T
 *
 * where X_z = X + z * stride_x (strides in ELEMENTS of the operand: A and B
 * in their input format, C and bias in floats; 0 repeats one operand for
 * every problem, e.g. a shared weight), and bias_z is a row of N floats
 * added to every row of C_z (elainafan.one "全连接层": the linear layer
 * computes X*W^T + b; its input keeps a batch dimension).  bias may be NULL
 * (no bias); it is added after the BLAS form, unscaled, also when
 * alpha == 0 or K == 0.  Every other argument is as for gemm_ex.
 * Requirements: batch >= 0 (0 does nothing), strides in [0, 2^48), the
 * problems' C ranges disjoint (stride_c * 4 bytes at least the span of one
 * C when batch > 1), C disjoint from every A, B and bias range.  Any batch
 * size is accepted; the library splits it into launches of at most 65535
 * problems, queued in order on `stream`. */
int gemm_strided_batched(int dtype, int trans_a, int trans_b, int variant,
                         int M, int N, int K, float alpha,
                         const void* A, int lda, int64_t stride_a,
                         const void* B, int ldb, int64_t stride_b,
                         float beta, float* C, int ldc, int64_t stride_c,
                         const float* bias, int64_t stride_bias, int batch,
                         void* stream);

/* Split-K, for shapes with too few output tiles to fill the GPU (e.g. a
 * small M x N with a long K).  Same operation and arguments as gemm_ex with
 * GEMM_VARIANT_AUTO, computed in two phases queued on `stream`: the K range
 * is cut into slices (whole multiples of 128 except the last), each slice's
 * product is written to the caller's `workspace` as fp32 partials (M x N
 * per slice), and a second kernel sums the slices in a fixed order and
 * applies alpha and beta -- deterministic, no atomics, nothing allocated.
 * The pages do not describe split-K; they note that a launch whose blocks
 * are partly idle leaves compute unused (elainafan.one "朴素 CUDA 实现",
 * after the launch code), and this is the case where the whole grid is too
 * small: the reduction dimension supplies the missing parallelism.
 * `splits` = 0 picks the number of slices that fills the GPU's workgroup
 * slots (128 x 128 tiles: one per CU for fp32, two for 16-bit inputs; a
 * skinny column strip per CU for M <= 64; each slice at least 128 deep)
 * and runs them as one launch; a positive value is a request (at
 * most 64; rounding of the slice length may give fewer).  With one slice
 * the call is gemm_ex and needs no workspace.  The workspace (device
 * memory, 16-byte aligned, at least gemm_splitk_workspace_size bytes) must
 * not overlap A, B or C and must stay untouched until the work on `stream`
 * has finished; its contents on return are unspecified. */
int gemm_splitk(int dtype, int trans_a, int trans_b, int M, int N, int K,
                float alpha, const void* A, int lda, const void* B, int ldb,
                float beta, float* C, int ldc, int splits, void* workspace,
                int64_t workspace_bytes, void* stream);

/* gemm_splitk for callers that cannot allocate device memory at all --
 * code recorded under HIP graph capture, tight serving loops, harnesses
 * that forbid allocation -- and so cannot hand in a workspace either.
 * Same operation, arguments, slicing and kernels as gemm_splitk (results
 * are bit-identical to it), but the fp32 partials go to a fixed scratch
 * array of DGT_GEMM_NOALLOC_SCRATCH_BYTES that the library holds on every
 * GPU it has run on until the process ends.  The call allocates nothing:
 * no hipMalloc, no hipFree, no allocating library routine.
 *   - Size limit: a shape whose partials (gemm_splitk_workspace_size for
 *     the same dtype, shape and splits) exceed the scratch returns
 *     GEMM_ERR_SCRATCH before anything is queued; a shape that needs no
 *     split runs as gemm_ex and uses no scratch.
 *   - Sharing: all calls on one GPU share that GPU's scratch, which keeps
 *     the last call's partials.  Calls on one GPU must not overlap in time
 *     (queue them on one stream, or order their streams); overlapping calls
 *     race on the scratch and give wrong results.  No part of the scratch
 *     needs to start at zero (every partial is written before it is read).
 *   - The first call on a GPU looks up that GPU's scratch address (a host
 *     query, no allocation); a failure there returns GEMM_ERR_LAUNCH.
 * Every other error is as for gemm_splitk. */
#define DGT_GEMM_NOALLOC_SCRATCH_BYTES (64ll << 20)
int gemm_splitk_noalloc(int dtype, int trans_a, int trans_b, int M, int N,
                        int K, float alpha, const void* A, int lda,
                        const void* B, int ldb, float beta, float* C, int ldc,
                        int splits, void* stream);

/* Number of K slices gemm_splitk uses for this shape and request (>= 1), or
 * a negative status.  Host only. */
int gemm_splitk_slices(int dtype, int M, int N, int K, int splits);

/* Bytes of workspace gemm_splitk needs for this shape and request: slices x
 * M x N x 4, or 0 with one slice; a negative status for bad arguments.
 * Host only. */
int64_t gemm_splitk_workspace_size(int dtype, int M, int N, int K, int splits);

/* Stream-K: the same operation and arguments as gemm_ex with
 * GEMM_VARIANT_AUTO, for shapes whose 256 x 256 output tiles do not divide
 * evenly among the 256 compute units (the last wave of tiles of a
 * data-parallel launch then runs on part of the chip).  The pages note that
 * a launch whose blocks are partly idle leaves compute unused
 * (elainafan.one "朴素 CUDA 实现", after the launch code); stream-K deals out
 * the tiles' K iterations (128 k each for 16-bit inputs, 64 k for FP32) in
 * equal contiguous ranges to one workgroup per compute unit instead of whole
 * tiles.  A tile covered by one workgroup is written directly; the parts of
 * a tile split between workgroups go to the caller's `workspace` as fp32
 * partial sums, and a second kernel queued on `stream` sums them in k order
 * and applies alpha, beta -- deterministic, no atomics, nothing allocated.
 * Covered: FP32, BF16 and FP16 inputs, M > 64, operands whose stored rows
 * are 16-byte aligned with pitches below 2^24 elements (2^23 for FP32).
 * Anything else (M <= 64, unaligned operands, alpha == 0 or K == 0) runs as
 * gemm_ex with GEMM_VARIANT_AUTO and needs no workspace.  The workspace (device memory,
 * 16-byte aligned, at least gemm_streamk_workspace_size bytes: two
 * 256 x 256 fp32 tiles per workgroup, 128 MiB at most) must not overlap A, B
 * or C and must stay untouched until the work on `stream` has finished; its
 * contents on return are unspecified.  Errors as for gemm_splitk.
 * gemm_f32 / gemm_bf16 / gemm_f16 and GEMM_VARIANT_AUTO take no workspace
 * and never split K; for the shapes above this call is the faster form. */
int gemm_streamk(int dtype, int trans_a, int trans_b, int M, int N, int K,
                 float alpha, const void* A, int lda, const void* B, int ldb,
                 float beta, float* C, int ldc, void* workspace,
                 int64_t workspace_bytes, void* stream);

/* Bytes of workspace gemm_streamk needs for this shape (0 when the call
 * runs as gemm_ex), or a negative status for bad arguments.  Host only. */
int64_t gemm_streamk_workspace_size(int dtype, int M, int N, int K);

/* ------------------------------------------------------------------ MX4
 *
 * Microscaled 4-bit operands (the MXFP4 format of the OCP Microscaling
 * Formats specification 1.0).  A row of K elements is cut into blocks of 32
 * consecutive k; element k stands for
 *
 *     value(code) * 2^(s - 127)
 *
 * with s the block's scale byte (255 stands for NaN: the whole block is NaN)
 * and code 4 bits: bit 3 the sign, bits 2..0 one of the magnitudes 0, 0.5,
 * 1, 1.5, 2, 3, 4, 6.  Storage of an M x K operand, two byte arrays:
 *     codes   row i at Q + i*ldq, k in the low (k even) or high (k odd) half
 *             of byte k/2; ldq >= gemm_mx4_code_pitch(K) = 16*ceil(K/32)
 *             bytes.  The codes of k >= K in the last block are zero.
 *     scales  row i at S + i*lds, block k/32 at byte k/32;
 *             lds >= gemm_mx4_scale_pitch(K) = 16*ceil(K/512) bytes.  The
 *             bytes past block (K-1)/32 are never used.
 * Pitches and bases are multiples of 16 bytes (GEMM_ERR_ALIGN otherwise), and
 * pitches at most DGT_GEMM_MX4_MAX_PITCH (a pitch outside the two limits is
 * GEMM_ERR_LD; K is so limited to 2^25).  Blocks always run along the
 * summation index, so both operands of a product are stored with k
 * contiguous: A as M x K, B as N x K (a linear layer's weight as it is).  The
 * three products of a training step of Y = X*W^T take the operands quantised
 * along their own summation index (gemm_mx4_quantize with trans = 1 reads
 * the stored transpose): X and W along [in]; G and W^T along [out]; G^T and
 * X^T along the batch.
 *
 * Checks run in this order: dtype and flags, dimensions, pitches, quick
 * return for an empty result, null pointers, alignment, overlap.  A call that
 * needs more workgroups than one launch holds (2^32 threads: products from
 * 2^23 strips of 64 rows by 128 columns on, 16-bit A off 16-byte rows from strips of
 * 16 rows) is GEMM_ERR_DIM. */

#define DGT_GEMM_MX4_MAX_PITCH (1 << 24)

/* Smallest row pitches in bytes for K elements (0 for K <= 0).  Host only. */
int64_t gemm_mx4_code_pitch(int K);
int64_t gemm_mx4_scale_pitch(int K);

/* Q, S <- the M x K matrix op(X) quantised: op(X)(i,k) = X[i*ldx + k]
 * (trans = 0, X stored M x K) or X[k*ldx + i] (trans = 1, X stored K x M);
 * X in the input format `dtype`, any alignment.  Per block: with amax the
 * largest magnitude, e = floor(log2(amax)) - 2 clamped to [-127, 127] (-127
 * when amax = 0) and s = e + 127; each element x becomes the code nearest to
 * x * 2^-e, ties to the even code, magnitudes above 6 to 6.  A block that
 * holds an infinity or a NaN gets s = 255 and zero codes.  The codes past K
 * in the last block are written as zeros, and the scale bytes past the last
 * block up to gemm_mx4_scale_pitch(K) as 127; nothing past those pitches is
 * written. */
int gemm_mx4_quantize(int dtype, int trans, int M, int K, const void* X, int ldx,
                      uint8_t* Q, int ldq, uint8_t* S, int lds, void* stream);

/* Y (M x K, row pitch ldy elements, format `dtype`) <- the values of Q, S.
 * FP32 and BF16 hold every value exactly (a block's 6 * 2^127 and its like
 * overflow to infinity); FP16 is rounded to nearest even. */
int gemm_mx4_dequantize(int dtype, int M, int K, const uint8_t* Q, int ldq,
                        const uint8_t* S, int lds, void* Y, int ldy, void* stream);

/* C <- alpha*A*B^T + beta*C + bias with MX4 A (M x K; codes A, scales SA) and
 * B (N x K; codes B, scales SB), fp32 accumulate and output; bias is NULL or
 * N floats added to every row of C, unscaled.  alpha == 0 or K == 0 reads
 * neither operand. */
int gemm_mx4(int M, int N, int K, float alpha, const uint8_t* A, int lda,
             const uint8_t* SA, int ldsa, const uint8_t* B, int ldb,
             const uint8_t* SB, int ldsb, float beta, float* C, int ldc,
             const float* bias, void* stream);

/* The same with 16-bit A (GEMM_DTYPE_BF16 or GEMM_DTYPE_F16, M x K, row pitch
 * lda elements, any alignment) against MX4 B: the products of a 16-bit and a
 * 4-bit value are exact and summed in fp32 (with BF16 A a weight of 2^128 or
 * more, which gemm_mx4_quantize never writes, counts as infinite).  For
 * batches of up to some hundred rows: from about 800 (BF16) or 300 (FP16) rows on,
 * gemm_mx4_dequantize and the dense product take less time, where there is
 * room for the result.  A whose rows are not on 16-byte boundaries (K, or a
 * padded pitch, not a multiple of 8) streams B once per 16 or 32 rows and takes
 * 2 to 6 times as long from 8 rows on; a padded copy of A is faster. */
int gemm_mx4_a16(int dtype, int M, int N, int K, float alpha, const uint16_t* A,
                 int lda, const uint8_t* B, int ldb, const uint8_t* SB, int ldsb,
                 float beta, float* C, int ldc, const float* bias, void* stream);

/* ------------------------------------------------------- orthogonalisation
 *
 * O_z <- NS(G_z) for z = 0 .. batch-1: the M x N matrix G_z moved towards the
 * nearest matrix with orthonormal rows (M <= N) or columns (M > N) by `steps`
 * Newton-Schulz steps, as optimisers that orthogonalise a weight's update do:
 *
 *     X <- G / (|G|_F + eps)
 *     steps times:  M <= N:  S = X*X^T,  X <- a*X + (b*S + c*S*S)*X
 *                   M > N:   S = X^T*X,  X <- a*X + X*(b*S + c*S*S)
 *
 * G in the format `dtype` (row pitch ldg, problem stride stride_g elements),
 * O as raw bf16 bits (ldo, stride_o).  The norm is summed in 64 bits.  The
 * products take FP16 operands (scaled by powers of two into its range) and
 * sum in fp32; X itself is carried in two FP16 halves of together 22 bits,
 * and the term a*X uses both; the diagonal of b*S + c*S*S keeps 32 bits.
 * Normwise the result of five steps with the usual coefficients differs from
 * the exact iteration by 1.7e-3 (low rank, fast falling spectra) to 2.5e-3
 * (normal values, single rows), of which its own rounding to bf16 is 1.7e-3.  Every intermediate stays in range
 * while the iterates' singular values t do below 4 with
 * |b*t^2 + c*t^4| below 60.  A matrix holding an infinity or a NaN gives
 * NaN, and so does a zero matrix with eps = 0; neither touches the other
 * problems of the batch.
 *
 * The workspace (device memory, 16-byte aligned, at least
 * gemm_orthogonalize_workspace_size bytes) must not overlap G or O and must
 * stay untouched until the work on `stream` has finished; calls that may run
 * at the same time (other streams, captured graphs) need workspaces of their
 * own.  G is read completely before O is written, so O may be G's memory.
 * The problems' O ranges must be disjoint.  steps must be 1 to 64, a, b, c
 * finite and eps >= 0; batch 1 to 65535 (0 does nothing).  M is at most 2^26
 * and N at most 2^24 (GEMM_ERR_DIM otherwise, in both calls): longer rows pass the
 * kernels' 32-bit offsets, more rows leave FP16's range. */
int gemm_orthogonalize(int dtype, int M, int N, const void* G, int ldg,
                       int64_t stride_g, uint16_t* O, int ldo, int64_t stride_o,
                       int batch, int steps, float a, float b, float c, float eps,
                       void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace gemm_orthogonalize needs (0 for an empty call), or a
 * negative status for arguments outside its limits.  Host only. */
int64_t gemm_orthogonalize_workspace_size(int M, int N, int batch);

/* ------------------------------------------------- gated feed-forward block
 *
 * The first half of a gated feed-forward block, both projections, the
 * activation and the elementwise product in one kernel:
 *
 *     g = X*Wg^T + bias_g,   u = X*Wu^T + bias_u,   H = act(g) * u
 *
 * X is M x K, Wg and Wu are N x K (a linear layer's weights as stored), H is
 * M x N; X, the weights and H are raw 16-bit values of one format, `dtype`
 * (GEMM_DTYPE_BF16 or GEMM_DTYPE_F16).  The biases are fp32, N values, each
 * optional (NULL).  Sums are fp32; H, and g and u where they are asked for (G and U,
 * each optional: what the gradient needs), are each rounded once, to nearest
 * even, H from the unrounded g and u.  The two weights may be row halves, and G and U
 * column halves, of one matrix.  K == 0 leaves the biases (or zeros).
 *
 * Activations: */
enum gemm_activation {
    GEMM_ACT_SILU = 0,          /* x / (1 + exp(-x))                         */
    GEMM_ACT_GELU = 1,          /* x * P(normal variable < x)                */
    GEMM_ACT_GELU_TANH = 2,     /* x/2 * (1 + tanh(sqrt(2/pi) *
                                   (x + 0.044715*x^3)))                      */
    GEMM_ACT_RELU = 3,          /* max(x, 0); slope 0 at 0                   */
    GEMM_ACT_SIGMOID = 4,       /* 1 / (1 + exp(-x))                         */
    GEMM_ACT_IDENTITY = 5       /* x                                         */
};

/* Largest M, N and K of the gated calls and of those on 4-bit weights with
 * group scales (N: half of it for gemm_w4_gated; GEMM_ERR_DIM above). */
#define DGT_GEMM_GATED_MAX_DIM (1 << 28)

/* Any alignment of 2 bytes.  Rows on 16-byte boundaries (bases and pitches of X
 * and the weights) with pitches below 2^24 take the faster kernels.  H, G
 * and U must not overlap each other or an input (GEMM_ERR_OVERLAP; column
 * ranges of one matrix, with one pitch, do not overlap).  Checks run in this order:
 * dtype and activation, dimensions, pitches, quick return for an empty H, null
 * pointers, overlap.  A call that needs more workgroups than one launch holds (2^32
 * threads: from 2^24 tiles of 128 rows by 64 columns on) is GEMM_ERR_DIM. */
int gemm_gated(int dtype, int act, int M, int N, int K, const uint16_t* X, int ldx,
               const uint16_t* Wg, int ldwg, const uint16_t* Wu, int ldwu,
               const float* bias_g, const float* bias_u, uint16_t* H, int ldh,
               uint16_t* G, int ldg, uint16_t* U, int ldu, void* stream);

/* The gradient at the projections of a block whose second half is Y = H*Wd^T,
 * from dY (M x K) and Wd as stored (K x N):
 *
 *     dh = dY*Wd,  dG = dh * U * act'(G),  dU = dh * act(G)
 *
 * with G and U as gemm_gated kept them; H = act(G) * U again where it is asked
 * for (optional; what Wd's gradient dY^T*H needs), and the biases' gradients, the column sums of dG
 * and dU before their rounding (each optional, N floats).  dh itself never
 * reaches memory.  With dG and dU column halves of one matrix D and the weights row halves of
 * one matrix W, the rest of the block's gradient is two products: dX = D*W,
 * dW = D^T*X.  dG may be G's memory and dU may be U's (same base and pitch);
 * otherwise no output may overlap another or an input.
 *
 * Only calls that ask for a bias's gradient need the workspace (16-byte aligned,
 * gemm_gated_grad_workspace_size bytes; GEMM_ERR_WORKSPACE, GEMM_ERR_ALIGN); it must
 * stay untouched until the work on `stream` has finished, and calls that may run at
 * the same time need workspaces of their own.  The sums' order is fixed.  M == 0
 * writes zeros to them.  Checks as for gemm_gated. */
int gemm_gated_grad(int dtype, int act, int M, int N, int K, const uint16_t* dY,
                    int lddy, const uint16_t* Wd, int ldw, const uint16_t* G, int ldg,
                    const uint16_t* U, int ldu, uint16_t* dG, int lddg, uint16_t* dU,
                    int lddu, uint16_t* H, int ldh, float* dbias_g, float* dbias_u,
                    void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace a gemm_gated_grad call with a bias's gradient needs, or a
 * negative status.  Host only. */
int64_t gemm_gated_grad_workspace_size(int M, int N);

/* ------------------------------------- 4-bit weights with group scales (W4)
 *
 * A row of K elements is cut into groups of `group` (32, 64 or 128)
 * consecutive k; element k stands for
 *
 *     s * (q - z)
 *
 * with q its code 0 .. 15, s the group's scale and z its zero point.  Storage
 * of an operand of M rows:
 *     codes   as MX4's: row i at Q + i*ldq, k in the low (k even) or high (k
 *             odd) half of byte k/2; ldq >= gemm_mx4_code_pitch(K), at most
 *             DGT_GEMM_MX4_MAX_PITCH, and Q and ldq multiples of 16 bytes
 *             (GEMM_ERR_ALIGN).  What the last 16 bytes hold past K is never used.
 *     scales  row i at S + i*lds (16-bit elements of `scale_dtype`,
 *             GEMM_DTYPE_BF16 or GEMM_DTYPE_F16), lds >= ceil(K/group)
 *     zeros   row i at Z + i*ldz, one byte per group, 0 .. 255; Z == NULL: 8
 *             everywhere (ldz is not looked at)
 *
 * Checks run in this order: dtypes, activation and group, dimensions, pitches,
 * quick return for an empty result, null pointers, alignment, overlap.  A product that needs
 * more workgroups than one launch holds (2^32 threads: from 2^23 strips of 32 rows by 64
 * rows of the weight on, counted eight at a time along the weight) is GEMM_ERR_DIM. */

/* Q, S, Z <- the M x K matrix X in the input format `dtype`, any alignment.
 * Per group, over its elements and 0: with Z, s = (max - min)/15 and
 * z = -min/s to the nearest whole number, at most 15; with Z == NULL, s = max(max/7, -min/8).
 * s is rounded to fp32 and then to its type (past the type's largest value: that
 * value); x becomes the whole number nearest to x/s (ties to even) plus z, within
 * 0 .. 15.  A group whose scale comes out as 0 gets the code z.  A
 * group that holds an infinity or a NaN gets the scale NaN and zero codes.  The codes past K in the
 * last 16 bytes are written as zeros; nothing past those is written. */
int gemm_w4_quantize(int dtype, int group, int scale_dtype, int M, int K,
                     const void* X, int ldx, uint8_t* Q, int ldq, void* S, int lds,
                     uint8_t* Z, int ldz, void* stream);

/* Y (M x K, row pitch ldy elements, format `dtype`) <- the operand's values,
 * exact in FP32, rounded to nearest even otherwise. */
int gemm_w4_dequantize(int dtype, int group, int scale_dtype, int M, int K,
                       const uint8_t* Q, int ldq, const void* S, int lds,
                       const uint8_t* Z, int ldz, void* Y, int ldy, void* stream);

/* C <- alpha*A*W^T + beta*C + bias with 16-bit A (`dtype`, M x K, any alignment)
 * and W the N x K operand Q, S, Z: for products of few rows (from a few hundred rows on,
 * gemm_w4_dequantize and a dense product are faster).  Above 16 rows A is read fastest
 * from 16-byte rows with a pitch below 2^24.  Weights are not rounded:
 * within a group x*q and x are summed apart in fp32, and s*(sum xq - z*sum x) is
 * added up in fp32.  So the error goes by the sizes of s*q*x and s*z*x, also where the
 * two sums cancel; an infinite or NaN x makes its whole row of C (of H below) NaN; and a
 * group whose |x| add up to 2^119 or more, as only BF16 can, may become infinite or NaN
 * though s*(q - z)*x are not.  bias: NULL or N floats.  alpha == 0 or K == 0 reads neither
 * operand, beta == 0 does not read C. */
int gemm_w4_a16(int dtype, int group, int scale_dtype, int M, int N, int K,
                float alpha, const uint16_t* A, int lda, const uint8_t* Q, int ldq,
                const void* S, int lds, const uint8_t* Z, int ldz, float beta,
                float* C, int ldc, const float* bias, void* stream);

/* gemm_gated on such weights, one operand of 2N rows: Wg's, then Wu's.  H as
 * there, M x N; no pre-activations are kept. */
int gemm_w4_gated(int dtype, int act, int group, int scale_dtype, int M, int N, int K,
                  const uint16_t* X, int ldx, const uint8_t* Q, int ldq, const void* S,
                  int lds, const uint8_t* Z, int ldz, const float* bias_g,
                  const float* bias_u, uint16_t* H, int ldh, void* stream);

/* The rung GEMM_VARIANT_AUTO picks for this call (dtype: enum gemm_dtype;
 * trans_a, trans_b as for gemm_ex), or a negative status if the arguments
 * are invalid.  Host only: touches no device and queues nothing. */
int gemm_select_variant(int dtype, int trans_a, int trans_b, int M, int N,
                        int K, int lda, int ldb, int ldc);

/* Static string naming a status code (never NULL). */
const char* gemm_status_string(int status);

/* DGT_GEMM_ABI_VERSION of the built library. */
int gemm_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* DGT_GEMM_H */
