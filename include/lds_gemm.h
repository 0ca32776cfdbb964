/*
 * lds_gemm.h -- C ABI of the LDS-staged BF16/FP16 GEMM for AMD Instinct
 * MI355X (gfx950, CDNA4), and of the operators of a quantised linear layer
 * beside it: the RMS norm that makes a product's A operand (gemm_rmsnorm_run),
 * the E4M3 product with row and column scales (gemm_scaled_run) and the
 * product of a few rows with 4-bit weights (gemm_w4_run); of the products of
 * rows that belong to groups, each group with a matrix of its own, and their
 * gradients (gemm_grouped_run, gemm_grouped_wgrad_run); and of MXFP4, 4-bit
 * floats with a scale for 32 of them: conversions (gemm_mxfp4_quantize_run,
 * gemm_mxfp4_dequantize_run) and products (gemm_mxfp4_run,
 * gemm_grouped_mxfp4_run).
 *
 * Operation (gemm_run; the others say theirs): C <- A * B, with
 *     C[m][n] = sum_{k<K} a(m,k) * b(k,n)
 * accumulated in fp32 by the matrix cores and converted once when stored.
 *   - "An educational GEMM ladder for Helios GPUs", section "Educational GEMM
 *     Ladder": each rung computes C = AB, A in R^{MxK}, B in R^{KxN},
 *     C in R^{MxN}, BF16 inputs.
 *   - Same page, "Level 0 APIs" table: the matrix instruction accumulates the
 *     16-bit product into FP32 registers; the store converts the FP32
 *     accumulator and writes it to global memory.
 *   - Operand contiguity: "A Deep Dive into LDS Optimizations on AMD Instinct
 *     MI450 GPUs", Part I, "Why Is It Important?" (a K-contiguous or an
 *     N-contiguous operand reaches the matrix cores through LDS).
 *
 * Layout of the operands of gemm_run and gemm_scaled_run (leading dimensions
 * count ELEMENTS, not bytes):
 *     layoutA == GEMM_K_CONTIG : a(m,k) = A[m*lda + k]   (row-major M x K)
 *     layoutA == GEMM_MN_CONTIG: a(m,k) = A[k*lda + m]   (column-major M x K)
 *     layoutB == GEMM_MN_CONTIG: b(k,n) = B[k*ldb + n]   (row-major K x N)
 *     layoutB == GEMM_K_CONTIG : b(k,n) = B[n*ldb + k]   (column-major K x N)
 *     C is row-major:            C[m*ldc + n]
 * Only the M x N entries of C are written; C memory between N and ldc is
 * left untouched.  Inputs beyond M, N or K are never read.
 *
 * Ownership and asynchrony: the caller owns the operands (device memory of
 * the handle's device) and keeps them alive until the work queued on `stream`
 * has finished.  The library never allocates, frees or retains caller
 * memory and allocates no workspace.  The *_run functions only enqueue
 * work on `stream` and return without synchronising the host; each launches
 * one kernel and nothing else (no allocation, memset or copy), so a call made
 * while `stream` is being captured into a HIP graph is captured and replays.
 * A result depends on the operands alone: sums have a fixed order.
 *
 * Errors: every function returns a gemm_status.  Arguments are validated
 * before anything is launched; on an error nothing is enqueued and the outputs
 * are untouched.  Sizes (M, N, K, T) are below 2^30, leading dimensions and
 * strides below 2^40 where no other limit is given, and no operand spans 2^63
 * bytes or more.  No C++ exception crosses this interface.  Handles are
 * immutable after creation, so one handle may be used from several host
 * threads and streams at once.  Two operands overlap when the spans from
 * their first to their last element do.
 */
#ifndef LDS_GEMM_H
#define LDS_GEMM_H

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct gemm_ctx *gemm_handle_t;

/* Which index of an operand is unit-stride in memory. */
enum gemm_layout {
    GEMM_K_CONTIG = 0,   /* K is contiguous (A row-major, B column-major)  */
    GEMM_MN_CONTIG = 1   /* M (for A) or N (for B) is contiguous           */
};

/* Element types, named input_output; accumulation is always fp32.
 * E4M3 is the OCP 8-bit floating-point format with 4 exponent bits (bias 7),
 * 3 fraction bits and no infinities, one byte per element; its products run
 * on the gfx950 fp8 matrix instruction ("Lds Optimization", "MFMA Transpose
 * Load from LDS (gfx950 only)": DS_READ_B64_TR_B8 feeds 8-bit MFMA
 * operands). */
enum gemm_dtype {
    GEMM_BF16_F32 = 0,   /* bf16 A, B;  fp32 C                             */
    GEMM_BF16_BF16 = 1,  /* bf16 A, B;  bf16 C (round to nearest even)     */
    GEMM_F16_F16 = 2,    /* fp16 A, B;  fp16 C (round to nearest even)     */
    GEMM_F16_F32 = 3,    /* fp16 A, B;  fp32 C                             */
    GEMM_E4M3_F32 = 4,   /* fp8 E4M3 A, B;  fp32 C                         */
    GEMM_E4M3_BF16 = 5,  /* fp8 E4M3 A, B;  bf16 C (round to nearest even) */
    GEMM_E4M3_F16 = 6    /* fp8 E4M3 A, B;  fp16 C: gemm_scaled_run only   */
};

/* Added to gemm_scaled_run's dtype: sums of exact products in fp32 for 16-bit
 * output too, at up to twice the time (fp32 output always has them). */
enum { GEMM_EXACT_SUMS = 0x100 };

/* The 16- or 32-bit type beside MXFP4: of the matrix that is quantised, of the
 * values that come back, of a product's C. */
enum gemm_mxfp4_dtype {
    GEMM_MXFP4_BF16 = 0,
    GEMM_MXFP4_F16 = 1,
    GEMM_MXFP4_F32 = 2
};

/* Element types of gemm_rmsnorm_run, named input_output. */
enum gemm_norm_dtype {
    GEMM_NORM_BF16_BF16 = 0,
    GEMM_NORM_BF16_E4M3 = 1,
    GEMM_NORM_F16_F16 = 2,
    GEMM_NORM_F16_E4M3 = 3
};

enum gemm_status {
    GEMM_OK = 0,
    GEMM_ERR_INVALID_ARG = 1,   /* bad enum, negative size, NULL pointer, ld too small, an output overlaps another operand */
    GEMM_ERR_UNSUPPORTED = 2,   /* valid request the kernels cannot serve: misaligned pointer or ld, size of 2^30 or more, an operand spanning 2^63 bytes or more, a launch of 2^32 threads or more */
    GEMM_ERR_DEVICE = 3,        /* no device, not a gfx950 device, or the current device is not the handle's */
    GEMM_ERR_LAUNCH = 4         /* the HIP runtime rejected the kernel launch */
};

/* Create a handle bound to the calling thread's current HIP device.
 * Fails with GEMM_ERR_DEVICE unless that device is gfx950.  *out receives
 * the handle (NULL on failure); release it with gemm_destroy. */
int gemm_create(gemm_handle_t *out);

/* Enqueue C <- A*B on `stream` (0 = the device's null stream).
 *   A, B       device pointers to bf16/fp16 (2-byte) or E4M3 (1-byte)
 *              elements, 16-byte aligned; lda/ldb must be multiples of 16
 *              bytes (8 bf16/fp16 or 16 E4M3 elements).  E4M3 inputs further
 *              need the contiguous extents (K or M of A, N or K of B) to be
 *              multiples of 16 elements, else GEMM_ERR_UNSUPPORTED.
 *   C          device pointer to fp32 (4-byte aligned) or bf16/fp16
 *              (2-byte aligned) elements; must not overlap A or B.
 *   M, N, K    sizes, 0 <= size < 2^30; lda, ldb, ldc < 2^40; no operand may span 2^63 bytes
 *              or more ((rows - 1) * ld + row length, in bytes).  M == 0 or N == 0 is a no-op;
 *              K == 0 writes zeros (the empty sum) to the M x N block of C.
 *   lda        >= K (layoutA K-contig) or >= M (MN-contig)
 *   ldb        >= N (layoutB MN-contig) or >= K (K-contig)
 *   ldc        >= N
 *   layoutA/B  enum gemm_layout;  dtype  enum gemm_dtype.
 * Must be called with the handle's device current. */
int gemm_run(gemm_handle_t h, const void *A, const void *B, void *C,
             int64_t M, int64_t N, int64_t K,
             int64_t lda, int64_t ldb, int64_t ldc,
             int layoutA, int layoutB, int dtype, hipStream_t stream);

/* Enqueue C <- diag(SA) * A * B * diag(SB) on `stream`, for E4M3 operands:
 *     C[m][n] = round( (sum_k a(m,k) * b(k,n)) * SA[m*incA] * SB[n*incB] )
 * with the sum in fp32, the two factors applied to it in fp32 in that order,
 * and one rounding to C's type.  For fp32 output, for M <= 32 and where dtype
 * has GEMM_EXACT_SUMS, the sum is one of exact products in fp32.  For 16-bit
 * output of more rows the fp8 matrix instruction may make it, which takes eight
 * products at a time, aligns them to the largest and drops what lies 13 bits or
 * more below (the sum so far is not aligned to them and keeps fp32's bits): at
 * most 7 * 2^-13 of a group's largest product is lost, 2^-10 sum |a b| in all;
 * 1.5e-5 of the result on normal data and 5e-5 where one k in a hundred is twenty
 * times louder, against 1.7e-3 (bf16) or 2e-4 (fp16) of the output's rounding.
 * A sum of which large products cancel may lose all of a small result to it.
 *   SA, SB       device pointers to fp32 scales, 4-byte aligned: one for each
 *                row of A and each column of B (incA, incB = 1), or one for
 *                all of them (0).  They must not overlap C.
 *   dtype        GEMM_E4M3_F32, GEMM_E4M3_BF16 or GEMM_E4M3_F16, or one of them
 *                + GEMM_EXACT_SUMS.
 * Everything else is as for gemm_run with E4M3 operands, K == 0 included: the
 * empty sum is scaled like any other. */
int gemm_scaled_run(gemm_handle_t h, const void *A, const void *B, void *C,
                    const float *SA, const float *SB,
                    int64_t M, int64_t N, int64_t K,
                    int64_t lda, int64_t ldb, int64_t ldc,
                    int incA, int incB,
                    int layoutA, int layoutB, int dtype, hipStream_t stream);

/* Enqueue, on `stream`, the product of 16-bit rows with 4-bit weights that
 * carry a scale and a zero point for every `group` consecutive k:
 *     C[m][n] = round( sum_k A[m*lda + k] *
 *               S[(k/group)*lds + n] * (q(k,n) - Z[(k/group)*ldz + n]) )
 * summed in fp32, one rounding to C's type.  The zero point is taken off the
 * group's sum, sum A (16 + q) - (16 + Z) sum A, or, for fp16 of more than 16 rows,
 * off each weight; so before the rounding an entry is within
 *     2^-23 (min(group, K) + K/group + 21) sum_k |A S| (47 + Z)
 * of the formula; on ordinary data, also with activations far from zero in the
 * mean, the relative error (2-norm) is 3e-7 at most.  Meant for few rows (M <= 48:
 * the weights are read once); any M is computed, the weights being read again
 * for every 32 or 48 rows.
 *   A            bf16/fp16, K-contiguous, 16-byte aligned; lda a multiple of 8.
 *   B            q(k,n) = bits 4*(k&1) .. 4*(k&1)+3 of byte (n*ldb + k)/2: two
 *                weights a byte, K-contiguous, even k in the low half.  16-byte
 *                aligned; ldb counts weights and is a multiple of 32.
 *   S            scales of A's type, one row of N for each group of k.
 *   Z            zero points, unsigned bytes, one row of N for each group; or
 *                NULL: every zero point is 8.
 *   K            a multiple of 32; K == 0 writes zeros and reads nothing.
 *   group        a power of two, 32 or more; the last group may be cut short
 *                by K, and a group of K or more is one scale for a column.
 *   lda, ldb >= K, lda < 2^24, ldb < 2^25; lds, ldc >= N, ldz >= N with Z, each
 *                < 2^40.
 * An entry whose sum over 16 + q and its correction is not finite is summed
 * again term by term in fp64, so infinities and NaNs come out as the formula has
 * them, and finite sums of terms beyond fp32 too.
 *   dtype        GEMM_BF16_F32, GEMM_BF16_BF16, GEMM_F16_F16 or GEMM_F16_F32.
 * C is 4-byte (fp32) or 2-byte aligned and overlaps no input. */
int gemm_w4_run(gemm_handle_t h, const void *A, const void *B, const void *S,
                const void *Z, void *C,
                int64_t M, int64_t N, int64_t K, int64_t group,
                int64_t lda, int64_t ldb, int64_t lds, int64_t ldz, int64_t ldc,
                int dtype, hipStream_t stream);

/* Enqueue the root-mean-square norm of the rows of X, or of X + R, on `stream`:
 *     h[m][n] = X[m*ldx + n] + R[m*ldr + n]        (without R: X alone)
 *     y[m][n] = h[m][n] * W[n] / sqrt(mean over n of h[m][n]^2 + eps)
 *     H[m*ldh + n] = h rounded to X's type
 *     Y[m*ldy + n] = y rounded to X's type, or, for E4M3 output,
 *     S[m] = max(max over n of |y[m][n]|, 2^-100) / 448 and
 *     Y[m*ldy + n] = y[m][n] / S[m] rounded to E4M3,
 * so that S and Y are the SA and A of gemm_scaled_run.  All arithmetic is
 * fp32, the squares included (rows whose squares' sum overflows there give
 * zeros; with eps == 0, rows whose squares all vanish there give NaN and
 * infinities), and y is computed from h before it is rounded.  A NaN in a row
 * makes all of its y NaN; an infinity is NaN at its place and makes the others
 * zero; with E4M3 output either one makes the row and S[m] NaN.
 *   X, R, W, H   elements of the input type, 2-byte aligned; R and H may be
 *                NULL (no residual; h not wanted).
 *   Y            input type (2-byte aligned) or E4M3; S is used for E4M3 only.
 *   ldx, ldy >= N, ldr >= N with R, ldh >= N with H; each < 2^40.
 *   eps >= 0;  M == 0 or N == 0 is a no-op.
 * H and a 16-bit Y may each stand in the place of X or of R (same address and
 * leading dimension); no other overlap with an output is allowed. */
int gemm_rmsnorm_run(gemm_handle_t h, const void *X, const void *R, const void *W,
                     void *H, void *Y, float *S,
                     int64_t M, int64_t N,
                     int64_t ldx, int64_t ldr, int64_t ldh, int64_t ldy,
                     float eps, int dtype, hipStream_t stream);

/* Enqueue the conversion of the M x K matrix X to MXFP4 on `stream`.
 *
 * MXFP4 (OCP Microscaling Formats 1.0): 4-bit E2M1 elements (0, 0.5, 1, 1.5, 2,
 * 3, 4, 6 and a sign) and one E8M0 scale, 2^(S - 127), for every block of 32
 * consecutive k.  An MXFP4 matrix of M rows is two arrays:
 *     Q    q(m,k) = bits 4*(k&1) .. 4*(k&1)+3 of byte (m*ldq + k)/2: two elements
 *          a byte, even k in the low half;
 *     S    S[(k/32)*lds + m]: a row of M scales for each 32 k.
 * For each block, with the largest |x| in it,
 *     S = 255 (NaN) and zero elements if the block holds an infinity or a NaN;
 *     S = max(floor(log2(max|x|)) - 2 + 127, 0), or 0 for a block of zeros, and
 *     q = x / 2^(S - 127), rounded to nearest even, sizes beyond 6 to 6.
 *   X            bf16, fp16 or fp32 elements (dtype), aligned to their size;
 *                layoutX GEMM_K_CONTIG: x(m,k) = X[m*ldx + k], ldx >= K;
 *                GEMM_MN_CONTIG: x(m,k) = X[k*ldx + m], ldx >= M.
 *   Q            16-byte aligned; ldq >= K counts elements, a multiple of 32.
 *   S            16-byte aligned bytes; lds >= M, a multiple of 16.
 *   M, K         sizes, K a multiple of 32; M == 0 or K == 0 is a no-op.
 * Of Q and S only what stands for the M x K elements is written.  X, Q and S do
 * not overlap. */
int gemm_mxfp4_quantize_run(gemm_handle_t h, const void *X, void *Q, void *S,
                            int64_t M, int64_t K, int64_t ldx, int64_t ldq, int64_t lds,
                            int layoutX, int dtype, hipStream_t stream);

/* Enqueue the values of an MXFP4 matrix on `stream`:
 *     Y[m*ldy + k] = q(m,k) * 2^(S[(k/32)*lds + m] - 127)
 * rounded to dtype's type, to nearest even (bf16 and fp32 hold every such value
 * but those beyond their range); a NaN scale makes its block NaN.  Arguments as
 * for gemm_mxfp4_quantize_run, with ldy >= K; Y does not overlap Q or S. */
int gemm_mxfp4_dequantize_run(gemm_handle_t h, const void *Q, const void *S, void *Y,
                              int64_t M, int64_t K, int64_t ldq, int64_t lds, int64_t ldy,
                              int dtype, hipStream_t stream);

/* Enqueue the product of two MXFP4 matrices on `stream`, B being N x K:
 *     C[m][n] = round( sum_k qa(m,k) 2^(SA[(k/32)*ldsa + m] - 127)
 *                          * qb(n,k) 2^(SB[(k/32)*ldsb + n] - 127) )
 * Products are exact and summed in fp32 by the matrix cores, with one rounding to
 * C's type: before it an entry is within
 *     (K/128 + 8) (2^-21 sum_k |a b| + 2^-149)
 * of the formula (1e-7 of the result, in the 2-norm, on ordinary data), the second
 * term for products and sums below fp32's normal numbers.  Where sum_k |a b| is
 * 2^127 or more, sums on the way may overflow: such an entry may be infinite or NaN
 * whatever the formula gives.  A NaN scale makes its row or column NaN.
 *   A, SA, B, SB MXFP4 matrices as gemm_mxfp4_quantize_run writes them.  The bytes
 *                between M (N) and the next multiple of 16 in a row of scales
 *                belong to the array (its last row too), whatever they hold.
 *   lda, ldb     >= K, multiples of 32, < 2^23;  ldsa >= M, ldsb >= N, multiples
 *                of 16, < 2^27.
 *   C            of dtype's type, aligned to its size, ldc >= N, overlaps no input.
 * K == 0 writes zeros; M == 0 or N == 0 is a no-op. */
int gemm_mxfp4_run(gemm_handle_t h, const void *A, const void *B, void *C,
                   const void *SA, const void *SB,
                   int64_t M, int64_t N, int64_t K,
                   int64_t lda, int64_t ldb, int64_t ldc, int64_t ldsa, int64_t ldsb,
                   int dtype, hipStream_t stream);

/* Grouped products: T rows, sorted by group (expert), of which group g has rows
 * ends[g-1] .. ends[g]-1, the first group from row 0.  `ends` are G int32 on the
 * device, read when the work runs; nothing about the groups is known to the host.
 * An end below the ends before it counts as the largest of them, a negative one
 * as 0 and one beyond T as T, so that groups are disjoint and inside the T rows
 * whatever `ends` holds.  Groups may be empty, and rows behind the last group
 * belong to none.  G is at most 65536, and `ends` 4-byte aligned.  Ends that are
 * written while the work runs give wrong entries of C (no other memory is read or
 * written for it, and the work ends). */

/* Enqueue, on `stream`, each group's rows times the group's own matrix:
 *     C[t*ldc + n] = round( sum_k A[t*lda + k] * b(g,k,n) )   for t in group g
 *     layoutB == GEMM_K_CONTIG : b(g,k,n) = B[g*strideb + n*ldb + k]
 *     layoutB == GEMM_MN_CONTIG: b(g,k,n) = B[g*strideb + k*ldb + n]
 * Rows of C that belong to no group are left as they were.  With dC in A's place
 * and B's other layout (N and K exchanged) it is the gradient of the rows.
 *   A, B         bf16 or fp16, 16-byte aligned; lda >= K, ldb >= K (or N),
 *                lda, ldb < 2^21; lda, ldb and strideb >= 0 multiples of 8
 *                (0: one matrix for all groups).
 *   K            a multiple of 8, and N too where B is MN-contiguous.  K == 0
 *                writes zeros.  G == 0, T == 0 or N == 0 is a no-op.
 *   C            aligned to its elements, ldc >= N, overlaps no input.
 *   dtype        GEMM_BF16_F32, GEMM_BF16_BF16, GEMM_F16_F16 or GEMM_F16_F32. */
int gemm_grouped_run(gemm_handle_t h, const void *A, const void *B, void *C,
                     const int32_t *ends, int64_t G, int64_t T, int64_t N, int64_t K,
                     int64_t lda, int64_t ldb, int64_t strideb, int64_t ldc,
                     int layoutB, int dtype, hipStream_t stream);

/* Enqueue, on `stream`, the gradient of the groups' matrices:
 *     C[g*stridec + m*ldc + n] = round( sum over t in group g of
 *                                       A[t*lda + m] * B[t*ldb + n] )
 * An empty group's matrix is all zeros.  A and B are the forward's rows and the
 * gradient of its C, in the order that gives C the layout wanted.
 *   A, B         bf16 or fp16, 16-byte aligned; lda >= M, ldb >= N, multiples of
 *                8, < 2^21; M and N multiples of 8.
 *   C            aligned to its elements, ldc >= N, 2^60 > stridec >= (M-1)*ldc + N
 *                (with one group any); overlaps no input.  G == 0, M == 0 or N == 0 is a no-op.
 *   dtype        as for gemm_grouped_run. */
int gemm_grouped_wgrad_run(gemm_handle_t h, const void *A, const void *B, void *C,
                           const int32_t *ends, int64_t G, int64_t T, int64_t M, int64_t N,
                           int64_t lda, int64_t ldb, int64_t ldc, int64_t stridec,
                           int dtype, hipStream_t stream);

/* Enqueue, on `stream`, each group's MXFP4 rows times the group's own MXFP4
 * matrix of N x K: gemm_grouped_run's groups, gemm_mxfp4_run's operands and sums.
 * Group g's elements stand at element g*strideb of B (a multiple of 32) and its
 * scales at byte g*stridesb of SB (a multiple of 16). */
int gemm_grouped_mxfp4_run(gemm_handle_t h, const void *A, const void *B, void *C,
                           const void *SA, const void *SB, const int32_t *ends,
                           int64_t G, int64_t T, int64_t N, int64_t K,
                           int64_t lda, int64_t ldb, int64_t strideb, int64_t ldc,
                           int64_t ldsa, int64_t ldsb, int64_t stridesb,
                           int dtype, hipStream_t stream);

/* Release a handle.  NULL is accepted and returns GEMM_OK. */
int gemm_destroy(gemm_handle_t h);

/* Static English text for a gemm_status value ("unknown status" otherwise). */
const char *gemm_status_str(int status);

#ifdef __cplusplus
}
#endif

#endif /* LDS_GEMM_H */
