/*
 * sgemm_i8 — products of 8-bit integers with a scale for each row of both
 * operands (tokens and channels), and the quantisation that makes them, for AMD
 * Instinct MI355X (gfx950).
 *
 * The same library, statuses and conventions as sgemm_f32.h and sgemm_f8.h:
 * row-major DEVICE pointers owned by the caller, leading dimensions in elements,
 * arguments checked on the host before any HIP call, work enqueued on `stream`
 * with no synchronisation, no allocation and no device-side state kept between
 * calls.
 */
#ifndef SGEMM_I8_H
#define SGEMM_I8_H

#include "sgemm_f8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest K: the sum of that many products of 8-bit integers (at most 2^14 each)
 * fits 32 bits. */
#define SGEMM_I8_MAX_K 131071

/*
 * C <- alpha * diag(SA) * A * B^T * diag(SB) + beta * C:
 *   A   M x K 8-bit integers (-128 .. 127), SA M consecutive scales (a token's each);
 *   B   N x K 8-bit integers, SB N consecutive scales (a channel's each);
 *   C   M x N of type c_type (sgemm_type).
 * The sum over k is exact in 32-bit integers, is turned into FP32 (one rounding from
 * 2^24 on) and multiplied by SA[m], SB[n] and alpha in that order in FP32; beta * C is
 * added and C rounded once.  The result does not depend on the workspace.
 * alpha == 0 or K == 0: C <- beta * C and A, B and their scales are not read.
 *
 * A, lda, B and ldb may have any alignment; bases and leading dimensions that are
 * multiples of 16 (and at most 2^22) run on the fast kernels, which read the 16 bytes
 * holding the last values of a row whole and ignore those past K.
 *
 * workspace (NULL or 16-byte aligned, workspace_bytes long, overlapping no operand):
 * where too few output tiles exist to fill the GPU, k is split over workgroups whose
 * partial sums go there; operands at other alignments are laid out there where that
 * is faster.  sgemm_i8_gemm_workspace says how many bytes serve; with fewer, or none,
 * the call takes the fastest way that fits.  Calls, and captured graphs, that share a
 * workspace must not run at once.
 *
 * SGEMM_ERR_INVALID_VALUE: an unknown type; a dimension below 0, K above
 * SGEMM_I8_MAX_K, M or N above 2^31 - 1025; a leading dimension below its row
 * length; NULL or misaligned (for its element type) pointers to operands that are
 * touched; workspace_bytes below 0; a grid beyond one launch.  SGEMM_ERR_ALIAS: C or
 * the workspace overlaps an operand.
 */
int sgemm_i8_gemm(int c_type, int64_t M, int64_t N, int64_t K, float alpha, const int8_t *A, int64_t lda,
                  const float *SA, const int8_t *B, int64_t ldb, const float *SB, float beta, void *C, int64_t ldc,
                  void *workspace, int64_t workspace_bytes, void *stream);

/* Host-only planning query: the kernel (0: nothing or no product to compute), its
 * grid of output tiles, the k-splits it makes with a sufficient workspace and the
 * bytes of their partial sums (0: unsplit), operands staying where they are.
 * `aligned`: whether A, lda, B and ldb are all multiples of 16 and lda and ldb at
 * most 2^22.  Output pointers may be NULL. */
int sgemm_i8_gemm_plan(int64_t M, int64_t N, int64_t K, int aligned, int *kernel_id, int64_t *tiles_m,
                       int64_t *tiles_n, int64_t *splits, int64_t *workspace_bytes);

/* Host-only query: the workspace with which sgemm_i8_gemm is fastest (0: none). */
int sgemm_i8_gemm_workspace(int64_t M, int64_t N, int64_t K, int aligned, int64_t *workspace_bytes);

/*
 * Quantise each row of X (rows x cols of x_type) to 8-bit integers:
 *     a = max(max|x|, 2^-90),  S[row] = a / 127,  q = 127 * x / a
 * to the nearest integer, ties to even, exactly (of the real quotient, not of a
 * rounded one); |q| <= 127.  A row holding a NaN or an infinity gets a NaN or
 * infinite scale and q = 0 throughout, so that what it stands for is NaN.
 * S is rows consecutive FP32 values.  X, Q and S do not overlap (SGEMM_ERR_ALIAS).
 * Rows or cols of 0: nothing is touched.  The rows' work-items (16 a row up to 128
 * columns, 32 up to 256, 64 up to 1024, 256 up to 4096, 512 up to 8192 and 1024
 * above) have to fit one launch of 2^32 - 1: SGEMM_ERR_INVALID_VALUE.
 */
int sgemm_i8_quantize(int x_type, int64_t rows, int64_t cols, const void *X, int64_t ldx, int8_t *Q, int64_t ldq,
                      float *S, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_I8_H */
