/*
 * sgemm_f8 — 8-bit block-scaled products, their quantisation, and the
 * root-mean-square norm that feeds them, for AMD Instinct MI355X (gfx950).
 *
 * The same library, statuses and conventions as sgemm_f32.h: row-major DEVICE
 * pointers owned by the caller, leading dimensions in elements, arguments
 * checked on the host before any HIP call, work enqueued on `stream` (a
 * hipStream_t; NULL: the null stream) with no synchronisation, no allocation
 * and no device-side state kept between calls.
 *
 * 8-bit operands.  A block of 128 values x with a = max(max|x|, 2^-90) is held
 * as q = round(x * (L / a)) (to nearest, ties to even) in an 8-bit format whose
 * largest value is L, with one FP32 scale s = a / L; x is about q * s.
 *   SGEMM_F8_E4M3  4 exponent and 3 mantissa bits, no infinities, L = 448
 *   SGEMM_F8_E5M2  5 exponent and 2 mantissa bits, L = 57344
 * A block holding a NaN or an infinity gets a NaN or infinite scale, and what
 * it stands for is NaN throughout: it is never silently lost.  Blocks are
 *   SGEMM_F8_ROW   128 consecutive values of one row (the last block of a row
 *                  may be shorter).  The scale of block b of row i is at
 *                  S[b*lds + i], lds >= rows: k-block major, so that a product
 *                  reads the scales of one k-block of many rows together.
 *   SGEMM_F8_TILE  128 x 128 values (shorter at the edges); the scale of tile
 *                  (i, b) is at S[i*lds + b], lds >= ceil(cols/128).
 */
#ifndef SGEMM_F8_H
#define SGEMM_F8_H

#include "sgemm_f32.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { SGEMM_F8_E4M3 = 1, SGEMM_F8_E5M2 = 2 } sgemm_f8_format;
typedef enum { SGEMM_F8_ROW = 0, SGEMM_F8_TILE = 1 } sgemm_f8_block;
/* Element types of the operands that are not 8 bits wide. */
typedef enum { SGEMM_TYPE_F32 = 0, SGEMM_TYPE_FP16 = 1, SGEMM_TYPE_BF16 = 2 } sgemm_type;

/*
 * C <- alpha * A * B^T + beta * C, A and B in 8 bits with scales per block:
 *   A   M x K in format_a, row blocks along K, scales SA (ceil(K/128) x M,
 *       leading dimension ldsa >= M);
 *   B   N x K in format_b, b_block says its blocks: SGEMM_F8_TILE (weights;
 *       scales ceil(N/128) x ceil(K/128), ldsb >= ceil(K/128)) or
 *       SGEMM_F8_ROW (ceil(K/128) x N, ldsb >= N);
 *   C   M x N of type c_type.
 * The sum of each k-block of 128 comes from the matrix cores, is multiplied by
 * (sA * sB) (one FP32 product) and added to an FP32 sum over the k-blocks; C is
 * rounded once.  With an FP32 C the k-block's sum is FP32 too (the operands go
 * through the 16-bit matrix cores, which hold every 8-bit value exactly); with
 * a 16-bit C it is that of the 8-bit matrix cores, which add products in groups
 * of 8 consecutive k, a product keeping 13 bits below the largest of its group:
 * off by at most 7 * 2^-13 of the sum of the products' absolute values, and by
 * 1.5e-5 of its size on normally distributed operands.  Where products cancel to
 * less than that, ask for an FP32 C.  The product sA * sB loses bits below 2^-126
 * (two e5m2 blocks whose maxima multiply to less than 2^-94, two e4m3 blocks to
 * less than 2^-108) and is infinite from 2^128 on.  alpha == 0 or
 * K == 0: C <- beta * C and A, B and their scales are not read.
 *
 * A, lda, B and ldb may have any alignment.  Bases and leading dimensions that
 * are multiples of 16 (and at most 2^22) run on the fast kernels, which read the
 * 16 bytes holding the last values of a row whole and ignore those past K;
 * others are assembled in registers, or (K up to 2^22) first laid out anew in the
 * workspace.  Tile scales with ldsb above 2^22 and N above 128 keep a call off the
 * fast kernels.
 *
 * workspace (NULL or 16-byte aligned, workspace_bytes long, overlapping no
 * operand): where too few output tiles exist to fill the GPU, k is split over
 * workgroups whose partial sums go there and are added in a fixed order; and
 * operands at other alignments are laid out there where that is faster.
 * sgemm_f8_gemm_workspace says how many bytes serve; with fewer, or none, the
 * call takes the fastest way that fits.  Results are the same from call to call
 * with the same workspace size.
 *
 * SGEMM_ERR_INVALID_VALUE: an unknown format, block or type; a dimension below
 * 0 or above 2^31 - 1025; a leading dimension below its row length; NULL or
 * misaligned (for its element type) pointers to operands that are touched;
 * workspace_bytes below 0; a grid beyond one launch.  SGEMM_ERR_ALIAS: C or
 * the workspace overlaps an operand.
 */
int sgemm_f8_gemm(int format_a, int format_b, int b_block, int c_type, int64_t M, int64_t N, int64_t K,
                  float alpha, const void *A, int64_t lda, const float *SA, int64_t ldsa, const void *B,
                  int64_t ldb, const float *SB, int64_t ldsb, float beta, void *C, int64_t ldc,
                  void *workspace, int64_t workspace_bytes, void *stream);

/* Host-only planning query: the kernel (0: nothing or no product to compute),
 * its grid of output tiles, the k-splits it makes with a sufficient workspace
 * and the bytes of their partial sums (0: unsplit), operands staying where they
 * are.  `aligned`: whether A, lda, B and ldb are all multiples of 16 and lda and
 * ldb (so K too) at most 2^22.  Output pointers may be NULL. */
int sgemm_f8_gemm_plan(int b_block, int64_t M, int64_t N, int64_t K, int aligned, int *kernel_id,
                       int64_t *tiles_m, int64_t *tiles_n, int64_t *splits, int64_t *workspace_bytes);

/* Host-only query: the workspace with which sgemm_f8_gemm is fastest (0: none). */
int sgemm_f8_gemm_workspace(int b_block, int64_t M, int64_t N, int64_t K, int aligned, int64_t *workspace_bytes);

/*
 * Quantise X (rows x cols of x_type) to 8 bits, in one pass over X, in either
 * or both of two ways; a NULL Q (or QT) leaves that one out (its S or ST is
 * then ignored):
 *   Q   rows x cols, blocks of X (scales S as above for rows x cols);
 *   QT  cols x rows, blocks of X^T (scales ST as above for cols x rows): the
 *       operand of a product that sums over X's rows.
 * With SGEMM_F8_TILE both hold the same values.  Rows or cols of 0: nothing is
 * touched.  Padding columns of Q and QT are not written.  More than 2^24 - 1 tiles
 * of 128 x 128 are beyond one launch: SGEMM_ERR_INVALID_VALUE.
 */
int sgemm_f8_quantize(int block, int format, int x_type, int64_t rows, int64_t cols, const void *X, int64_t ldx,
                      void *Q, int64_t ldq, float *S, int64_t lds, void *QT, int64_t ldqt, float *ST,
                      int64_t ldst, void *stream);

/*
 * Root-mean-square norm of each row, after an addition, with an 8-bit output:
 *     h = x + r      rstd = 1 / sqrt(mean(h^2) + eps)      y = h * rstd * w
 * in FP32 (h enters the norm unrounded).  X, R, H and Y are rows x cols of
 * `type`, W is cols values of w_type (`type` or FP32).  R may be NULL (h = x);
 * H (h rounded once), Y (y rounded once), Q with S (y in e4m3 with row blocks)
 * and rstd (rows FP32 values, for the backward pass) may each be NULL, and what
 * is NULL is not written.  H may be X or R itself (same pointer and leading
 * dimension); other overlaps of an output are SGEMM_ERR_ALIAS.
 * cols <= SGEMM_RMSNORM_MAX_COLS, eps >= 0 and finite.  Rows or cols of 0: nothing
 * is touched.  A row is held by 16 work-items up to 128 columns, 32 up to 256, 64 up
 * to 1024, 256 up to 4096, 512 up to 8192 and 1024 above; a call whose rows need more
 * than one launch's 2^32 - 1 of them is SGEMM_ERR_INVALID_VALUE.
 */
#define SGEMM_RMSNORM_MAX_COLS 32768
int sgemm_f8_rmsnorm(int type, int w_type, int64_t rows, int64_t cols, const void *X, int64_t ldx, const void *R,
                     int64_t ldr, const void *W, float eps, void *H, int64_t ldh, void *Y, int64_t ldy, void *Q,
                     int64_t ldq, float *S, int64_t lds, float *rstd, void *stream);

/*
 * Backward pass of the norm, from the gradient DY of y, the kept H and rstd:
 *     g = dy * w,  n = h * rstd,  dx = rstd * (g - n * mean(g * n)) + dh,
 *     dw = sum over rows of dy * n
 * in FP32.  dx is the gradient of x and of r alike; DH (NULL: none) is the
 * gradient that reaches h along the residual path.  DX is rows x cols of
 * `type`, rounded once, and may be DY, DH or H itself (same pointer and
 * leading dimension).  DW is cols FP32 values, summed in a fixed order, or
 * NULL; with DW the call needs the workspace that
 * sgemm_f8_rmsnorm_bwd_plan reports (16-byte aligned), else
 * SGEMM_ERR_INVALID_VALUE.  rows == 0: DW is set to 0.
 */
int sgemm_f8_rmsnorm_bwd(int type, int w_type, int64_t rows, int64_t cols, const void *DY, int64_t lddy,
                         const void *H, int64_t ldh, const void *W, const float *rstd, const void *DH, int64_t lddh,
                         void *DX, int64_t lddx, float *DW, void *workspace, int64_t workspace_bytes, void *stream);

/* Host-only query: the workspace bytes sgemm_f8_rmsnorm_bwd needs for DW. */
int sgemm_f8_rmsnorm_bwd_plan(int64_t rows, int64_t cols, int64_t *workspace_bytes);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_F8_H */
