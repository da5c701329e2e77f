/*
 * sgemm_norm — the root-mean-square norms after and before a block of layers,
 * fused with the block's gate and the residual's scale, and their backward pass,
 * for AMD Instinct MI355X (gfx950).
 *
 * The same library, statuses and conventions as sgemm_f32.h and sgemm_f8.h:
 * row-major DEVICE pointers owned by the caller, leading dimensions in elements,
 * arguments checked on the host before any HIP call, work enqueued on `stream`
 * with no synchronisation, no allocation and no device-side state kept between
 * calls.
 */
#ifndef SGEMM_NORM_H
#define SGEMM_NORM_H

#include "sgemm_f8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* 8-bit integers with one FP32 scale per row: a = max(max|y|, 2^-90), s = a / 127,
 * q = y * (127 / a) to the nearest integer, ties to even (sgemm_i8.h).  A row
 * with a NaN or an infinity gets a NaN or infinite scale and stands for NaN. */
#define SGEMM_Q_I8 3

/*
 * Between two blocks, in FP32, for each row i (o: the block's output, x: the
 * residual stream):
 *     rstd_post = 1 / sqrt(mean(o^2) + eps)       z = o * rstd_post * w_post
 *     h = alpha * x + gate * z
 *     rstd = 1 / sqrt(mean(h^2) + eps)            y = h * rstd * w
 * X, O, H and Y are rows x cols of `type`; W, W_post (cols values) and GATE are
 * of w_type (`type` or FP32).  GATE has ceil(rows/gate_rows) rows of cols values,
 * row i of x takes row i / gate_rows of it (gate_rows = rows: a gate per
 * channel; a sequence's length: one for each sequence; 1: one for each token); it is at
 * least 1, or 0 where rows is.
 *   O NULL:      no block: h = alpha * x (W_post, GATE, O8 and rstd_post are ignored)
 *   W_post NULL: no norm after the block: z = o (rstd_post is then not written)
 *   GATE NULL:   gate 1 (gate_rows and ldg are ignored)
 * Outputs, each NULL or written: H (h, rounded once; it enters the second norm
 * unrounded), Y (y, rounded once), Q with S (y in 8 bits), H8 with SH and O8 with
 * SO (h before it is rounded and o, in e4m3 with row blocks: what the backward
 * pass can take in their place), rstd and rstd_post (rows FP32 values).  q_format:
 *   SGEMM_F8_E4M3: Q in e4m3 with row blocks, S (ceil(cols/128) x rows, leading
 *                  dimension lds >= rows)
 *   SGEMM_Q_I8:    Q in 8-bit integers, S rows consecutive values (lds is ignored)
 * W may be NULL if neither Y nor Q is given.  H may be X or O itself (same pointer
 * and leading dimension); other overlaps of an output are SGEMM_ERR_ALIAS.
 * alpha is finite, eps >= 0 and finite, cols <= SGEMM_RMSNORM_MAX_COLS, and the rows'
 * work-items (as sgemm_f8_rmsnorm counts them) within one launch, else
 * SGEMM_ERR_INVALID_VALUE.  Rows or cols of 0: nothing is touched.
 */
int sgemm_block_norm(int type, int w_type, int64_t rows, int64_t cols, const void *X, int64_t ldx, const void *O,
                     int64_t ldo, const void *W, const void *W_post, const void *GATE, int64_t ldg, int64_t gate_rows,
                     float alpha, float eps, void *H, int64_t ldh, void *Y, int64_t ldy, int q_format, void *Q,
                     int64_t ldq, float *S, int64_t lds, void *H8, int64_t ldh8, float *SH, int64_t ldsh, void *O8,
                     int64_t ldo8, float *SO, int64_t ldso, float *rstd, float *rstd_post, void *stream);

/*
 * Its backward pass, in FP32, from DY (the gradient of y), DH (what reaches h along
 * the residual path) and what the forward pass kept:
 *     n = h * rstd,  g = dy * w,  d = rstd * (g - n * mean(g * n)) + dh
 *     dx = alpha * d            dw = sum over rows of dy * n
 *     dgate = sum over the rows of a gate of d * z
 *     m = o * rstd_post,  p = gate * d * w_post      dw_post = sum over rows of gate * d * m
 *     do = rstd_post * (p - m * mean(p * m))
 * and without W_post z = o, do = gate * d.
 *   DY NULL:     nothing reaches y: d = dh (H, W and rstd are not read; DW, if
 *                given, is set to 0); DH NULL: nothing along the residual path.  One
 *                of the two is needed.
 *   kept: 0: H and O are rows x cols of `type`; 1: both in e4m3 with row blocks and
 *                scales SH, SO (leading dimensions ldsh, ldso >= rows).
 *   O:           read only for DGATE or with W_post, and may be NULL otherwise.  GATE,
 *                W_post and rstd_post are read only if DO, DGATE or DW_post is given.
 * Outputs, each NULL or written: DX and DO (rows x cols of `type`, rounded once),
 * DW, DW_post (cols FP32 values), DGATE (FP32, a row of cols values for each of
 * GATE's, leading dimension lddg); the last three are summed in a fixed order, in
 * the workspace that sgemm_block_norm_bwd_plan reports (16-byte aligned; none is
 * needed if none of them is given; calls that share one must not run at once).  DW_post needs W_post, DGATE needs GATE.
 * DX may be DY, DH or (kept = 0) H itself, and DO may be DY, DH or (kept = 0) O
 * itself, with the same pointer and leading dimension; other overlaps are
 * SGEMM_ERR_ALIAS.  rows == 0: DW and DW_post are set to 0.
 */
int sgemm_block_norm_bwd(int type, int w_type, int64_t rows, int64_t cols, const void *DY, int64_t lddy,
                         const void *DH, int64_t lddh, int kept, const void *H, int64_t ldh, const float *SH,
                         int64_t ldsh, const void *O, int64_t ldo, const float *SO, int64_t ldso, const void *W,
                         const void *W_post, const float *rstd, const float *rstd_post, const void *GATE, int64_t ldg,
                         int64_t gate_rows, float alpha, void *DX, int64_t lddx, void *DO, int64_t lddo, float *DW,
                         float *DW_post, float *DGATE, int64_t lddg, void *workspace, int64_t workspace_bytes,
                         void *stream);

/* Host-only query: the workspace bytes that serve that call, whichever of its outputs
 * are given.  gate_rows: as there; rows (or 0) without a gate. */
int sgemm_block_norm_bwd_plan(int64_t rows, int64_t cols, int64_t gate_rows, int64_t *workspace_bytes);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_NORM_H */
