// Internal declarations of the products of 8-bit integers and their quantisation.
#pragma once

#include "f8_internal.h"
#include "sgemm_i8.h"

namespace sgemm {

enum I8KernelId : int {
    KID_I8_NONE = 0,
    KID_I8_SKINNY = 90,   // up to 16 rows of A (32 where B is small): 16 or 32 columns of C per workgroup, k split over its wavefronts
    KID_I8_ANY = 91,      // rows at any alignment: 64 x 64 tile, 4 or 16 wavefronts
    KID_I8_S = 92,        // 64 x 64 tile, two workgroups to a CU
    KID_I8_N = 93,        // 128 x 64 tile
    KID_I8_M = 94,        // 128 x 128 tile
    KID_I8_L = 95,        // 256 x 256 tile
};

struct I8GemmArgs {
    const uint8_t *A, *B;
    const float *SA, *SB;
    void *C;
    int *ws;                              // the workspace; in a tile's kernel: partial sums [split][M][N], NULL: unsplit
    int64_t lda, ldb, ldc;
    int M, N, K;
    int tiles_m, tiles_n;                 // output tiles
    int kb_split;                         // k-blocks of 128 per split
    float alpha, beta;
    int c_type;
};

struct I8GemmPlan {
    int kid = KID_I8_NONE;
    int64_t tiles_m = 0, tiles_n = 0, splits = 1;
    int64_t bytes = 0;      // of the workspace that it takes
    int64_t pack = 0;       // of them, its first, for operands laid out anew
    int threads = 256;      // work-items of a workgroup
};
// The plan for a workspace of `room` bytes.  aligned: the pipelined kernels can take the
// operands where they are; may_pack: operands may be laid out anew in the workspace.
I8GemmPlan i8_gemm_plan(int64_t M, int64_t N, int64_t K, bool aligned, int64_t room, bool may_pack);
hipError_t launch_i8_gemm(I8GemmArgs a, const I8GemmPlan &p, hipStream_t s);
// Up to 32 rows of A, with 16 columns a workgroup, or 32 columns for up to 16 rows.
hipError_t launch_i8_skinny(const I8GemmArgs &a, int cols, int splits, hipStream_t s);
// The pipelined kernel of a tile (KID_I8_S to KID_I8_L).
hipError_t launch_i8_tile(const I8GemmArgs &a, int kid, int splits, hipStream_t s);

struct I8QuantArgs {
    const void *X;
    uint8_t *Q;
    float *S;
    int64_t ldx, ldq;
    int rows, cols;
};
int64_t i8_quantize_work_items(int64_t rows, int64_t cols);  // of its launch
hipError_t launch_i8_quantize(const I8QuantArgs &a, int x_type, hipStream_t s);

}  // namespace sgemm
