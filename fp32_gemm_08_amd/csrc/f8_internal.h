// Internal declarations of the 8-bit block-scaled family: products,
// quantisation and the root-mean-square norm.
#pragma once

#include "sgemm_f8.h"
#include "sgemm_internal.h"

namespace sgemm {

constexpr int F8_BLOCK = 128;            // values per scale
constexpr float F8_FLOOR = 0x1p-90f;     // least block maximum: scales stay normal numbers
// Largest leading dimension of the pipelined kernels' operands, and of the tile scales
// they read across tiles: they hold a row's offset within a tile of 256 rows, the byte
// count of a tile's last rows and the offset of a tile's second row of scales in 32 bits.
constexpr int64_t F8_MAX_LD = int64_t{1} << 22;

enum F8KernelId : int {
    KID_F8_NONE = 0,
    KID_F8_SKINNY = 80,   // up to 64 rows of A: 16 to 64 columns of C per workgroup, k split over its wavefronts
    KID_F8_ANY = 81,      // rows at any alignment: 64 x 64 tile
    KID_F8_S = 82,        // 64 x 64 tile
    KID_F8_N = 83,        // 128 x 64 tile
    KID_F8_M = 84,        // 128 x 128 tile
    KID_F8_L = 85,        // 256 x 256 tile
};

struct F8GemmArgs {
    const uint8_t *A, *B;
    const float *SA, *SB;
    void *C;
    float *ws;                            // the workspace; in a tile's kernel: partial sums [split][M][N], NULL: unsplit
    int64_t lda, ldb, ldsa, ldsb, ldc;
    int M, N, K;
    int tiles_m, tiles_n;                 // output tiles
    int kb_split;                         // k-blocks per split
    float alpha, beta;
    int c_type;
};

struct F8GemmPlan {
    int kid = KID_F8_NONE;
    int64_t tiles_m = 0, tiles_n = 0, splits = 1;
    int64_t bytes = 0;      // of the workspace that it takes
    int64_t pack = 0;       // of them, its first, for operands laid out anew
};
// The plan for a workspace of `room` bytes.  aligned: the pipelined kernels can take the
// operands where they are; may_pack: operands may be laid out anew in the workspace.
F8GemmPlan f8_gemm_plan(bool row_b, int64_t M, int64_t N, int64_t K, bool aligned, int64_t room, bool may_pack);
// The plan of a call; rows_on_16: the rows of A and of B start on 16-byte boundaries.
F8GemmPlan f8_call_plan(const F8GemmArgs &a, bool rows_on_16, bool row_b, int64_t room);
hipError_t launch_f8_gemm(F8GemmArgs a, const F8GemmPlan &p, int format_a, int format_b, bool row_b, hipStream_t s);
// The tiles of aligned operands, a.kb_split k-blocks to each of `splits` (with
// several, their partial sums go to a.ws).
hipError_t launch_f8_small(const F8GemmArgs &a, int splits, int format_a, int format_b, bool row_b, hipStream_t s);
hipError_t launch_f8_narrow(const F8GemmArgs &a, int splits, int format_a, int format_b, bool row_b, hipStream_t s);
hipError_t launch_f8_medium(const F8GemmArgs &a, int splits, int format_a, int format_b, bool row_b, hipStream_t s);
hipError_t launch_f8_large(const F8GemmArgs &a, int splits, int format_a, int format_b, bool row_b, hipStream_t s);
// Few rows of A: columns per workgroup, and the launch.
int f8_skinny_cols(bool row_b, int64_t N);
hipError_t launch_f8_skinny(const F8GemmArgs &a, int format_a, int format_b, bool row_b, hipStream_t s);
// The rows of A, then those of B, laid out anew with whole lines a row, zeros past K.
constexpr int64_t F8_MAX_PACKED = int64_t{1} << 40;  // bytes of an operand that this is done for
inline int64_t f8_packed_ld(int64_t K) { return ceil_div(K, 128) * 128; }
hipError_t launch_f8_pack(const F8GemmArgs &a, uint8_t *to, hipStream_t s);
// C <- beta * C for a rows x cols C of any type.
hipError_t launch_f8_scale(void *C, int64_t ldc, int rows, int cols, int c_type, float beta, hipStream_t s);

struct F8QuantArgs {
    const void *X;
    uint8_t *Q, *QT;
    float *S, *ST;
    int64_t ldx, ldq, lds, ldqt, ldst;
    int rows, cols;
    int tiles_c;            // tiles along the columns
    const float *SX = nullptr;  // scales of X's row blocks, where it is in 8 bits itself
    int64_t ldsx = 0;
};
// The transposed output alone, from an X in 8 bits with row blocks.
hipError_t launch_f8_requantize(const F8QuantArgs &a, int format_x, int format, hipStream_t s);
hipError_t launch_f8_quantize(F8QuantArgs a, bool tile, int format, int x_type, hipStream_t s);

struct NormArgs {
    const void *X, *R, *W;
    void *H, *Y;
    uint8_t *Q;
    float *S, *rstd;
    int64_t ldx, ldr, ldh, ldy, ldq, lds;
    int rows, cols;
    float eps;
    int w_f32;              // W is FP32 (else of the rows' type)
};
int64_t rmsnorm_work_items(int64_t rows, int64_t cols);  // of its launch
hipError_t launch_rmsnorm(const NormArgs &a, int type, hipStream_t s);

struct NormBwdArgs {
    const void *DY, *H, *W, *DH;
    const float *rstd;
    void *DX;
    float *DW, *ws;         // ws: [groups][cols] partial sums of DW
    int64_t lddy, ldh, lddh, lddx;
    int rows, cols, groups;
    int w_f32;
};
int64_t rmsnorm_bwd_groups(int64_t rows, int64_t cols);
hipError_t launch_rmsnorm_bwd(const NormBwdArgs &a, int type, hipStream_t s);

}  // namespace sgemm
