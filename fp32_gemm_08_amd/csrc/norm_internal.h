// Internal declarations of the norms around a block.
#pragma once

#include "f8_internal.h"
#include "sgemm_norm.h"

namespace sgemm {

struct BlockNormArgs {
    const void *X, *O, *W, *WP, *G;
    void *H, *Y;
    uint8_t *Q, *H8, *O8;
    float *S, *SH, *SO, *rstd, *rstd_post;
    int64_t ldx, ldo, ldg, ldh, ldy, ldq, lds, ldh8, ldsh, ldo8, ldso;
    int rows, cols, gate_rows;
    float alpha, eps;
    int w_f32;              // W, WP and G are FP32 (else of the rows' type)
    int q_i8;               // Q holds integers with a scale per row
};
hipError_t launch_block_norm(const BlockNormArgs &a, int type, hipStream_t s);

struct BlockNormBwdArgs {
    const void *DY, *DH, *H, *O, *W, *WP, *G;
    const float *SH, *SO, *rstd, *rstd_post;
    void *DX, *DO;
    float *DW, *DWP, *DG;
    float *ws;              // partial sums, see BlockNormSums
    int64_t lddy, lddh, ldh, ldsh, ldo, ldso, ldg, lddx, lddo, lddg;
    int rows, cols, gate_rows;
    float alpha;
    int w_f32;
    int groups;             // workgroups
    int team;               // of them, those of a gate; 0: several gates a walker
    int chunk;              // then: consecutive rows of a walker
};

// Who sums what of the backward pass.  A walker is the work-items that hold a row (a
// workgroup, or 16 to 64 lanes of one).  Few gates: each has a team of workgroups, which
// leave their sums of dy n, of d m and (more gates than one) of gate d m.  Many: a walker
// takes `chunk` consecutive rows, its workgroup leaves the sums of dy n and of gate d m, and
// walkers leave their sums of d m for those gates of which they do not have all rows: for
// the first that they meet at 2 * walker, for another one (the last) at 2 * walker + 1.
struct BlockNormSums {
    int64_t groups = 0, team = 0, walkers = 0, chunk = 1;
    int64_t parts = 0;      // arrays of cols floats in the workspace
};
BlockNormSums block_norm_sums(int64_t rows, int64_t cols, int64_t gate_rows);
// Gates that the second kernel looks at, of those whose sums are wanted: with teams all; else
// none where every gate lies in one walker's rows, all of those longer than a walker's rows, or
// for each walker the one that its last row belongs to.
inline int64_t block_norm_gates_to_join(const BlockNormSums &n, int64_t rows, int64_t gate_rows)
{
    if (!n.team && n.chunk % gate_rows == 0)
        return 0;
    return n.team || gate_rows > n.chunk ? ceil_div(rows, gate_rows) : n.walkers;
}
hipError_t launch_block_norm_bwd(BlockNormBwdArgs a, int type, bool kept, hipStream_t s);

}  // namespace sgemm
