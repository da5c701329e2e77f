// Backward pass of the norms around a block for rows of float, h and o kept in 8 bits.
#include "block_norm_bwd.h"

namespace sgemm {

template <> void launch_block_norm_bwd_from<float, true>(const BlockNormBwdArgs &a, hipStream_t s)
{
    bwd_by_cols<float>(a.cols, Bwd<true>{a, s});
}

}  // namespace sgemm
