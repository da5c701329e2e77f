// Backward pass of the norms around a block for rows of float.
#include "block_norm_bwd.h"

namespace sgemm {

template <> void launch_block_norm_bwd_from<float, false>(const BlockNormBwdArgs &a, hipStream_t s)
{
    bwd_by_cols<float>(a.cols, Bwd<false>{a, s});
}

}  // namespace sgemm
