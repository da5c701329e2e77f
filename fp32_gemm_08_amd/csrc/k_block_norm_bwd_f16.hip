// Backward pass of the norms around a block for rows of _Float16.
#include "block_norm_bwd.h"

namespace sgemm {

template <> void launch_block_norm_bwd_from<_Float16, false>(const BlockNormBwdArgs &a, hipStream_t s)
{
    bwd_by_cols<_Float16>(a.cols, Bwd<false>{a, s});
}

}  // namespace sgemm
