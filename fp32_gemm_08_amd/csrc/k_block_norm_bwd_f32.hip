// Backward pass of the norms around a block for rows of float.
#include "block_norm_bwd.h"

namespace sgemm {

template <> void launch_block_norm_bwd_rows<float>(const BlockNormBwdArgs &a, bool kept, bool several, hipStream_t s)
{
    bwd_by_cols<float>(a.cols, Bwd{a, kept, several, s});
}

}  // namespace sgemm
