// Backward pass of the norms around a block for rows of __bf16.
#include "block_norm_bwd.h"

namespace sgemm {

template <> void launch_block_norm_bwd_rows<__bf16>(const BlockNormBwdArgs &a, bool kept, bool several, hipStream_t s)
{
    bwd_by_cols<__bf16>(a.cols, Bwd{a, kept, several, s});
}

}  // namespace sgemm
