// Backward pass of the norms around a block for rows of __bf16, h and o kept in 8 bits.
#include "block_norm_bwd.h"

namespace sgemm {

template <> void launch_block_norm_bwd_from<__bf16, true>(const BlockNormBwdArgs &a, hipStream_t s)
{
    bwd_by_cols<__bf16>(a.cols, Bwd<true>{a, s});
}

}  // namespace sgemm
