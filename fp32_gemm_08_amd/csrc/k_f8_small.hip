// 8-bit block-scaled products on tiles of 128 x 64 and 64 x 64.
#include "f8_pipe.h"

namespace sgemm {

hipError_t launch_f8_narrow(const F8GemmArgs &a, int splits, int fa, int fb, bool row_b, hipStream_t s)
{
    return launch_pipe<F8Geo<128, 64, 4, 2>, 6, true>(a, splits, fa, fb, row_b, s);
}
hipError_t launch_f8_small(const F8GemmArgs &a, int splits, int fa, int fb, bool row_b, hipStream_t s)
{
    return launch_pipe<F8Geo<64, 64, 2, 4>, 8, true>(a, splits, fa, fb, row_b, s);
}

}  // namespace sgemm
