// 8-bit block-scaled products on tiles of 256 x 256 and 128 x 128.
#include "f8_pipe.h"

namespace sgemm {

hipError_t launch_f8_large(const F8GemmArgs &a, int splits, int fa, int fb, bool row_b, hipStream_t s)
{
    return launch_pipe<F8Geo<256, 256, 2, 4>, 2, false>(a, splits, fa, fb, row_b, s);
}
hipError_t launch_f8_medium(const F8GemmArgs &a, int splits, int fa, int fb, bool row_b, hipStream_t s)
{
    return launch_pipe<F8Geo<128, 128, 2, 4>, 4, true>(a, splits, fa, fb, row_b, s);
}

}  // namespace sgemm
