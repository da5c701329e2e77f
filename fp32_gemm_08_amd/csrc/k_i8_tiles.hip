// Products of 8-bit integers on pipelined tiles.
#include "i8_pipe.h"

namespace sgemm {

// Blocks of 16 x 16; with 32 x 32 ones (half the operand reads of the matrix cores), measured
// before the scales were requested ahead, 128 x 128 tiles took 38.4 against 33.3 us at 4096 x
// 4096 x 1024, 64 x 64 ones 45.5 against 44.0, 256 x 256 ones 487 to 497 against 445 to 505 at
// 8192^3.
hipError_t launch_i8_tile(const I8GemmArgs &a, int kid, int splits, hipStream_t s)
{
    const unsigned grid = (unsigned)((int64_t)a.tiles_m * a.tiles_n * splits);
    switch (kid) {
    case KID_I8_S:
        i8_flat_kernel<F8Geo<64, 64, 2, 2>, 4><<<grid, 256, 0, s>>>(a);
        break;
    case KID_I8_N:
        i8_flat_kernel<F8Geo<128, 64, 4, 2>, 6><<<grid, 512, 0, s>>>(a);
        break;
    case KID_I8_M:
        i8_flat_kernel<F8Geo<128, 128, 2, 4>, 4><<<grid, 512, 0, s>>>(a);
        break;
    default:
        i8_pipe_kernel<F8Geo<256, 256, 2, 4>, 2><<<grid, 512, 0, s>>>(a);
        break;
    }
    return hipGetLastError();
}

}  // namespace sgemm
