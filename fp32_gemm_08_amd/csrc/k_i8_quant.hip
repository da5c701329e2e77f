// Quantisation of rows to 8-bit integers:
//
//     a = max(max|x| over the row, 2^-90),  s = a / 127,  q = 127 x / a, rounded
//
// L work-items hold a row (norm_rows.h), which is read once.  127 x / a is computed as
// x * fl(127 / a): two roundings, off by at most 127 * 2^-23 = 1.6e-5.  Only where that
// lies within 2e-5 of the middle between two integers can it decide wrongly; there
// 254 x and (2 i + 1) a, which are exact in 64 bits (31 and 32 bits), are compared.
//
// Bound by memory: 16384 x 4096 bf16 33.9 us, 5.9 TB/s; packed rows of 4095 40.8, whose
// stores of 8 bytes straddle lines.  One row of 4096 3.7 us, the launch.
#include "i8_internal.h"
#include "norm_rows.h"

namespace sgemm {
namespace {

__device__ __forceinline__ int i8_nearest(float x, float a, float inv)
{
    const float t = x * inv, r = rintf(t);
    if (fabsf(t - r) < 0.49998f)
        return (int)r;
    if (!(t == t))
        return 0;
    const float low = floorf(t);                              // the middle is low + 1/2
    const double d = 254.0 * (double)x - (2.0 * (double)low + 1.0) * (double)a;
    const int i = (int)low;
    return d > 0.0 ? i + 1 : d < 0.0 ? i : i + (i & 1);
}

template <typename T, int NT, int L, int V>
__global__ __launch_bounds__(NT) void i8_quantize_kernel(I8QuantArgs g)
{
    __shared__ uint32_t top[NT / 64];
    const int lane = threadIdx.x % L;                                    // of the row's
    const int64_t row = (int64_t)blockIdx.x * (NT / L) + threadIdx.x / L;
    if (row >= g.rows)
        return;  // whole rows of lanes, and only where no row needs the workgroup
    const T *x = static_cast<const T *>(g.X) + row * g.ldx;
    float v[V][8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        row_load8<true>(x, 8 * (lane + L * i), g.cols, v[i]);
        m = max(m, abs_max8(v[i]));
    }
    // rows beyond what the work-items hold are read twice
    for (int64_t c = 8 * (lane + L * V); c < g.cols; c += 8 * L) {
        float u[8];
        row_load8<false>(x, (int)c, g.cols, u);
        m = max(m, abs_max8(u));
    }
    m = row_max<NT, L>(m, top);
    float inv, scale;
    i8_scale(m, inv, scale);
    const float a = __uint_as_float(max(m, __float_as_uint(F8_FLOOR)));
    if (lane == 0)
        g.S[row] = scale;
    auto put = [&](int c, const float (&u)[8]) {
        int q[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            q[j] = i8_nearest(u[j], a, inv);
        row_store8b(g.Q + row * g.ldq, c, g.cols, i8_pack4(q[0], q[1], q[2], q[3]), i8_pack4(q[4], q[5], q[6], q[7]));
    };
#pragma unroll
    for (int i = 0; i < V; ++i)
        put(8 * (lane + L * i), v[i]);
    for (int64_t c = 8 * (lane + L * V); c < g.cols; c += 8 * L) {
        float u[8];
        row_load8<false>(x, (int)c, g.cols, u);
        put((int)c, u);
    }
}

struct Launch {
    const I8QuantArgs &a;
    hipStream_t s;
    template <typename T, int NT, int L, int V> void run()
    {
        i8_quantize_kernel<T, NT, L, V><<<(unsigned)ceil_div(a.rows, NT / L), NT, 0, s>>>(a);
    }
};

}  // namespace

int64_t i8_quantize_work_items(int64_t rows, int64_t cols) { return rmsnorm_work_items(rows, cols); }

hipError_t launch_i8_quantize(const I8QuantArgs &a, int x_type, hipStream_t s)
{
    by_type(x_type, a.cols, Launch{a, s});
    return hipGetLastError();
}

}  // namespace sgemm
