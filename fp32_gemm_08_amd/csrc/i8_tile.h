// What the products of 8-bit integers share: matrix instructions and the way from the
// accumulators to C.
#pragma once
#include "f8_tile.h"
#include "i8_internal.h"

namespace sgemm {

// Blocks of MB x MB elements of C.  The instructions take rows of B as their first operand
// and rows of A as their second: lane l holds row m = l % MB of C, and of its columns groups
// of 4 consecutive ones, the first at 4 * (l / MB), each next one 256 / MB further.  Lane l
// supplies of row l % MB of each operand 16 consecutive values for a slice of 1024 / MB
// values of k, at chunk l / MB of the slice (which place is free as long as both agree).
template <int MB> struct I8Block;
template <> struct I8Block<16> {
    typedef f8_i32x4 Acc;
    static __device__ __forceinline__ Acc mma(f8_i32x4 b, f8_i32x4 a, Acc c)
    {
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(b, a, c, 0, 0, 0);
    }
};
template <int MB> struct I8Frag {
    static constexpr int NS = MB / 8;           // slices of a k-block of 128
    f8_i32x4 v[NS];
};

// Columns n .. n+7 of row m of C <- alpha * (v * sa) * sb + beta * C.
template <typename T>
__device__ __forceinline__ void i8_put8(const I8GemmArgs &g, int m, int n, const int *v, float sa, const float (&sb)[8])
{
    T *row = static_cast<T *>(g.C) + (int64_t)m * g.ldc;
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        o[i] = g.alpha * ((float)v[i] * sa * sb[i]);
    if (g.beta != 0.0f) {
        float old[8];
        row_load8<false>(row, n, g.N, old);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            o[i] = fmaf(g.beta, old[i], o[i]);
    }
    row_store8(row, n, g.N, o);
}
__device__ __forceinline__ void i8_put8(const I8GemmArgs &g, int m, int n, const int *v, float sa, const float (&sb)[8])
{
    if (g.c_type == SGEMM_TYPE_F32)
        i8_put8<float>(g, m, n, v, sa, sb);
    else if (g.c_type == SGEMM_TYPE_BF16)
        i8_put8<__bf16>(g, m, n, v, sa, sb);
    else
        i8_put8<_Float16>(g, m, n, v, sa, sb);
}

// Sums of 8 columns as they are: partial sums [M][N] of a split.
__device__ __forceinline__ void i8_put_part(int *row, int n, int cols, const int *v)
{
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        o[i] = __int_as_float(v[i]);
    row_store8(reinterpret_cast<float *>(row), n, cols, o);
}

// The scales of what a lane writes of its wavefront's FM x FN blocks from (m, n) on, requested
// before the products: at their end the latency of a first access would be the kernel's.
template <int MB, int FM, int FN> struct I8Scales {
    static constexpr int LANES = MB * FN / 8, TURNS = MB * LANES / 64;  // lanes of a row; rows of a lane in a block
    static_assert(64 % LANES == 0 && TURNS * 64 == MB * LANES, "whole turns of the lanes");
    float sa[FM][TURNS], sb[8];
    __device__ __forceinline__ I8Scales(const I8GemmArgs &g, int m, int n)
    {
        const int lane = threadIdx.x & 63;
        row_load8<false>(g.SB, n + 8 * (lane % LANES), g.N, sb);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int t = 0; t < TURNS; ++t)
                sa[i][t] = g.SA[min(m + MB * i + lane / LANES + t * (64 / LANES), g.M - 1)];
    }
};

// A wavefront's MB rows of FN blocks of C, block row i, through `buf` (MB x (MB FN + 4) words
// of this wavefront's own), so that the lanes of a row write it together.  `part`: this
// split's partial sums.
template <int MB, int FM, int FN>
__device__ __forceinline__ void i8_store_rows(const I8GemmArgs &g, int *buf, int m, int n, int i,
                                              const typename I8Block<MB>::Acc (&acc)[FN], const I8Scales<MB, FM, FN> &sc,
                                              int *part = nullptr)
{
    constexpr int PITCH = MB * FN + 4, LANES = MB * FN / 8;
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int x = 0; x < MB * MB / 256; ++x)
            *reinterpret_cast<f8_i32x4 *>(buf + lane % MB * PITCH + MB * j + 4 * (lane / MB) + 256 / MB * x) =
                f8_i32x4{acc[j][4 * x], acc[j][4 * x + 1], acc[j][4 * x + 2], acc[j][4 * x + 3]};
#pragma unroll
    for (int t = 0; t < I8Scales<MB, FM, FN>::TURNS; ++t) {
        const int r = lane / LANES + t * (64 / LANES), c = 8 * (lane % LANES);
        if (m + r >= g.M || n + c >= g.N)
            continue;
        const int *v = buf + r * PITCH + c;
        if (part)
            i8_put_part(part + (int64_t)(m + r) * g.N, n + c, g.N, v);
        else
            i8_put8(g, m + r, n + c, v, sc.sa[i][t], sc.sb);
    }
}

}  // namespace sgemm
