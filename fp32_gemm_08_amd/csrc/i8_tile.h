// What the products of 8-bit integers share: matrix instructions and the way from the
// accumulators to C.
#pragma once
#include "f8_tile.h"
#include "i8_internal.h"

namespace sgemm {

// Blocks of 16 x 16 elements of C.  The instruction takes rows of B as its first operand and
// rows of A as its second: lane l holds row m = l % 16 of C, columns 4 * (l / 16) .. +3.  Lane l
// supplies of row l % 16 of each operand 16 consecutive values for a slice of 64 values of k,
// at chunk l / 16 of the slice (which place is free as long as both agree).
__device__ __forceinline__ f8_i32x4 i8_mma(f8_i32x4 b, f8_i32x4 a, f8_i32x4 c)
{
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(b, a, c, 0, 0, 0);
}
struct I8Frag {
    f8_i32x4 v[2];                              // slices of a k-block of 128
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
template <int FM, int FN> struct I8Scales {
    static constexpr int LANES = 2 * FN, TURNS = FN / 2;        // lanes of a row; rows of a lane in a block
    static_assert(64 % LANES == 0 && TURNS * 64 == 16 * LANES, "whole turns of the lanes");
    float sa[FM][TURNS], sb[8];
    __device__ __forceinline__ I8Scales(const I8GemmArgs &g, int m, int n)
    {
        const int lane = threadIdx.x & 63;
        row_load8<false>(g.SB, n + 8 * (lane % LANES), g.N, sb);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int t = 0; t < TURNS; ++t)
                sa[i][t] = g.SA[min(m + 16 * i + lane / LANES + t * (64 / LANES), g.M - 1)];
    }
};

// A wavefront's 16 rows of FN blocks of C, block row i, through `buf` (16 x (16 FN + 4) words
// of this wavefront's own), so that the lanes of a row write it together.  `part`: this
// split's partial sums.
template <int FM, int FN>
__device__ __forceinline__ void i8_store_rows(const I8GemmArgs &g, int *buf, int m, int n, int i, const f8_i32x4 (&acc)[FN],
                                              const I8Scales<FM, FN> &sc, int *part = nullptr)
{
    constexpr int PITCH = 16 * FN + 4, LANES = 2 * FN;
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int j = 0; j < FN; ++j)
        *reinterpret_cast<f8_i32x4 *>(buf + lane % 16 * PITCH + 16 * j + 4 * (lane / 16)) = acc[j];
#pragma unroll
    for (int t = 0; t < I8Scales<FM, FN>::TURNS; ++t) {
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
