// What the products of 8-bit integers share: matrix instructions and the way from the
// accumulators to C.
#pragma once
#include "f8_tile.h"
#include "i8_internal.h"

namespace sgemm {

// 16 x 16 products of 64 values of k.  The instruction takes rows of B as its first
// operand and rows of A as its second, so that lane l holds C[m = l % 16][n = 4*(l/16)
// .. +3]; lane l supplies 16 consecutive values of row l % 16 of each, which 16 is free
// as long as both agree.
__device__ __forceinline__ f8_i32x4 i8_mma(f8_i32x4 b, f8_i32x4 a, f8_i32x4 c)
{
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(b, a, c, 0, 0, 0);
}

// Columns n .. n+7 of row m of C <- alpha * (v * SA[m]) * SB[n] + beta * C.
template <typename T>
__device__ __forceinline__ void i8_put8(const I8GemmArgs &g, int m, int n, const int *v)
{
    T *row = static_cast<T *>(g.C) + (int64_t)m * g.ldc;
    const float sa = g.SA[m];
    float o[8], sb[8];
    row_load8<false>(g.SB, n, g.N, sb);
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
__device__ __forceinline__ void i8_put8(const I8GemmArgs &g, int m, int n, const int *v)
{
    if (g.c_type == SGEMM_TYPE_F32)
        i8_put8<float>(g, m, n, v);
    else if (g.c_type == SGEMM_TYPE_BF16)
        i8_put8<__bf16>(g, m, n, v);
    else
        i8_put8<_Float16>(g, m, n, v);
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

// A wavefront's 16 rows of WN columns of C, of which lane l holds row l % 16, columns
// 16j + 4*(l/16) .. +3: through `buf` (16 x (WN + 4) words of this wavefront's own), so
// that WN/8 lanes write one row together.  `part`: this split's partial sums.
template <int FN>
__device__ __forceinline__ void i8_store_rows(const I8GemmArgs &g, int *buf, int m, int n, const f8_i32x4 (&acc)[FN],
                                              int *part = nullptr)
{
    constexpr int PITCH = 16 * FN + 4, LANES = 2 * FN;  // lanes of a row
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int j = 0; j < FN; ++j)
        *reinterpret_cast<f8_i32x4 *>(buf + (lane & 15) * PITCH + 16 * j + 4 * (lane >> 4)) = acc[j];
#pragma unroll 1
    for (int e = lane; e < 16 * LANES; e += 64) {
        const int r = e / LANES, c = 8 * (e % LANES);
        if (m + r >= g.M || n + c >= g.N)
            continue;
        const int *v = buf + r * PITCH + c;
        if (part)
            i8_put_part(part + (int64_t)(m + r) * g.N, n + c, g.N, v);
        else
            i8_put8(g, m + r, n + c, v);
    }
}

}  // namespace sgemm
