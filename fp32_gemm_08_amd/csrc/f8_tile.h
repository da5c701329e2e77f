// What the tiled 8-bit products share: a tile's geometry, the order of the tiles and
// the way from the accumulators to C.
#pragma once
#include "f8_mma.h"

namespace sgemm {

// Columns n .. n+7 of row m of C <- alpha * v + beta * C.
template <typename T>
__device__ __forceinline__ void put8(const F8GemmArgs &g, int m, int n, const float *v)
{
    T *row = static_cast<T *>(g.C) + (int64_t)m * g.ldc;
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        o[i] = g.alpha * v[i];
    if (g.beta != 0.0f) {
        float old[8];
        row_load8<false>(row, n, g.N, old);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            o[i] = fmaf(g.beta, old[i], o[i]);
    }
    row_store8(row, n, g.N, o);
}

// A wavefront's 16 rows of WN columns of C, of which lane l holds row l % 16,
// columns 16j + 4*(l/16) .. +3: through `buf` (16 x (WN + 4) floats of this
// wavefront's own), so that WN/8 lanes write one row together.
// `part`: this split's partial sums [M][N], which take the place of C.
template <int FN>
__device__ __forceinline__ void store_rows(const F8GemmArgs &g, float *buf, int m, int n, const f8_f32x4 (&acc)[FN],
                                           float *part = nullptr)
{
    constexpr int PITCH = 16 * FN + 4, LANES = 2 * FN;  // lanes of a row
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int j = 0; j < FN; ++j)
        *reinterpret_cast<f8_f32x4 *>(buf + (lane & 15) * PITCH + 16 * j + 4 * (lane >> 4)) = acc[j];
#pragma unroll 1
    for (int e = lane; e < 16 * LANES; e += 64) {
        const int r = e / LANES, c = 8 * (e % LANES);
        if (m + r >= g.M || n + c >= g.N)
            continue;
        const float *v = buf + r * PITCH + c;
        if (part) {
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                o[i] = v[i];
            row_store8(part + (int64_t)(m + r) * g.N, n + c, g.N, o);
        } else if (g.c_type == SGEMM_TYPE_F32)
            put8<float>(g, m + r, n + c, v);
        else if (g.c_type == SGEMM_TYPE_BF16)
            put8<__bf16>(g, m + r, n + c, v);
        else
            put8<_Float16>(g, m + r, n + c, v);
    }
}

// BM rows of A and BN rows of B per workgroup, WGM x WGN wavefronts.  A stage
// is one k-block of 128 bytes of every row.  In LDS a row's eight 16-byte chunks
// are permuted by (r >> 1) & 7.  A 16-byte read takes its lanes 16 at a time
// over 64 banks, in the groups 0-3, 12-15, 20-27 / 4-11, 16-19, 28-31 (and the
// same of the upper half): each holds 16 rows, some at chunk q and some at
// q ^ 1, which this permutation spreads over all banks.  (With the lanes' natural
// order in mind, (r ^ (r >> 3)) & 7, half of the LDS cycles were bank conflicts.)
template <int BM_, int BN_, int WGM_, int WGN_>
struct F8Geo {
    static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_;
    static constexpr int NW = WGM * WGN, NT = 64 * NW;
    static constexpr int WM = BM / WGM, WN = BN / WGN, FM = WM / 16, FN = WN / 16;
    static constexpr int ROWS = BM + BN;
    static constexpr int LOADS = ROWS / 8 / NW;     // 1 KB blocks of 8 rows per wavefront per stage
    static constexpr int SC = ROWS * 4;             // scales of a stage, bytes
    static constexpr int STAGE = ROWS * 128 + SC;
    static_assert(WM % 16 == 0 && WN % 16 == 0 && (128 % WN == 0 || WN % 128 == 0), "whole 16 x 16 blocks");
    static constexpr int OUT = 16 * (WN + 4);       // floats that a wavefront's 16 rows of C pass through
    static_assert(NW * OUT * 4 <= STAGE, "they fit into a stage");
    static_assert(LOADS * 8 * NW == ROWS, "every wavefront loads whole blocks");
    static_assert(2 * STAGE <= 160 * 1024, "two stages in the LDS");
};

template <typename T> __device__ __forceinline__ T f8_pick(bool first, T a, T b) { return first ? a : b; }

__device__ __forceinline__ int f8_swz(int r) { return (r >> 1) & 7; }

// Workgroup -> output tile: one contiguous run of tiles per XCD, walked 8
// tile-rows at a time.
__device__ __forceinline__ void f8_map_tile(int bid, int nbm, int nbn, int &tm, int &tn)
{
    const int nb = nbm * nbn;
    const int id = (nb % 8 == 0) ? (bid % 8) * (nb / 8) + bid / 8 : bid;
    const int group = 8 * nbn;
    const int g = id / group, first_m = g * 8;
    const int gm = min(nbm - first_m, 8);
    tm = first_m + (id % group) % gm;
    tn = (id % group) / gm;
}

}  // namespace sgemm
