// Quantisation to 8 bits with one FP32 scale per block of 128 values, of a
// matrix and of its transpose in one pass over it.
//
//   a = max(max|x| over the block, 2^-90),  q = rne8(x * (L / a)),  s = a / L
//
// A workgroup of 256 holds a 128 x 128 tile of X in registers, each work-item
// an 8 x 8 piece of it (8 consecutive rows, 8 consecutive columns).  The 16
// lanes of a data-parallel row hold one row of the tile, so a row block's
// maximum is four lane permutations; a column block's maximum crosses the
// wavefronts through 2 KB of LDS.  One work-item divides for each row and each
// column, and the factors go round through the LDS.  The transposed output goes
// through an LDS tile of bytes: a work-item's 8 rows of one column are 8
// consecutive bytes of it.  X is read once, each output is written once.
#include "f8_types.h"

namespace sgemm {
namespace {

constexpr int QT = 128;          // tile side
constexpr int QT_PITCH = QT + 8; // bytes per column in the transposed tile

template <typename T, int FMT, bool TILE>
__global__ __launch_bounds__(256) void f8_quantize_kernel(F8QuantArgs g)
{
    __shared__ __attribute__((aligned(16))) uint8_t tile[QT * QT_PITCH];
    __shared__ uint32_t colmax[4][QT];
    __shared__ uint32_t wavemax[4];
    __shared__ __attribute__((aligned(16))) float factor[2][QT];  // of the rows, of the columns
    poison_lds(tile, (int)sizeof(tile));

    const int tr = blockIdx.x / g.tiles_c, tc = blockIdx.x % g.tiles_c;
    const int r0 = tr * QT, c0 = tc * QT;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int pr = 8 * (threadIdx.x / 16), pc = 8 * (threadIdx.x % 16);  // this work-item's piece
    const int c = c0 + pc;

    float v[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = r0 + pr + i;
        if (r < g.rows && c < g.cols) {
            row_load8<true>(static_cast<const T *>(g.X) + (int64_t)r * g.ldx, c, g.cols, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[i][j] = 0.0f;
        }
    }

    float inv_r[8], inv_c[8];  // factors of this piece's rows and columns
    if constexpr (TILE) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            m = max(m, abs_max8(v[i]));
        m = max16(m);
        m = max(m, (uint32_t)__shfl_xor((int)m, 16));
        m = max(m, (uint32_t)__shfl_xor((int)m, 32));
        if (lane == 0)
            wavemax[w] = m;
        __syncthreads();
        m = max(max(wavemax[0], wavemax[1]), max(wavemax[2], wavemax[3]));
        float inv, scale;
        block_scale<FMT>(m, inv, scale);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            inv_r[i] = inv_c[i] = inv;
        if (threadIdx.x == 0) {
            if (g.Q)
                g.S[(int64_t)tr * g.lds + tc] = scale;
            if (g.QT)
                g.ST[(int64_t)tc * g.ldst + tr] = scale;
        }
    } else {
        if (g.Q) {
            // the lane i of a row of 16 takes the row pr + i
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t mi = max16(abs_max8(v[i]));
                m = threadIdx.x % 16 == i ? mi : m;
            }
            const int i = threadIdx.x % 16;
            if (i < 8) {
                float inv, scale;
                block_scale<FMT>(m, inv, scale);
                factor[0][pr + i] = inv;
                if (r0 + pr + i < g.rows)
                    g.S[(int64_t)tc * g.lds + r0 + pr + i] = scale;
            }
        }
        if (g.QT) {
            uint32_t m[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                m[j] = abs_bits(v[0][j]);
#pragma unroll
                for (int i = 1; i < 8; ++i)
                    m[j] = max(m[j], abs_bits(v[i][j]));
                m[j] = max(m[j], (uint32_t)__shfl_xor((int)m[j], 16));
                m[j] = max(m[j], (uint32_t)__shfl_xor((int)m[j], 32));
            }
            if (lane < 16) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    colmax[w][pc + j] = m[j];
            }
            __syncthreads();
            if (threadIdx.x < QT) {
                const int t = threadIdx.x;
                float inv, scale;
                block_scale<FMT>(max(max(colmax[0][t], colmax[1][t]), max(colmax[2][t], colmax[3][t])), inv, scale);
                factor[1][t] = inv;
                if (c0 + t < g.cols)
                    g.ST[(int64_t)tr * g.ldst + c0 + t] = scale;
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            inv_r[i] = factor[0][pr + i];
            inv_c[i] = factor[1][pc + i];
        }
    }

    if (g.Q) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = r0 + pr + i;
            const float f = inv_r[i];
            const uint32_t lo = f8_pack4<FMT>(v[i][0] * f, v[i][1] * f, v[i][2] * f, v[i][3] * f);
            const uint32_t hi = f8_pack4<FMT>(v[i][4] * f, v[i][5] * f, v[i][6] * f, v[i][7] * f);
            if (r < g.rows && c < g.cols)
                row_store8b(g.Q + (int64_t)r * g.ldq, c, g.cols, lo, hi);
        }
    }
    if (g.QT) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float f = inv_c[j];
            const uint32_t lo = f8_pack4<FMT>(v[0][j] * f, v[1][j] * f, v[2][j] * f, v[3][j] * f);
            const uint32_t hi = f8_pack4<FMT>(v[4][j] * f, v[5][j] * f, v[6][j] * f, v[7][j] * f);
            *reinterpret_cast<f8_u32x2 *>(tile + (pc + j) * QT_PITCH + pr) = f8_u32x2{lo, hi};
        }
        __syncthreads();
        // 16 lanes write one column's 128 bytes
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int col = 16 * i + threadIdx.x / 16, at = 8 * (threadIdx.x % 16);
            if (c0 + col < g.cols && r0 + at < g.rows) {
                const f8_u32x2 x = *reinterpret_cast<const f8_u32x2 *>(tile + col * QT_PITCH + at);
                row_store8b(g.QT + (int64_t)(c0 + col) * g.ldqt, r0 + at, g.rows, x[0], x[1]);
            }
        }
    }
}

template <typename T>
void launch_t(const F8QuantArgs &a, unsigned grid, bool tile, int format, hipStream_t s)
{
    if (format == SGEMM_F8_E4M3) {
        if (tile)
            f8_quantize_kernel<T, 0, true><<<grid, 256, 0, s>>>(a);
        else
            f8_quantize_kernel<T, 0, false><<<grid, 256, 0, s>>>(a);
    } else {
        if (tile)
            f8_quantize_kernel<T, 1, true><<<grid, 256, 0, s>>>(a);
        else
            f8_quantize_kernel<T, 1, false><<<grid, 256, 0, s>>>(a);
    }
}

}  // namespace

hipError_t launch_f8_quantize(F8QuantArgs a, bool tile, int format, int x_type, hipStream_t s)
{
    const int64_t tr = ((int64_t)a.rows + QT - 1) / QT, tc = ((int64_t)a.cols + QT - 1) / QT;
    a.tiles_c = (int)tc;
    const unsigned grid = (unsigned)(tr * tc);
    if (x_type == SGEMM_TYPE_F32)
        launch_t<float>(a, grid, tile, format, s);
    else if (x_type == SGEMM_TYPE_FP16)
        launch_t<_Float16>(a, grid, tile, format, s);
    else
        launch_t<__bf16>(a, grid, tile, format, s);
    return hipGetLastError();
}

}  // namespace sgemm
