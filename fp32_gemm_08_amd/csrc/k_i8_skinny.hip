// Products of 8-bit integers with few rows of A (single tokens of a batch): the bytes of B
// bound them.
#include "i8_tile.h"

namespace sgemm {
namespace {

// Columns n .. n+3 of row m of C.
template <typename T>
__device__ __forceinline__ void i8_put4(const I8GemmArgs &g, int m, int n, f8_i32x4 v, float sa, f8_f32x4 sb)
{
    typedef T V4 __attribute__((ext_vector_type(4)));
    typedef V4 V4any __attribute__((aligned(1)));
    T *p = static_cast<T *>(g.C) + (int64_t)m * g.ldc + n;
    if (n + 4 <= g.N) {
        f8_f32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = g.alpha * ((float)v[i] * sa * sb[i]);
        if (g.beta != 0.0f) {
            const V4 old = *reinterpret_cast<const V4any *>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[i] = fmaf(g.beta, (float)old[i], o[i]);
        }
        V4 u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            u[i] = (T)o[i];
        *reinterpret_cast<V4any *>(p) = u;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i < g.N) {
                const float o = g.alpha * ((float)v[i] * sa * sb[i]);
                p[i] = (T)(g.beta != 0.0f ? fmaf(g.beta, (float)p[i], o) : o);
            }
    }
}

// Up to 16 FM rows of A: a workgroup has 16 FN columns of C, and its 8 wavefronts take the
// k-blocks of its split in turn, each lane loading its operands straight into registers,
// DEPTH k-blocks ahead.  The wavefronts' sums are added through the LDS.
//
// 1 x 4096 x 4096 5.3 us for 3.3 of B's bytes: a trip to memory, the join and the launch;
// 16 x 16384 x 4096 15.2, 4.5 TB/s.
template <int FM, int FN, int DEPTH>
__global__ __launch_bounds__(512) void i8_skinny_kernel(I8GemmArgs g)
{
    constexpr int NW = 8, NF = FM + FN;
    __shared__ f8_i32x4 part[NW][FM * FN][64];
    poison_lds(part, (int)sizeof(part));
    const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int split = blockIdx.x / g.tiles_n, n0 = blockIdx.x % g.tiles_n * 16 * FN;
    const int first = split * g.kb_split, nk = min((g.K + 127) / 128 - first, g.kb_split);

    // rows past the matrix repeat its last one (their results are not stored)
    const uint8_t *row[NF];
#pragma unroll
    for (int i = 0; i < FM; ++i)
        row[i] = g.A + (int64_t)min(16 * i + l16, g.M - 1) * g.lda + 16 * q;
#pragma unroll
    for (int j = 0; j < FN; ++j)
        row[FM + j] = g.B + (int64_t)min(n0 + 16 * j + l16, g.N - 1) * g.ldb + 16 * q;

    struct Block {
        f8_i32x4 lo[NF], hi[NF];
    } blk[DEPTH];
    auto load = [&](Block &b, int kb) {
        const int at = (first + kb) * 128;
        if (at + 128 <= g.K) {
#pragma unroll
            for (int i = 0; i < NF; ++i) {
                b.lo[i] = *reinterpret_cast<const f8_i32x4_any *>(row[i] + at);
                b.hi[i] = *reinterpret_cast<const f8_i32x4_any *>(row[i] + at + 64);
            }
        } else {
            const int valid = g.K - at - 16 * q;
#pragma unroll
            for (int i = 0; i < NF; ++i) {
                b.lo[i] = load16_any(row[i] + at, min(valid, 16));
                b.hi[i] = load16_any(row[i] + at + 64, min(valid - 64, 16));
            }
        }
    };

    // the scales of what this lane writes, requested before the products (see I8Scales)
    static_assert(FM * FN <= NW, "a block per wavefront at the end");
    const int m = 16 * (w / FN) + l16, n = n0 + 16 * (w % FN) + 4 * q;
    const float sa = g.SA[min(m, g.M - 1)];
    f8_f32x4 sb;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        sb[i] = g.SB[min(n + i, g.N - 1)];
    f8_i32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = f8_i32x4{};
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
        if (w + d * NW < nk)
            load(blk[d], w + d * NW);
    for (int base = w; base < nk; base += DEPTH * NW) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            const int kb = base + d * NW;
            if (kb >= nk)
                break;
            Block &b = blk[d];
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) {
                    acc[i][j] = i8_mma(b.lo[FM + j], b.lo[i], acc[i][j]);
                    acc[i][j] = i8_mma(b.hi[FM + j], b.hi[i], acc[i][j]);
                }
            if (kb + DEPTH * NW < nk)
                load(b, kb + DEPTH * NW);
        }
    }
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            part[w][i * FN + j][lane] = acc[i][j];
    __syncthreads();
    const int used = min(NW, nk);
    if (w >= FM * FN || m >= g.M || n >= g.N)
        return;
    f8_i32x4 v = part[0][w][lane];
    for (int x = 1; x < used; ++x)
        v += part[x][w][lane];
    if (g.ws) {
        int *p = g.ws + ((int64_t)split * g.M + m) * g.N + n;
        if (n + 4 <= g.N) {
            *reinterpret_cast<f8_i32x4_any *>(p) = v;
        } else {
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (n + i < g.N)
                    p[i] = v[i];
        }
    } else if (g.c_type == SGEMM_TYPE_F32)
        i8_put4<float>(g, m, n, v, sa, sb);
    else if (g.c_type == SGEMM_TYPE_BF16)
        i8_put4<__bf16>(g, m, n, v, sa, sb);
    else
        i8_put4<_Float16>(g, m, n, v, sa, sb);
}

}  // namespace

hipError_t launch_i8_skinny(const I8GemmArgs &a, int cols, int splits, hipStream_t s)
{
    const unsigned grid = (unsigned)(a.tiles_n * splits);
    if (a.M > 16)
        i8_skinny_kernel<2, 1, 4><<<grid, 512, 0, s>>>(a);
    else if (cols == 16)
        i8_skinny_kernel<1, 1, 4><<<grid, 512, 0, s>>>(a);
    else
        i8_skinny_kernel<1, 2, 4><<<grid, 512, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace sgemm
