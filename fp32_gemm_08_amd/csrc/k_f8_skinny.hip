// 8-bit block-scaled products with few rows of A (single tokens of a batch): the
// bytes of B bound them.  The operation is that of k_f8_gemm.hip.
#include "f8_mma.h"

namespace sgemm {
namespace {

// Columns n .. n+3 of row m of C <- alpha * v + beta * C.
template <typename T>
__device__ __forceinline__ void put4(const F8GemmArgs &g, int m, int n, f8_f32x4 v)
{
    typedef T V4 __attribute__((ext_vector_type(4)));
    typedef V4 V4any __attribute__((aligned(1)));
    T *p = static_cast<T *>(g.C) + (int64_t)m * g.ldc + n;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] *= g.alpha;
    if (n + 4 <= g.N) {
        if (g.beta != 0.0f) {
            const V4 old = *reinterpret_cast<const V4any *>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = fmaf(g.beta, (float)old[i], v[i]);
        }
        V4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = (T)v[i];
        *reinterpret_cast<V4any *>(p) = o;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i < g.N)
                p[i] = (T)(g.beta != 0.0f ? fmaf(g.beta, (float)p[i], v[i]) : v[i]);
    }
}

// Up to 16 FM rows of A: a workgroup has 16 FN columns of C, and its 8
// wavefronts take the k-blocks in turn, each lane loading its operands straight
// into registers, DEPTH k-blocks ahead.  The wavefronts' sums are added in order
// through the LDS.
template <int FM, int FN, int DEPTH, int FA, int FB, bool ROWB, bool EXACT>
__global__ __launch_bounds__(512) void f8_skinny_kernel(F8GemmArgs g)
{
    constexpr int NW = 8, NF = FM + FN;
    __shared__ f8_f32x4 part[NW][FM * FN][64];
    poison_lds(part, (int)sizeof(part));
    const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x * 16 * FN;
    const int nk = (int)(((int64_t)g.K + 127) / 128);

    // rows past the matrix repeat its last one (their results are not stored)
    const uint8_t *row[NF];
#pragma unroll
    for (int i = 0; i < FM; ++i)
        row[i] = g.A + (int64_t)min(16 * i + l16, g.M - 1) * g.lda + 16 * q;
#pragma unroll
    for (int j = 0; j < FN; ++j)
        row[FM + j] = g.B + (int64_t)min(n0 + 16 * j + l16, g.N - 1) * g.ldb + 16 * q;

    struct Block {
        f8_i32x8 x[NF];
        float sa[FM], sb[ROWB ? 4 * FN : 1];
    } blk[DEPTH];
    auto load = [&](Block &b, int kb) {
        if ((int64_t)kb * 128 + 128 <= g.K) {
#pragma unroll
            for (int i = 0; i < NF; ++i)
                b.x[i] = f8_join(*reinterpret_cast<const f8_i32x4_any *>(row[i] + (int64_t)kb * 128),
                                 *reinterpret_cast<const f8_i32x4_any *>(row[i] + (int64_t)kb * 128 + 64));
        } else {
            const int valid = g.K - kb * 128 - 16 * q;
#pragma unroll
            for (int i = 0; i < NF; ++i) {
                const uint8_t *p = row[i] + (int64_t)kb * 128;
                b.x[i] = f8_join(load16_any(p, min(valid, 16)), load16_any(p + 64, min(valid - 64, 16)));
            }
        }
#pragma unroll
        for (int i = 0; i < FM; ++i)
            b.sa[i] = g.SA[kb * g.ldsa + min(16 * i + l16, g.M - 1)];
        if constexpr (ROWB) {
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    b.sb[4 * j + x] = g.SB[kb * g.ldsb + min(n0 + 16 * j + 4 * q + x, g.N - 1)];
        } else {
            b.sb[0] = g.SB[(int64_t)(n0 / 128) * g.ldsb + kb];
        }
    };

    f8_f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = f8_f32x4{};
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
            Frag<FB, EXACT> fb[FN];
#pragma unroll
            for (int j = 0; j < FN; ++j)
                fb[j].set(b.x[FM + j]);
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                Frag<FA, EXACT> fa;
                fa.set(b.x[i]);
#pragma unroll
                for (int j = 0; j < FN; ++j) {
                    const f8_f32x4 t = f8_mma<FA, FB>(fb[j], fa);
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        acc[i][j][x] = fmaf(t[x], b.sa[i] * b.sb[ROWB ? 4 * j + x : 0], acc[i][j][x]);
                }
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
#pragma unroll
    for (int f = w; f < FM * FN; f += NW) {
        const int m = 16 * (f / FN) + l16, n = n0 + 16 * (f % FN) + 4 * q;
        if (m >= g.M || n >= g.N)
            continue;
        f8_f32x4 v = part[0][f][lane];
        for (int x = 1; x < used; ++x)
            v += part[x][f][lane];
        if (g.c_type == SGEMM_TYPE_F32)
            put4<float>(g, m, n, v);
        else if (g.c_type == SGEMM_TYPE_BF16)
            put4<__bf16>(g, m, n, v);
        else
            put4<_Float16>(g, m, n, v);
    }
}

template <int FM, int FN, bool ROWB>
void launch(const F8GemmArgs &a, int fa, int fb, hipStream_t s)
{
    // k-blocks in flight; of the largest operands (4 and 4 blocks of 16 rows) one is already
    // more than the 256 registers hold: 15 are spilled with a 16-bit C, 39 with an FP32 C
    constexpr int DEPTH = FM + FN <= 2 ? 4 : FM + FN <= 5 ? 2 : 1;
    const dim3 grid((unsigned)a.tiles_n), block(512);
    on_format(fa, [&](auto FA) { on_format(fb, [&](auto FB) { on_bool(a.c_type == SGEMM_TYPE_F32, [&](auto EX) {
        f8_skinny_kernel<FM, FN, DEPTH, FA(), FB(), ROWB, EX()><<<grid, block, 0, s>>>(a);
    }); }); });
}

}  // namespace

// Columns per workgroup: as many as leave a workgroup per CU, since the rows of
// A are read once per workgroup.  Measured with 16 / 32 / 64 columns (K = 4096,
// bf16 C): 48 x 16384 35.1 / 24.3 / 18.2 us, 16 x 16384 17.8 / 15.8 / 13.4;
// 32 x 8192 (K = 8192) 25.1 / 18.9 / 27.0; 1 x 4096 5.4 / 7.1 / 10.6, 64 x 4096
// 12.8 / 15.5 / 18.9.  Row blocks of B need a scale per column: 16 columns.
int f8_skinny_cols(bool row_b, int64_t N) { return row_b || N < 32 * 256 ? 16 : N < 64 * 256 ? 32 : 64; }

hipError_t launch_f8_skinny(const F8GemmArgs &a, int fa, int fb, bool row_b, hipStream_t s)
{
    const int fm = (a.M + 15) / 16, cols = f8_skinny_cols(row_b, a.N);
    auto with = [&](auto FM) {
        row_b        ? launch<FM(), 1, true>(a, fa, fb, s)
        : cols == 64 ? launch<FM(), 4, false>(a, fa, fb, s)
        : cols == 32 ? launch<FM(), 2, false>(a, fa, fb, s)
                     : launch<FM(), 1, false>(a, fa, fb, s);
    };
    fm == 1 ? with(Int<1>{}) : fm == 2 ? with(Int<2>{}) : fm == 3 ? with(Int<3>{}) : with(Int<4>{});
    return hipGetLastError();
}

}  // namespace sgemm
