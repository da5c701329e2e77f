// Products of 8-bit integers C = alpha * diag(SA) A B^T diag(SB) + beta * C on the matrix
// cores.  v_mfma_i32_16x16x64_i8 adds 64 products of each of 16 x 16 elements exactly in
// 32-bit integers; the scales meet the sum once, in the epilogue.
#include "i8_tile.h"

#include <algorithm>

namespace sgemm {
namespace {

// Rows at any byte address: a k-block of 128 goes through registers into the LDS, the
// next one is requested before it is multiplied.
template <class G>
__global__ __launch_bounds__(G::NT) void i8_tile_kernel(I8GemmArgs g)
{
    __shared__ __attribute__((aligned(1024))) uint8_t smem[G::STAGE];
    int tm, tn;
    f8_map_tile(blockIdx.x, g.tiles_m, g.tiles_n, tm, tn);
    const int m0 = tm * G::BM, n0 = tn * G::BN;
    const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = w / G::WGN, wn = w % G::WGN;

    f8_i32x4 acc[G::FM][G::FN];
#pragma unroll
    for (int i = 0; i < G::FM; ++i)
#pragma unroll
        for (int j = 0; j < G::FN; ++j)
            acc[i][j] = f8_i32x4{};

    // this work-item's chunks of a stage: rows 0 .. BM-1 are A's, the others B's; rows
    // past the matrix repeat its last one (their results are not stored)
    constexpr int NC = G::ROWS * 8 / G::NT;
    static_assert(NC * G::NT == G::ROWS * 8 && G::NT % 8 == 0, "whole chunks");
    const int c = threadIdx.x & 7;
    const uint8_t *row[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int r = (threadIdx.x + i * G::NT) >> 3;
        row[i] = (r < G::BM ? g.A + (int64_t)min(m0 + r, g.M - 1) * g.lda
                            : g.B + (int64_t)min(n0 + r - G::BM, g.N - 1) * g.ldb) + 16 * c;
    }
    f8_i32x4 x[NC];
    auto request = [&](int kb) {
        const int valid = min(g.K - kb * 128 - 16 * c, 16);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const uint8_t *p = row[i] + kb * 128;
            if (valid == 16)
                x[i] = *reinterpret_cast<const f8_i32x4_any *>(p);
            else
                x[i] = load16_any(p, valid);
        }
    };
    const int nkb = (g.K + 127) / 128;
    request(0);
    for (int kb = 0; kb < nkb; ++kb) {
        poison_lds(smem, G::STAGE);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int r = (threadIdx.x + i * G::NT) >> 3;
            *reinterpret_cast<f8_i32x4 *>(smem + r * 128 + 16 * (c ^ f8_swz(r))) = x[i];
        }
        __syncthreads();
        if (kb + 1 < nkb)
            request(kb + 1);
        auto read = [&](int r, int chunk) {
            return *reinterpret_cast<const f8_i32x4 *>(smem + r * 128 + 16 * (chunk ^ f8_swz(r)));
        };
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            f8_i32x4 b[G::FN];
#pragma unroll
            for (int j = 0; j < G::FN; ++j)
                b[j] = read(G::BM + wn * G::WN + 16 * j + l16, q + 4 * half);
#pragma unroll
            for (int i = 0; i < G::FM; ++i) {
                const f8_i32x4 a = read(wm * G::WM + 16 * i + l16, q + 4 * half);
#pragma unroll
                for (int j = 0; j < G::FN; ++j)
                    acc[i][j] = i8_mma(b[j], a, acc[i][j]);
            }
        }
        __syncthreads();
    }
    int *buf = reinterpret_cast<int *>(smem) + w * G::OUT;
#pragma unroll
    for (int i = 0; i < G::FM; ++i)
        i8_store_rows<G::FN>(g, buf, m0 + wm * G::WM + 16 * i, n0 + wn * G::WN, acc[i]);
}

typedef F8Geo<64, 64, 2, 2> GS;

}  // namespace

I8GemmPlan i8_gemm_plan(int64_t M, int64_t N, int64_t, bool, int64_t, bool)
{
    I8GemmPlan p;
    p.kid = KID_I8_ANY;
    p.tiles_m = ceil_div(M, GS::BM);
    p.tiles_n = ceil_div(N, GS::BN);
    p.threads = GS::NT;
    return p;
}

hipError_t launch_i8_gemm(I8GemmArgs a, const I8GemmPlan &p, hipStream_t s)
{
    a.tiles_m = (int)p.tiles_m;
    a.tiles_n = (int)p.tiles_n;
    i8_tile_kernel<GS><<<(unsigned)(p.tiles_m * p.tiles_n), GS::NT, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace sgemm
