// Products of 8-bit integers C = alpha * diag(SA) A B^T diag(SB) + beta * C on the matrix
// cores.  v_mfma_i32_16x16x64_i8 adds 64 products of each of 16 x 16 elements exactly in
// 32-bit integers; the scales meet the sum once, in the epilogue.
#include "i8_tile.h"

#include <algorithm>

namespace sgemm {
namespace {

// Rows at any byte address: a k-block of 128 goes through registers into the LDS, the
// next one is requested before it is multiplied.  GROUPS times G::NW wavefronts take the
// k-blocks in turn, each group in a stage of its own; their sums meet in the LDS.
//
// 1000 x 1017 x 999 packed 9.1 us, 8 k-blocks: about 10 bytes per CU and cycle however they
// are loaded (one group and operands from memory 11.6; requested 2 or 4 blocks ahead then 10.4
// to 11.1, two blocks a step 10.4, whole lines shifted in registers 12.2, in words of 4 bytes
// 15.2, and four groups 10.2): a row's 128 bytes lie in two lines, which the next block needs
// again.
template <class G, int GROUPS>
__global__ __launch_bounds__(G::NT *GROUPS) void i8_tile_kernel(I8GemmArgs g)
{
    constexpr int SUMS = G::BM * G::BN * 4;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[GROUPS * G::STAGE];
    int tm, tn;
    f8_map_tile(blockIdx.x, g.tiles_m, g.tiles_n, tm, tn);
    const int m0 = tm * G::BM, n0 = tn * G::BN;
    const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4, own = threadIdx.x % G::NT;
    const int w = __builtin_amdgcn_readfirstlane(own >> 6);
    const int group = __builtin_amdgcn_readfirstlane(threadIdx.x / G::NT);
    const int wm = w / G::WGN, wn = w % G::WGN;
    uint8_t *const st = smem + group * G::STAGE;

    const I8Scales<G::FM, G::FN> scales(g, m0 + wm * G::WM, n0 + wn * G::WN);
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
    const int c = own & 7;
    const uint8_t *row[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int r = (own + i * G::NT) >> 3;
        row[i] = (r < G::BM ? g.A + (int64_t)min(m0 + r, g.M - 1) * g.lda
                            : g.B + (int64_t)min(n0 + r - G::BM, g.N - 1) * g.ldb) + 16 * c;
    }
    const int nkb = (g.K + 127) / 128;
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
    if (group < nkb)
        request(group);
    // (all groups take as many steps, for the barriers' sake)
    for (int kb = group; kb - group < nkb; kb += GROUPS) {
        poison_lds(smem, GROUPS * G::STAGE);
        if (kb < nkb) {
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int r = (own + i * G::NT) >> 3;
                *reinterpret_cast<f8_i32x4 *>(st + r * 128 + 16 * (c ^ f8_swz(r))) = x[i];
            }
        }
        __syncthreads();
        if (kb + GROUPS < nkb)
            request(kb + GROUPS);
        auto read = [&](int r, int chunk) {
            return *reinterpret_cast<const f8_i32x4 *>(st + r * 128 + 16 * (chunk ^ f8_swz(r)));
        };
        if (kb < nkb) {
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
        }
        __syncthreads();
    }
    // the sums of the other groups go to the first, which stores them
    constexpr int NB = G::FM * G::FN;
    f8_i32x4 *const sums = reinterpret_cast<f8_i32x4 *>(smem);
    if (group > 0) {
#pragma unroll
        for (int f = 0; f < NB; ++f)
            sums[((group - 1) * NB + f) * G::NT + own] = acc[f / G::FN][f % G::FN];
    }
    if (GROUPS > 1)
        __syncthreads();
    if (group > 0)
        return;
#pragma unroll
    for (int x = 0; x < GROUPS - 1; ++x)
#pragma unroll
        for (int f = 0; f < NB; ++f)
            acc[f / G::FN][f % G::FN] += sums[(x * NB + f) * G::NT + own];
    // (each wavefront passes its rows through a place of its own, behind what others still read)
    int *buf = reinterpret_cast<int *>(smem + (GROUPS - 1) * SUMS) + w * G::OUT;
    static_assert((GROUPS - 1) * SUMS + G::NW * G::OUT * 4 <= GROUPS * G::STAGE, "LDS size");
#pragma unroll
    for (int i = 0; i < G::FM; ++i)
        i8_store_rows<G::FM, G::FN>(g, buf, m0 + wm * G::WM + 16 * i, n0 + wn * G::WN, i, acc[i], scales);
}

// C from the splits' partial sums, which are integers: their order does not matter.
__global__ __launch_bounds__(256) void i8_join_kernel(I8GemmArgs g, int splits)
{
    const int64_t per_row = ((int64_t)g.N + 7) / 8, total = per_row * g.M;
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total; e += (int64_t)gridDim.x * 256) {
        const int m = (int)(e / per_row), n = 8 * (int)(e % per_row);
        const float sa = g.SA[m];
        float sb[8];
        row_load8<false>(g.SB, n, g.N, sb);
        int v[8] = {};
        for (int x = 0; x < splits; ++x) {
            float u[8];  // (the bits of integers)
            row_load8<false>(reinterpret_cast<const float *>(g.ws) + ((int64_t)x * g.M + m) * g.N, n, g.N, u);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] += __float_as_int(u[i]);
        }
        i8_put8(g, m, n, v, sa, sb);
    }
}

typedef F8Geo<64, 64, 2, 2> GS;
// Groups of wavefronts to a workgroup for rows at any alignment: with no more than one tile to
// a CU, four (1 / 2 / 4, to FP32 without a workspace: 1000 x 1017 x 999 9.9 / 9.0 / 9.1 us, 20 x
// 8001 x 4001 31.1 / 24.1 / 21.1, 100 x 4001 x 4001 30.8 / 23.7 / 20.7, 300 x 2000 x 5001 36.5 /
// 27.9 / 24.0); with more, other tiles' workgroups fill the CU (1000 x 2001 x 1001 12.3 / 12.3 /
// 16.3, 2047^3 33.0 / 35.5 / 44.7).
int any_groups(int64_t tiles) { return tiles <= 256 ? 4 : 1; }
constexpr int64_t kMaxJoin = int64_t{64} << 20;  // bytes of partial sums a call may ask for

// What joining the splits' sums takes, in us.
double join_us(int64_t bytes) { return 2.5 + (double)bytes * 0.5e-6; }

// Which tile, and into how many parts the k-blocks are split: the least estimate of
//     2 us + the larger of (the rounds of workgroups that the 256 CUs take) and (2.2 us and
//     the operands' and C's bytes at 5 TB/s) + what joining the parts takes.
// A round of one workgroup on each CU takes (k-blocks of a part * step + ends); the 64 x 64
// tile leaves room for two, and a round of two takes (k-blocks * step2 + ends2).  The constants
// are of operands from memory; with operands in the caches the tiles take (bf16 C, us):
//                        64 x 64   128 x 64   128 x 128   256 x 256
//     256 x 4096 x 4096     11.6                               48.0
//     512 x 4096 x 1024      6.6        7.1         8.5
//     512 x 4096 x 4096     15.2       15.3        19.4        48.1
//     2048^3                17.4       18.5        12.7        29.8
//     1024 x 4096 x 4096               29.8        20.3        48.3
//     4096 x 4096 x 1024                           31.0        21.2
// and the estimate takes the fastest of each row but the third, where it is 0.1 off.
I8GemmPlan plan_tiles(int64_t M, int64_t N, int64_t K, int64_t room, double &us)
{
    static const struct { int kid, bm, bn, threads; double step, ends, step2, ends2; } kTiles[4] = {
        {KID_I8_S, 64, 64, 256, 0.30, 2.2, 0.517, 1.4}, {KID_I8_N, 128, 64, 512, 0.43, 2.5, 0, 0},
        {KID_I8_M, 128, 128, 512, 0.565, 3.1, 0, 0}, {KID_I8_L, 256, 256, 512, 1.62, 10.2, 0, 0}};
    I8GemmPlan p;
    const int64_t nk = ceil_div(K, F8_BLOCK);
    const double bytes_us = 2.2 + ((double)(M + N) * (double)K + 3.0 * (double)M * (double)N) / 5.0e6;
    for (const auto &t : kTiles) {
        const int64_t tm = ceil_div(M, t.bm), tn = ceil_div(N, t.bn);
        for (int64_t splits = 1; splits <= 16; splits *= 2) {
            const int64_t part = ceil_div(nk, splits), all = tm * tn * splits;
            if (splits > 1 && (part < 4 || (splits - 1) * part >= nk || all > 512 ||
                               splits * M * N * 4 > std::min(room, kMaxJoin)))
                break;
            const double one = (double)part * t.step + t.ends, two = (double)part * t.step2 + t.ends2;
            const double rounds = t.step2 > 0 ? (double)(all / 512) * two + (all % 512 > 256 ? two : all % 512 > 0 ? one : 0.0)
                                              : (double)ceil_div(all, 256) * one;
            const int64_t bytes = splits > 1 ? splits * M * N * 4 : 0;
            const double e = 2.0 + std::max(rounds, bytes_us) + (splits > 1 ? join_us(bytes) : 0.0);
            if (p.kid == KID_I8_NONE || e < us) {
                us = e;
                p = I8GemmPlan{t.kid, tm, tn, splits, bytes, 0, t.threads};
            }
        }
    }
    return p;
}

// Up to 16 rows: 16 columns per workgroup, 32 where that still leaves two workgroups to
// each CU (16 x 16384 x 4096 17.2 / 15.2 us, 8 x 8192 x 8192 14.5 / 18.0), k split where
// few workgroups go through a long k (1 x 1024 x 16384 11.3 us, in 8 parts with their join 9.6).
// Up to 32 rows the same with two blocks of rows, as long as one workgroup to a CU covers the
// columns and A's rows, which every workgroup reads, are short (64 x 64 tiles / this: 32 x 4096
// x 4096 9.5 / 7.9 us, 32 x 1024 x 8192 12.5 / 10.9, 17 x 500 x 1000 packed 6.6 / 3.9; but 32 x
// 8192 x 4096 11.3 / 14.1, 32 x 4096 x 16384 16.4 / 23.7).  With four blocks of rows 64 x 4096 x
// 4096 takes 11.5 against the tiles' 10.4, 64 x 8192 x 4096 21.9 against 11.4.
bool skinny(int64_t M, int64_t N, int64_t K) { return M <= 16 || (M <= 32 && N <= 4096 && K <= 8192); }
int skinny_cols(int64_t N) { return N < 16384 ? 16 : 32; }

I8GemmPlan plan_skinny(int64_t M, int64_t N, int64_t K, int64_t room)
{
    I8GemmPlan p;
    const int64_t nk = ceil_div(K, F8_BLOCK), tn = ceil_div(N, skinny_cols(N));
    double us = 0.0;
    for (int64_t splits = 1; splits <= 16; splits *= 2) {
        const int64_t part = ceil_div(nk, splits), bytes = splits > 1 ? splits * M * N * 4 : 0;
        if (splits > 1 && (part < 8 || (splits - 1) * part >= nk || tn * splits > 512 || bytes > std::min(room, kMaxJoin)))
            break;
        const double e = std::max(1.6 + 0.52 * (double)ceil_div(part, 8), (double)N * (double)K / 4.6e6) +
                         (splits > 1 ? join_us(bytes) : 0.0);
        if (splits == 1 || e < us) {
            us = e;
            p = I8GemmPlan{KID_I8_SKINNY, 1, tn, splits, bytes, 0, 512};
        }
    }
    return p;
}

}  // namespace

// Operands at other alignments go through the registers of the 64 x 64 tile, or, where that
// takes longer, are first laid out anew in the workspace with rows of whole lines.
I8GemmPlan i8_gemm_plan(int64_t M, int64_t N, int64_t K, bool aligned, int64_t room, bool may_pack)
{
    if (skinny(M, N, K))
        return plan_skinny(M, N, K, room);
    double us = 0.0;
    if (aligned && N > 1)  // (a single row of B has no distance to the next)
        return plan_tiles(M, N, K, room, us);
    I8GemmPlan p;
    p.kid = KID_I8_ANY;
    p.tiles_m = ceil_div(M, GS::BM);
    p.tiles_n = ceil_div(N, GS::BN);
    p.threads = GS::NT * any_groups(p.tiles_m * p.tiles_n);
    const int64_t ld = f8_packed_ld(K);
    if (may_pack && N > 1 && M <= F8_MAX_PACKED / ld && N <= F8_MAX_PACKED / ld && (M + N) * ld <= room) {
        const int64_t pack = (M + N) * ld;
        const I8GemmPlan q = plan_tiles(M, N, K, room - pack, us);
        const double any = 2.5 + (double)ceil_div(K, F8_BLOCK) * std::max(0.62, (double)p.tiles_m * (double)p.tiles_n * 0.9e-3);
        if (us + 4.0 + (double)pack * 0.35e-6 < any) {
            p = q;
            p.bytes += pack;
            p.pack = pack;
        }
    }
    return p;
}

hipError_t launch_i8_gemm(I8GemmArgs a, const I8GemmPlan &p, hipStream_t s)
{
    a.tiles_m = (int)p.tiles_m;
    a.tiles_n = (int)p.tiles_n;
    if (p.kid >= KID_I8_S && !p.pack && std::max(a.lda, a.ldb) > F8_MAX_LD)
        return hipErrorInvalidValue;  // (the pipelined kernels' offsets have 32 bits)
    if (p.pack) {
        F8GemmArgs f{};
        f.A = a.A;
        f.B = a.B;
        f.lda = a.lda;
        f.ldb = a.ldb;
        f.M = a.M;
        f.N = a.N;
        f.K = a.K;
        uint8_t *to = reinterpret_cast<uint8_t *>(a.ws);
        const hipError_t e = launch_f8_pack(f, to, s);
        if (e != hipSuccess)
            return e;
        const int64_t ld = f8_packed_ld(a.K);
        a.A = to;
        a.B = to + (int64_t)a.M * ld;
        a.lda = a.ldb = ld;
        a.ws = reinterpret_cast<int *>(to + p.pack);
    }
    if (p.splits == 1)
        a.ws = nullptr;
    const int splits = (int)p.splits;
    a.kb_split = (int)ceil_div(ceil_div(a.K, F8_BLOCK), splits);
    hipError_t e = hipSuccess;
    if (p.kid == KID_I8_SKINNY) {
        e = launch_i8_skinny(a, skinny_cols(a.N), splits, s);
    } else if (p.kid == KID_I8_ANY) {
        if (any_groups(p.tiles_m * p.tiles_n) == 4)
            i8_tile_kernel<GS, 4><<<(unsigned)(p.tiles_m * p.tiles_n), p.threads, 0, s>>>(a);
        else
            i8_tile_kernel<GS, 1><<<(unsigned)(p.tiles_m * p.tiles_n), p.threads, 0, s>>>(a);
        e = hipGetLastError();
    } else {
        e = launch_i8_tile(a, p.kid, splits, s);
    }
    if (e != hipSuccess || splits == 1)
        return e;
    i8_join_kernel<<<(unsigned)std::min<int64_t>(ceil_div((int64_t)a.M * ceil_div(a.N, 8), 256), 2048), 256, 0, s>>>(a, splits);
    return hipGetLastError();
}

}  // namespace sgemm
