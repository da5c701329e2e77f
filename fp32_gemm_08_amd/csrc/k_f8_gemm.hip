// 8-bit block-scaled product C = alpha * A * B^T + beta * C on the matrix
// cores, which add up one k-block of 128 products; the FP32 factor sA*sB of
// that k-block scales the sum, and a second FP32 sum runs over the k-blocks:
//
//   C[m][n] = alpha * sum_b sA[b][m] * sB[b][n] * (sum_{k in b} qA[m][k] * qB[n][k])
//
// A 16-bit C is computed by v_mfma_f32_16x16x128_f8f6f4, at twice the rate of the
// 16-bit instructions.  That instruction adds products in groups of 8, each group
// aligned to its largest product with 13 bits kept below it (measured: 2^16 + 8
// keeps the 8, 2^16 + 7 loses the 7).  Seven products of a group lose at most 2^-13
// of the largest each, so a k-block's sum is off by at most 7 * 2^-13 = 8.5e-4 of
// sum |qA qB|: below a bf16 C's half step of 2^-8, above an fp16 C's of 2^-11.  The
// losses mostly cancel: on normally distributed operands the sum of 128 is off by
// 1.5e-5 of its size (2-norm of the errors over that of the sums).  Relative to a sum
// whose products cancel it is more, and there it, not C's type, decides the error.
// An FP32 C is meant to hold more than that (a gradient that is accumulated over many
// calls): its 8-bit operands are turned into bf16, which holds every e4m3 and e5m2
// value, and go through v_mfma_f32_16x16x32_bf16, whose sums are FP32 (1e-8 on the
// same operands, in the same measure; the FP32 additions over the k-blocks bring C to
// 4e-8 at K = 128 and 1e-7 at K = 16384).
//
// The instructions take rows of B as their first operand and rows of A as their
// second, so that lane l holds C[m = l % 16][n = 4*(l/16) .. +3]: four
// consecutive columns of one row, one store, and one factor where a k-block's
// B scale is the same for 128 columns.  Lane l supplies 32 values of row
// l % 16 of each operand, the 16-byte chunks l/16 and 4 + l/16 of its 128
// (which 32 is free as long as both operands agree: the sum runs over all).
#include "f8_tile.h"

#include <algorithm>

namespace sgemm {
namespace {

// Rows at any byte address: a k-block goes through registers into the LDS, the next
// one is requested before it is multiplied.
template <class G, int FA, int FB, bool ROWB, bool EXACT>
__global__ __launch_bounds__(G::NT) void f8_tile_kernel(F8GemmArgs g)
{
    __shared__ __attribute__((aligned(1024))) uint8_t smem[G::STAGE];
    float *sc = reinterpret_cast<float *>(smem + G::ROWS * 128);
    int tm, tn;
    f8_map_tile(blockIdx.x, g.tiles_m, g.tiles_n, tm, tn);
    const int m0 = tm * G::BM, n0 = tn * G::BN;
    const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = w / G::WGN, wn = w % G::WGN;

    f8_f32x4 acc[G::FM][G::FN];
#pragma unroll
    for (int i = 0; i < G::FM; ++i)
#pragma unroll
        for (int j = 0; j < G::FN; ++j)
            acc[i][j] = f8_f32x4{};

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
    constexpr int NS = G::BM + (ROWB ? G::BN : 0);
    static_assert(NS <= G::NT, "a scale per work-item");
    f8_i32x4 x[NC];
    float scale = 0.0f, sb = 0.0f, sb_next = 0.0f;
    auto request = [&](int kb) {
        const int valid = (int)min<int64_t>(g.K - (int64_t)kb * 128 - 16 * c, 16);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const uint8_t *p = row[i] + (int64_t)kb * 128;
            if (valid == 16)
                x[i] = *reinterpret_cast<const f8_i32x4_any *>(p);
            else
                x[i] = load16_any(p, valid);
        }
        const int r = threadIdx.x;
        if (r < G::BM)
            scale = g.SA[kb * g.ldsa + min(m0 + r, g.M - 1)];
        else if (r < NS)
            scale = g.SB[kb * g.ldsb + min(n0 + r - G::BM, g.N - 1)];
        if constexpr (!ROWB)
            sb_next = g.SB[(int64_t)(min(n0 + wn * G::WN, g.N - 1) / 128) * g.ldsb + kb];
    };
    const int nkb = (int)(((int64_t)g.K + 127) / 128);
    request(0);
    for (int kb = 0; kb < nkb; ++kb) {
        poison_lds(smem, G::STAGE);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int r = (threadIdx.x + i * G::NT) >> 3;
            *reinterpret_cast<f8_i32x4 *>(smem + r * 128 + 16 * (c ^ f8_swz(r))) = x[i];
        }
        if (threadIdx.x < NS)
            sc[threadIdx.x] = scale;
        sb = sb_next;
        __syncthreads();
        if (kb + 1 < nkb)
            request(kb + 1);
        Frag<FB, EXACT> fb[G::FN];
#pragma unroll
        for (int j = 0; j < G::FN; ++j) {
            const int r = G::BM + wn * G::WN + 16 * j + l16;
            fb[j].set(f8_join(*reinterpret_cast<const f8_i32x4 *>(smem + r * 128 + 16 * (q ^ f8_swz(r))),
                              *reinterpret_cast<const f8_i32x4 *>(smem + r * 128 + 16 * ((q + 4) ^ f8_swz(r)))));
        }
#pragma unroll
        for (int i = 0; i < G::FM; ++i) {
            const int r = wm * G::WM + 16 * i + l16;
            Frag<FA, EXACT> fa;
            fa.set(f8_join(*reinterpret_cast<const f8_i32x4 *>(smem + r * 128 + 16 * (q ^ f8_swz(r))),
                           *reinterpret_cast<const f8_i32x4 *>(smem + r * 128 + 16 * ((q + 4) ^ f8_swz(r)))));
            const float sa = sc[r];
#pragma unroll
            for (int j = 0; j < G::FN; ++j) {
                const f8_f32x4 t = f8_mma<FA, FB>(fb[j], fa);
                if constexpr (ROWB) {
                    const f8_f32x4 s = *reinterpret_cast<const f8_f32x4 *>(sc + G::BM + wn * G::WN + 16 * j + 4 * q);
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        acc[i][j][x] = fmaf(t[x], sa * s[x], acc[i][j][x]);
                } else {
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        acc[i][j][x] = fmaf(t[x], sa * sb, acc[i][j][x]);
                }
            }
        }
        __syncthreads();
    }
    __syncthreads();
    float *buf = reinterpret_cast<float *>(smem) + w * G::OUT;
#pragma unroll
    for (int i = 0; i < G::FM; ++i)
        store_rows<G::FN>(g, buf, m0 + wm * G::WM + 16 * i, n0 + wn * G::WN, acc[i]);
}

template <typename T>
__global__ __launch_bounds__(256) void f8_scale_kernel(T *C, int64_t ldc, int rows, int cols, float beta)
{
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x)
        for (int64_t c = threadIdx.x; c < cols; c += 256)
            C[row * ldc + c] = (T)(beta != 0.0f ? beta * (float)C[row * ldc + c] : 0.0f);
}

// C <- alpha * (the splits' partial sums, in order) + beta * C.
template <typename T>
__global__ __launch_bounds__(256) void f8_join_kernel(F8GemmArgs g, int splits)
{
    const int64_t per_row = ((int64_t)g.N + 7) / 8, total = per_row * g.M;
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total; e += (int64_t)gridDim.x * 256) {
        const int m = (int)(e / per_row), n = 8 * (int)(e % per_row);
        float v[8];
        row_load8<false>(g.ws + (int64_t)m * g.N, n, g.N, v);
        for (int x = 1; x < splits; ++x) {
            float u[8];
            row_load8<false>(g.ws + ((int64_t)x * g.M + m) * g.N, n, g.N, u);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] += u[i];
        }
        put8<T>(g, m, n, v);
    }
}

// The rows of A, then those of B, laid out with `ld` bytes a row, zeros past K.
__global__ __launch_bounds__(256) void f8_pack_kernel(F8GemmArgs g, uint8_t *to, int64_t ld)
{
    const int64_t per_row = ld / 16, total = ((int64_t)g.M + g.N) * per_row;
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total; e += (int64_t)gridDim.x * 256) {
        const int64_t r = e / per_row, k = 16 * (e % per_row);
        const uint8_t *p = (r < g.M ? g.A + r * g.lda : g.B + (r - g.M) * g.ldb) + k;
        const int valid = (int)min<int64_t>(g.K - k, 16);
        *reinterpret_cast<f8_i32x4 *>(to + r * ld + k) =
            valid == 16 ? *reinterpret_cast<const f8_i32x4_any *>(p) : load16_any(p, valid);
    }
}

typedef F8Geo<64, 64, 2, 2> GS;
constexpr int64_t kMaxJoin = int64_t{64} << 20;  // bytes of partial sums a call may ask for

}  // namespace

// Which tile, and into how many parts the k-blocks are split: the least estimate of
//     2 us + rounds * (k-blocks of a part * step + ends) + what joining the parts takes,
// a round being a workgroup on each of the 256 CUs (a tile's LDS leaves room for one).
// The constants are measured, bf16 C: 64 x 64 tiles 1024^3 7.4 us, 256 x 4096 x 4096
// 16.1; 128 x 64 512 x 4096 x 1024 8.9, x 4096 20.4; 128 x 128 2048^3 15.1, 1024 x
// 4096 x 4096 25.3; 256 x 256 4096 x 4096 x 1024 22.1, 4096^3 59.6; joining 2 MB 3.5,
// 16 MB 10.5.  28 shapes from 65 x 1024 x 1024 to 8192 x 8192 x 1024 were timed with
// every tile and 1 to 16 parts.  Of a bf16 C and tile scales the estimate takes the
// fastest or one within 2.2% but for two: 128 x 512 x 16384 17.2 us where 14.9 is
// possible, 256 x 256 x 4096 10.5 where 9.8 is.  It does not know an FP32 C, which takes
// about twice the step with each tile: there, with row scales, it is within 2% but for
// 512 x 4096 x 16384 (91.3, possible 84.7) and 2048 x 2048 x 16384 (151, 140).  `us` is
// the estimate.
static F8GemmPlan plan_tiles(int64_t M, int64_t N, int64_t K, int64_t room, double &us)
{
    static const struct { int kid, bm, bn; double step, ends; } kTiles[4] = {{KID_F8_S, 64, 64, 0.36, 2.4},
                                                                              {KID_F8_N, 128, 64, 0.45, 3.0},
                                                                              {KID_F8_M, 128, 128, 0.6, 3.0},
                                                                              {KID_F8_L, 256, 256, 1.6, 7.5}};
    F8GemmPlan p;
    const int64_t nk = ceil_div(K, F8_BLOCK);
    for (const auto &t : kTiles) {
        const int64_t tm = ceil_div(M, t.bm), tn = ceil_div(N, t.bn);
        for (int64_t splits = 1; splits <= 16; splits *= 2) {
            const int64_t part = ceil_div(nk, splits);
            if (splits > 1 && (part < 4 || (splits - 1) * part >= nk || tm * tn * splits > 256 ||
                               splits * M * N * 4 > std::min(room, kMaxJoin)))
                break;
            const int64_t bytes = splits > 1 ? splits * M * N * 4 : 0;
            const double e = 2.0 + (double)ceil_div(tm * tn * splits, 256) * ((double)part * t.step + t.ends) +
                             (splits > 1 ? 2.5 + (double)bytes * 0.5e-6 : 0.0);
            if (p.kid == KID_F8_NONE || e < us) {
                us = e;
                p = F8GemmPlan{t.kid, tm, tn, splits, bytes, 0};
            }
        }
    }
    return p;
}

// Operands at other alignments go through the registers of the 64 x 64 tile, or, where
// that takes longer, are first laid out anew in the workspace with rows of whole lines.
// Measured (bf16 C, packed rows), through registers / laid out first: 1000 x 1017 x 999
// 10.9 / 12.8 us, 512 x 4096 x 4095 35.3 / 27.5, 2048 x 2048 x 2047 33.6 / 20.8, 4096 x
// 4096 x 4095 212 / 75.
F8GemmPlan f8_gemm_plan(bool row_b, int64_t M, int64_t N, int64_t K, bool aligned, int64_t room, bool may_pack)
{
    F8GemmPlan p;
    double us = 0.0;
    aligned = aligned && K <= F8_MAX_LD;  // (rows that do not overlap lie at least K apart)
    // few rows of A; of operands at other alignments up to 16 (N = K = 4096, through the
    // wavefronts' registers / through the 64 x 64 tile: 1 row 11.3 / 17.3 us, 16 rows
    // 17.6 / 17.7, 32 rows 25.0 / 18.0).  Aligned up to 64 (through registers / the fastest
    // tile, bf16 C and tile scales; FP32 C and row scales): 64 x 4096 x 4096 12.9 / 13.0;
    // 14.2 / 14.9, 64 x 1024 x 1024 5.6 / 6.8; 5.7 / 8.8, 32 x 4096 x 4096 9.2 / 11.7; 9.3 /
    // 13.7.  The rule does not look at N and K, and loses with many columns or a deep k:
    // 64 x 16384 x 4096 24.4 / 16.3; 48.6 / 23.9, 64 x 1024 x 16384 39.8 / 14.8; 42.2 / 18.0
    if (M <= (aligned ? 64 : 16)) {
        p.kid = KID_F8_SKINNY;
        p.tiles_m = 1;
        p.tiles_n = ceil_div(N, f8_skinny_cols(row_b, N));
        return p;
    }
    if (aligned && N > 1)  // (a single row of B has no distance to the next)
        return plan_tiles(M, N, K, room, us);
    p.kid = KID_F8_ANY;
    p.tiles_m = ceil_div(M, GS::BM);
    p.tiles_n = ceil_div(N, GS::BN);
    if (may_pack && N > 1 && f8_packed_ld(K) <= F8_MAX_LD && M <= F8_MAX_PACKED / f8_packed_ld(K) && N <= F8_MAX_PACKED / f8_packed_ld(K)) {
        const int64_t pack = (M + N) * f8_packed_ld(K);
        if (pack <= room) {
            const F8GemmPlan q = plan_tiles(M, N, K, room - pack, us);
            const double any = 3.0 + (double)ceil_div(K, F8_BLOCK) *
                                         std::max(1.0, (double)p.tiles_m * (double)p.tiles_n * 1.7e-3);
            if (us + 4.0 + (double)pack * 0.35e-6 < any) {
                p = q;
                p.bytes += pack;
                p.pack = pack;
            }
        }
    }
    return p;
}

// Whether the tile scales of B lie near enough for the pipelined kernels (a tile of up to
// 128 columns reads one row of them).
static bool f8_scales_near(const F8GemmArgs &a, bool row_b)
{
    return row_b || a.N <= 128 || a.ldsb <= F8_MAX_LD;
}

F8GemmPlan f8_call_plan(const F8GemmArgs &a, bool rows_on_16, bool row_b, int64_t room)
{
    const bool near = f8_scales_near(a, row_b);
    const bool aligned = rows_on_16 && near && (a.M <= 1 || a.lda <= F8_MAX_LD) && (a.N <= 1 || a.ldb <= F8_MAX_LD);
    return f8_gemm_plan(row_b, a.M, a.N, a.K, aligned, room, near);
}

hipError_t launch_f8_pack(const F8GemmArgs &a, uint8_t *to, hipStream_t s)
{
    const int64_t ld = f8_packed_ld(a.K), chunks = ((int64_t)a.M + a.N) * (ld / 16);
    f8_pack_kernel<<<(unsigned)std::min<int64_t>(ceil_div(chunks, 256), 16384), 256, 0, s>>>(a, to, ld);
    return hipGetLastError();
}

hipError_t launch_f8_gemm(F8GemmArgs a, const F8GemmPlan &p, int format_a, int format_b, bool row_b, hipStream_t s)
{
    a.tiles_m = (int)p.tiles_m;
    a.tiles_n = (int)p.tiles_n;
    if (p.kid >= KID_F8_S) {  // what the pipelined kernels' 32-bit offsets need
        const int64_t ld = p.pack ? f8_packed_ld(a.K) : std::max(a.lda, a.ldb);
        if (ld > F8_MAX_LD || !f8_scales_near(a, row_b))
            return hipErrorInvalidValue;
    }
    if (p.pack) {
        const int64_t ld = f8_packed_ld(a.K);
        uint8_t *to = reinterpret_cast<uint8_t *>(a.ws);
        const hipError_t e = launch_f8_pack(a, to, s);
        if (e != hipSuccess)
            return e;
        a.A = to;
        a.B = to + (int64_t)a.M * ld;
        a.lda = a.ldb = ld;
        a.ws = reinterpret_cast<float *>(to + p.pack);
    }
    if (p.splits == 1)
        a.ws = nullptr;
    const int nk = (int)ceil_div(a.K, F8_BLOCK), splits = (int)p.splits;
    a.kb_split = (nk + splits - 1) / splits;
    hipError_t e;
    switch (p.kid) {
    case KID_F8_SKINNY:
        return launch_f8_skinny(a, format_a, format_b, row_b, s);
    case KID_F8_ANY: {
        const dim3 grid((unsigned)(a.tiles_m * a.tiles_n)), block(GS::NT);
        on_format(format_a, [&](auto FA) { on_format(format_b, [&](auto FB) { on_bool(row_b, [&](auto ROWB) {
            on_bool(a.c_type == SGEMM_TYPE_F32, [&](auto EX) {
                f8_tile_kernel<GS, FA(), FB(), ROWB(), EX()><<<grid, block, 0, s>>>(a);
            }); }); }); });
        return hipGetLastError();
    }
    case KID_F8_S:
        e = launch_f8_small(a, splits, format_a, format_b, row_b, s);
        break;
    case KID_F8_N:
        e = launch_f8_narrow(a, splits, format_a, format_b, row_b, s);
        break;
    case KID_F8_M:
        e = launch_f8_medium(a, splits, format_a, format_b, row_b, s);
        break;
    default:
        e = launch_f8_large(a, splits, format_a, format_b, row_b, s);
        break;
    }
    if (e != hipSuccess || splits == 1)
        return e;
    const unsigned grid = (unsigned)std::min<int64_t>(ceil_div((int64_t)a.M * ceil_div(a.N, 8), 256), 2048);
    if (a.c_type == SGEMM_TYPE_F32)
        f8_join_kernel<float><<<grid, 256, 0, s>>>(a, splits);
    else if (a.c_type == SGEMM_TYPE_FP16)
        f8_join_kernel<_Float16><<<grid, 256, 0, s>>>(a, splits);
    else
        f8_join_kernel<__bf16><<<grid, 256, 0, s>>>(a, splits);
    return hipGetLastError();
}

hipError_t launch_f8_scale(void *C, int64_t ldc, int rows, int cols, int c_type, float beta, hipStream_t s)
{
    const unsigned grid = (unsigned)std::min(rows, 1 << 20);  // (within one launch's work-items)
    if (c_type == SGEMM_TYPE_F32)
        f8_scale_kernel<<<grid, 256, 0, s>>>(static_cast<float *>(C), ldc, rows, cols, beta);
    else if (c_type == SGEMM_TYPE_FP16)
        f8_scale_kernel<<<grid, 256, 0, s>>>(static_cast<_Float16 *>(C), ldc, rows, cols, beta);
    else
        f8_scale_kernel<<<grid, 256, 0, s>>>(static_cast<__bf16 *>(C), ldc, rows, cols, beta);
    return hipGetLastError();
}

}  // namespace sgemm
