// The pipelined products of 8-bit integers, for operands whose rows start on 16-byte
// boundaries.  Stages of one k-block of 128 rotate in the LDS, filled by direct loads
// (f8_pipe.h); the sums stay in 32-bit integers from the first product to the epilogue, so
// a step is loads, fragment reads and matrix instructions alone.
#pragma once
#include "f8_pipe.h"
#include "i8_tile.h"

namespace sgemm {
namespace {

__device__ __forceinline__ F8GemmArgs i8_as_f8(const I8GemmArgs &g)
{
    F8GemmArgs a{};
    a.A = g.A;
    a.B = g.B;
    a.lda = g.lda;
    a.ldb = g.ldb;
    a.M = g.M;
    a.N = g.N;
    a.K = g.K;
    a.kb_split = g.kb_split;
    return a;
}

template <class G, int S, int MB>
struct I8Geo {
    static constexpr int FM = G::WM / MB, FN = G::WN / MB;      // blocks of a wavefront
    static constexpr int STAGE = G::ROWS * 128, BYTES = S * STAGE;
    static constexpr int OUT = MB * (G::WN + 4);                // words that MB rows of C pass through
    static_assert(G::WM % MB == 0 && G::WN % MB == 0, "whole blocks");
    static_assert(BYTES <= 160 * 1024 && G::NW * OUT * 4 <= BYTES, "LDS size");
};

// At the start of a step the fragments of the B rows and of the first A rows are in
// registers.  Each row of blocks reads the next A rows under its products.  In the last row
// every wavefront has read all of this stage: there the wavefronts meet, the stage S ahead
// is requested into its place, and the next stage's fragments are read under the last row's
// products.
//
// Bound by the matrix cores at the clock that power leaves them: 8192^3 to bf16 419 us,
// 2.62 Pop/s, from 944 with a tile that goes through registers into the LDS; the cores are
// busy 57 to 61% of the cycles at 1.76 to 1.97 GHz.  Operands of zeros take 405 us, operands
// that stay in the L2 336 to 357.
template <class G, int S, int MB>
__global__ __launch_bounds__(G::NT) void i8_pipe_kernel(I8GemmArgs g)
{
    typedef I8Geo<G, S, MB> P;
    typedef I8Block<MB> Blk;
    typedef I8Frag<MB> Frg;
    constexpr int FM = P::FM, FN = P::FN, NS = Frg::NS, LOADS = G::LOADS;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[P::BYTES];
    int tm, tn;
    const int tiles = g.tiles_m * g.tiles_n, split = blockIdx.x / tiles;
    f8_map_tile(blockIdx.x % tiles, g.tiles_m, g.tiles_n, tm, tn);
    const int m0 = tm * G::BM, n0 = tn * G::BN;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = w / G::WGN, wn = w % G::WGN;
    const F8Stages<G, S, false, false> in(i8_as_f8(g), smem, m0, n0, w, split);
    const I8Scales<MB, FM, FN> scales(g, m0 + wm * G::WM, n0 + wn * G::WN);

    typename Blk::Acc acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = typename Blk::Acc{};

    // slice s of this lane's row of a block lies at (its chunk ^ the row's swizzle) ^ 128/NS s
    const uint32_t at = lane % MB * 128, x0 = 16 * ((lane / MB) ^ f8_swz(lane % MB));
    const uint32_t at_a = wm * G::WM * 128, at_b = (G::BM + wn * G::WN) * 128;
    auto read = [&](const uint8_t *st, uint32_t first, int i, Frg &f) {
#pragma unroll
        for (int s = 0; s < NS; ++s)
            f.v[s] = *reinterpret_cast<const f8_i32x4 *>(st + first + i * MB * 128 + at + (x0 ^ (128 / NS * s)));
    };

    poison_lds(smem, P::BYTES);
    for (int st = 0; st < S - 1; ++st)
#pragma unroll
        for (int j = 0; j < LOADS; ++j)
            in.fetch(st, w, j);
    f8_wait_barrier<(S - 2) * LOADS>();
    // a row's products: NP; of a step's loads EARLY go under the last row's, the others
    // under the next step's first rows, PER at a time
    constexpr int NP = FN * NS, EARLY = LOADS < NP / 2 ? LOADS : NP / 2, FREE = (FM - 1) * NP;
    constexpr int PER = (LOADS - EARLY + FREE - 1) / FREE;
#pragma unroll
    for (int j = 0; j < EARLY; ++j)
        in.fetch(S - 1, w, j);
    if (in.nk == 1 && in.tail % 16)
        in.mask_tail();
    Frg fb[FN], ra[2];
#pragma unroll
    for (int j = 0; j < FN; ++j)
        read(smem, at_b, j, fb[j]);
    read(smem, at_a, 0, ra[0]);
    for (int kb = 0; kb < in.nk; ++kb) {
        const uint8_t *st = in.stage(kb), *next = in.stage(kb + 1);
#pragma unroll
        for (int i = 0; i < FM; ++i) {
#pragma unroll
            for (int e = 0; e < NP; ++e) {
                const int s = e / FN, j = e % FN;
                acc[i][j] = Blk::mma(fb[j].v[s], ra[i & 1].v[s], acc[i][j]);
                __builtin_amdgcn_sched_barrier(0);
                if (i + 1 < FM) {
                    if (e == 0)
                        read(st, at_a, i + 1, ra[(i + 1) & 1]);
#pragma unroll
                    for (int y = EARLY + (i * NP + e) * PER; y < EARLY + (i * NP + e + 1) * PER && y < LOADS; ++y)
                        in.fetch(kb + S - 1, w, y);
                } else {
                    if (e == 0) {
                        f8_wait_barrier<(S - 2) * LOADS>();      // stage kb+1 has landed
                        poison_lds(in.stage(kb + S), P::STAGE);
                        if (kb + 2 == in.nk && in.tail % 16)
                            in.mask_tail();
                        read(next, at_a, 0, ra[FM & 1]);
                    }
                    if (e < EARLY)
                        in.fetch(kb + S, w, e);
                    // a slice of B that this row is done with
                    if (e >= FN || NS == 1) {
                        const int ps = (e - FN) / FN, pj = (e - FN) % FN;
                        fb[pj].v[ps] = *reinterpret_cast<const f8_i32x4 *>(next + at_b + pj * MB * 128 + at +
                                                                           (x0 ^ (128 / NS * ps)));
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int j = 0; j < FN; ++j)
            fb[j].v[NS - 1] = *reinterpret_cast<const f8_i32x4 *>(next + at_b + j * MB * 128 + at + (x0 ^ (128 / NS * (NS - 1))));
        if (FM & 1)
            ra[0] = ra[1];
    }
    // the stages requested past the last one land before the LDS is used again
    f8_wait_barrier<0>();
    int *buf = reinterpret_cast<int *>(smem) + w * P::OUT;
#pragma unroll
    for (int i = 0; i < FM; ++i)
        i8_store_rows<MB, FM, FN>(g, buf, m0 + wm * G::WM + MB * i, n0 + wn * G::WN, i, acc[i], scales,
                                  g.ws ? g.ws + (int64_t)split * g.M * g.N : nullptr);
}

// The same for tiles of few blocks a wavefront: all fragments of the next stage are read
// before this stage's products, into a second set of registers.  The wavefronts meet once a
// step, when each has its set: the stage S ahead is requested into the place of the one in
// the registers.  64 x 16384 x 4096 from memory 17.9 us (3.9 TB/s of B's bytes; 13.2 with B
// still in the cache behind the L2), 23.7 on the tile that goes through registers.
template <class G, int S, int MB>
__global__ __launch_bounds__(G::NT) void i8_flat_kernel(I8GemmArgs g)
{
    typedef I8Geo<G, S, MB> P;
    typedef I8Block<MB> Blk;
    typedef I8Frag<MB> Frg;
    constexpr int FM = P::FM, FN = P::FN, NS = Frg::NS, LOADS = G::LOADS;
    static_assert((S - 1) * LOADS <= 63, "vmcnt range");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[P::BYTES];
    int tm, tn;
    const int tiles = g.tiles_m * g.tiles_n, split = blockIdx.x / tiles;
    f8_map_tile(blockIdx.x % tiles, g.tiles_m, g.tiles_n, tm, tn);
    const int m0 = tm * G::BM, n0 = tn * G::BN;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = w / G::WGN, wn = w % G::WGN;
    const F8Stages<G, S, false, false> in(i8_as_f8(g), smem, m0, n0, w, split);
    const I8Scales<MB, FM, FN> scales(g, m0 + wm * G::WM, n0 + wn * G::WN);

    typename Blk::Acc acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = typename Blk::Acc{};

    const uint32_t at = lane % MB * 128, x0 = 16 * ((lane / MB) ^ f8_swz(lane % MB));
    struct Set {
        Frg a[FM], b[FN];
    } set[2];
    auto read = [&](Set &x, int kb) {
        const uint8_t *a = in.stage(kb) + wm * G::WM * 128 + at, *b = in.stage(kb) + (G::BM + wn * G::WN) * 128 + at;
#pragma unroll
        for (int s = 0; s < NS; ++s) {
#pragma unroll
            for (int j = 0; j < FN; ++j)
                x.b[j].v[s] = *reinterpret_cast<const f8_i32x4 *>(b + j * MB * 128 + (x0 ^ (128 / NS * s)));
#pragma unroll
            for (int i = 0; i < FM; ++i)
                x.a[i].v[s] = *reinterpret_cast<const f8_i32x4 *>(a + i * MB * 128 + (x0 ^ (128 / NS * s)));
        }
    };
    auto step = [&](const Set &x, Set &next, int kb) {
        f8_wait_barrier<(S - 2) * LOADS>();  // this stage is read, and stage kb+1 has landed
        poison_lds(in.stage(kb), P::STAGE);
        if (kb + 2 == in.nk && in.tail % 16)
            in.mask_tail();
        read(next, kb + 1);
        __builtin_amdgcn_sched_barrier(0);
        constexpr int NP = FM * FN * NS, PER = (LOADS + NP - 1) / NP;
#pragma unroll
        for (int e = 0; e < NP; ++e) {
            const int s = e / (FM * FN), i = e / FN % FM, j = e % FN;
            acc[i][j] = Blk::mma(x.b[j].v[s], x.a[i].v[s], acc[i][j]);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int y = e * PER; y < (e + 1) * PER && y < LOADS; ++y)
                in.fetch(kb + S, w, y);
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    poison_lds(smem, P::BYTES);
    for (int st = 0; st < S; ++st)
#pragma unroll
        for (int j = 0; j < LOADS; ++j)
            in.fetch(st, w, j);
    f8_wait_barrier<(S - 1) * LOADS>();
    if (in.nk == 1 && in.tail % 16)
        in.mask_tail();
    read(set[0], 0);
    for (int kb = 0; kb < in.nk; kb += 2) {
        step(set[0], set[1], kb);
        if (kb + 1 < in.nk)
            step(set[1], set[0], kb + 1);
    }
    // the stages requested past the last one land before the LDS is used again
    f8_wait_barrier<0>();
    int *buf = reinterpret_cast<int *>(smem) + w * P::OUT;
#pragma unroll
    for (int i = 0; i < FM; ++i)
        i8_store_rows<MB, FM, FN>(g, buf, m0 + wm * G::WM + MB * i, n0 + wn * G::WN, i, acc[i], scales,
                                  g.ws ? g.ws + (int64_t)split * g.M * g.N : nullptr);
}

}  // namespace
}  // namespace sgemm
