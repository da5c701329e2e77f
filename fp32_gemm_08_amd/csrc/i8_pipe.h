// The pipelined products of 8-bit integers, for operands whose rows start on 16-byte
// boundaries.  Stages of one k-block of 128 rotate in the LDS, filled by direct loads
// (f8_pipe.h); the sums stay in 32-bit integers from the first product to the epilogue, so
// a step is loads, fragment reads and matrix instructions alone.
#pragma once
#include "f8_pipe.h"
#include "i8_tile.h"

namespace sgemm {
namespace {

template <class G, int S> using I8Stages = F8Stages<G, S, false, false, false>;

template <class G, int S>
struct I8Pipe {
    static constexpr int STAGE = G::ROWS * 128, BYTES = S * STAGE;
    static_assert(BYTES <= 160 * 1024 && G::NW * G::OUT * 4 <= BYTES, "LDS size");
};

// At the start of a step the fragments of the B rows and of the first A rows are in
// registers.  Each row of blocks reads the next A rows under its products.  In the last row
// every wavefront has read all of this stage: there the wavefronts meet, the stage S ahead
// is requested into its place, and the next stage's fragments are read under the last row's
// products.
//
// Bound by the loads: 8192^3 to bf16 takes 417 to 426 us, 2.6 Pop/s (944 with a tile that goes
// through registers into the LDS), operands that stay in the L2 336 to 357, and operands of
// zeros, which draw less power, still 405; the matrix cores are busy 57 to 61% of the cycles,
// at 1.76 GHz in long runs and 1.97 in short ones.
template <class G, int S>
__global__ __launch_bounds__(G::NT) void i8_pipe_kernel(I8GemmArgs g)
{
    typedef I8Pipe<G, S> P;
    constexpr int FM = G::FM, FN = G::FN, LOADS = G::LOADS;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[P::BYTES];
    int tm, tn;
    const int tiles = g.tiles_m * g.tiles_n, split = blockIdx.x / tiles;
    f8_map_tile(blockIdx.x % tiles, g.tiles_m, g.tiles_n, tm, tn);
    const int m0 = tm * G::BM, n0 = tn * G::BN;
    const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = w / G::WGN, wn = w % G::WGN;
    const I8Stages<G, S> in(g, smem, m0, n0, w, split);
    const I8Scales<FM, FN> scales(g, m0 + wm * G::WM, n0 + wn * G::WN);

    f8_i32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = f8_i32x4{};

    // slice s of this lane's row of a block lies at (its chunk ^ the row's swizzle) ^ 64 s
    const uint32_t at = l16 * 128, x0 = 16 * (q ^ f8_swz(l16));
    const uint32_t at_a = wm * G::WM * 128, at_b = (G::BM + wn * G::WN) * 128;
    auto read = [&](const uint8_t *st, uint32_t first, int i, I8Frag &f) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
            f.v[s] = *reinterpret_cast<const f8_i32x4 *>(st + first + i * 2048 + at + (x0 ^ (64 * s)));
    };

    poison_lds(smem, P::BYTES);
    for (int st = 0; st < S - 1; ++st)
#pragma unroll
        for (int j = 0; j < LOADS; ++j)
            in.fetch(st, w, j);
    f8_wait_barrier<(S - 2) * LOADS>();
    // a row's products: NP; of a step's loads EARLY go under the last row's, the others
    // under the next step's first rows, PER at a time
    constexpr int NP = 2 * FN, EARLY = LOADS < NP / 2 ? LOADS : NP / 2, FREE = (FM - 1) * NP;
    constexpr int PER = (LOADS - EARLY + FREE - 1) / FREE;
#pragma unroll
    for (int j = 0; j < EARLY; ++j)
        in.fetch(S - 1, w, j);
    if (in.nk == 1 && in.tail % 16)
        in.mask_tail();
    I8Frag fb[FN], ra[2];
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
                acc[i][j] = i8_mma(fb[j].v[s], ra[i & 1].v[s], acc[i][j]);
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
                    // the first slices of B, which this row is done with
                    if (e >= FN)
                        fb[e - FN].v[0] = *reinterpret_cast<const f8_i32x4 *>(next + at_b + (e - FN) * 2048 + at + x0);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int j = 0; j < FN; ++j)
            fb[j].v[1] = *reinterpret_cast<const f8_i32x4 *>(next + at_b + j * 2048 + at + (x0 ^ 64));
        if (FM & 1)
            ra[0] = ra[1];
    }
    // the stages requested past the last one land before the LDS is used again
    f8_wait_barrier<0>();
    int *buf = reinterpret_cast<int *>(smem) + w * G::OUT;
#pragma unroll
    for (int i = 0; i < FM; ++i)
        i8_store_rows<FM, FN>(g, buf, m0 + wm * G::WM + 16 * i, n0 + wn * G::WN, i, acc[i], scales,
                                  g.ws ? g.ws + (int64_t)split * g.M * g.N : nullptr);
}

// The same for tiles of few blocks a wavefront: all fragments of the next stage are read
// before this stage's products, into a second set of registers.  The wavefronts meet once a
// step, when each has its set: the stage S ahead is requested into the place of the one in
// the registers.  64 x 16384 x 4096 from memory 17.9 us (3.9 TB/s of B's bytes); with B still
// in the cache behind the L2 13.2, 15.7 on the tile that goes through registers.
template <class G, int S>
__global__ __launch_bounds__(G::NT) void i8_flat_kernel(I8GemmArgs g)
{
    typedef I8Pipe<G, S> P;
    constexpr int FM = G::FM, FN = G::FN, LOADS = G::LOADS;
    static_assert((S - 1) * LOADS <= 63, "vmcnt range");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[P::BYTES];
    int tm, tn;
    const int tiles = g.tiles_m * g.tiles_n, split = blockIdx.x / tiles;
    f8_map_tile(blockIdx.x % tiles, g.tiles_m, g.tiles_n, tm, tn);
    const int m0 = tm * G::BM, n0 = tn * G::BN;
    const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = w / G::WGN, wn = w % G::WGN;
    const I8Stages<G, S> in(g, smem, m0, n0, w, split);
    const I8Scales<FM, FN> scales(g, m0 + wm * G::WM, n0 + wn * G::WN);

    f8_i32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = f8_i32x4{};

    const uint32_t at = l16 * 128, x0 = 16 * (q ^ f8_swz(l16));
    struct Set {
        I8Frag a[FM], b[FN];
    } set[2];
    auto read = [&](Set &x, int kb) {
        const uint8_t *a = in.stage(kb) + wm * G::WM * 128 + at, *b = in.stage(kb) + (G::BM + wn * G::WN) * 128 + at;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int j = 0; j < FN; ++j)
                x.b[j].v[s] = *reinterpret_cast<const f8_i32x4 *>(b + j * 2048 + (x0 ^ (64 * s)));
#pragma unroll
            for (int i = 0; i < FM; ++i)
                x.a[i].v[s] = *reinterpret_cast<const f8_i32x4 *>(a + i * 2048 + (x0 ^ (64 * s)));
        }
    };
    auto step = [&](const Set &x, Set &next, int kb) {
        f8_wait_barrier<(S - 2) * LOADS>();  // this stage is read, and stage kb+1 has landed
        poison_lds(in.stage(kb), P::STAGE);
        if (kb + 2 == in.nk && in.tail % 16)
            in.mask_tail();
        read(next, kb + 1);
        __builtin_amdgcn_sched_barrier(0);
        constexpr int NP = 2 * FM * FN, PER = (LOADS + NP - 1) / NP;
#pragma unroll
        for (int e = 0; e < NP; ++e) {
            const int s = e / (FM * FN), i = e / FN % FM, j = e % FN;
            acc[i][j] = i8_mma(x.b[j].v[s], x.a[i].v[s], acc[i][j]);
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
    int *buf = reinterpret_cast<int *>(smem) + w * G::OUT;
#pragma unroll
    for (int i = 0; i < FM; ++i)
        i8_store_rows<FM, FN>(g, buf, m0 + wm * G::WM + 16 * i, n0 + wn * G::WN, i, acc[i], scales,
                                  g.ws ? g.ws + (int64_t)split * g.M * g.N : nullptr);
}

}  // namespace
}  // namespace sgemm
