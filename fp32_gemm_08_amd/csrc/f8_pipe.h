// The pipelined 8-bit products, for operands whose rows start on 16-byte boundaries:
// tiles of every size are instances of one kernel.
#pragma once
#include "f8_tile.h"

namespace sgemm {
namespace {

typedef __attribute__((address_space(3))) void f8_lds;

// S stages rotate, filled by direct global -> LDS loads.
template <class G, int S_, bool ROWB, bool LATE>
struct F8Pipe {
    static constexpr int S = S_;
    static constexpr int SCALES = G::BM + (ROWB ? G::BN : 64);  // floats of a stage
    static constexpr int NSC = SCALES / 64;                     // loads that fetch them
    static constexpr int STAGE = G::ROWS * 128;                 // bytes of a stage's rows
    // LATE: scales are read in a stage's last row, where the place of the stage is given
    // to the one S ahead already: they have twice the places.
    static constexpr int SLOTS = LATE ? 2 * S : S;
    static constexpr int BYTES = S * STAGE + SLOTS * SCALES * 4;
    static constexpr int LOADS = G::LOADS + 1;                  // per wavefront and stage
    static_assert(NSC <= G::NW && SCALES % 64 == 0, "one scale load per wavefront fetches all");
    // a step's loads: EARLY under the last products of the step before, PER under each
    // of its own products before the last row
    static constexpr int EARLY = G::FN - 1, FREE = (G::FM - 1) * G::FN;
    static constexpr int PER = (LOADS - EARLY + FREE - 1) / FREE;
    static_assert(EARLY <= LOADS, "fewer loads than places");
    static_assert(BYTES <= 160 * 1024 && (S - 2) * LOADS <= 63, "LDS size, vmcnt range");
};

// Direct global -> LDS loads of 16 (or 4) bytes per lane from `base` + the lane's
// offset, lane i landing at byte 16 * i (or 4 * i).  They are buffer loads: the
// base stays in scalar registers, and offsets from `bytes` on deliver zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t f8_rsrc(const void *base, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, bytes, 0x00020000);
}
__device__ __forceinline__ void f8_load_lds16(__amdgpu_buffer_rsrc_t rsrc, uint32_t off, uint32_t k, uint8_t *lds)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (f8_lds *)lds, 16, off, k, 0, 0);
}
__device__ __forceinline__ void f8_load_lds4(const void *base, uint32_t bytes, uint32_t off, uint8_t *lds)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(f8_rsrc(base, bytes), (f8_lds *)lds, 4, off, 0, 0, 0);
}
// The range check takes each 4 bytes by their own offset against the count of
// bytes, so the offset that is meant to be out of range starts at that count.
constexpr uint32_t F8_ALL = 0xfffffff0u;
constexpr uint32_t F8_PAST = F8_ALL;

// Wait until at most N of this wavefront's direct loads are outstanding and
// its LDS accesses are done, then meet the others (gfx9 encoding: vmcnt bits
// 3:0 and 15:14, expcnt 6:4 left at 7, lgkmcnt 11:8 = 0).
template <int N>
__device__ __forceinline__ void f8_wait_barrier()
{
    static_assert(N >= 0 && N <= 63, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 0xF) | (0x7 << 4) | ((N >> 4) << 14));
    asm volatile("s_barrier" ::: "memory");
}

// What a wavefront loads of each stage.  SCALED: the stages have scales; without, Args are
// another family's with the same operands.
template <class G, int S, bool ROWB, bool LATE, bool SCALED = true>
struct F8Stages {
    typedef F8Pipe<G, S, ROWB, LATE> P;
    uint8_t *smem;
    // Operand rows: load j has the 8 rows from 8 * (w * LOADS + j) of the stage on,
    // lane l row l/8, chunk (l % 8) ^ swizzle of that row (which repeats every 16 rows).
    // Rows past the matrix and chunks past K deliver zeros by the range check: the row
    // after the last one starts at `bytes` (several rows lie at least K apart, and 256
    // of them within 2^32 bytes: the caller's conditions).  With FEW loads a wavefront
    // keeps an offset of each in the operand's tile, and k goes along beside it; with
    // more, which are too many registers, the 8 rows' base is moved in scalars and the
    // offset is one of two.
    static constexpr bool FEW = G::LOADS <= 4;
    static constexpr bool MIXED = G::BM / 8 % G::LOADS != 0;    // a wavefront loads of both operands
    static constexpr int BASES = FEW ? 1 + MIXED : G::LOADS;
    const uint8_t *base[BASES];
    uint32_t bytes[BASES];
    uint32_t off[FEW ? G::LOADS : 2];
    bool past[2];                   // the lane's chunk is past K in the last stage
    // This lane's scale: those of A's rows in the order (row % 16, row / 16) of a
    // wavefront's rows, so that a lane reads its own together; those of B's
    // columns in order, or of each fourth column.
    const float *sbase;
    int64_t sstep;
    uint32_t soff, sblock;
    int nk, tail;                   // stages, values of the last stage's rows

    template <class Args>
    __device__ __forceinline__ F8Stages(const Args &g, uint8_t *lds, int m0, int n0, int w, int split)
        : smem(lds)
    {
        const int lane = threadIdx.x & 63;
        const int all = (int)(((int64_t)g.K + 127) / 128), first = split * g.kb_split;
        nk = min(all - first, g.kb_split);
        tail = first + nk == all ? g.K - (all - 1) * 128 : 128;
        static_assert(FEW || !MIXED, "offsets of one operand");
#pragma unroll
        for (int x = 0; x < BASES; ++x) {
            const int r = FEW ? 0 : 8 * (w * G::LOADS + x) % G::BM;   // (its operand's tile has BM rows, or FEW)
            const bool in_a = FEW ? x == 0 && (MIXED || 8 * w * G::LOADS < G::BM) : 8 * (w * G::LOADS + x) < G::BM;
            const int row = (in_a ? m0 : n0) + r, left = (in_a ? g.M : g.N) - row;
            const int64_t ld = in_a ? g.lda : g.ldb;
            base[x] = f8_pick(in_a, g.A, g.B) + (left > 0 ? row * ld : 0) + (int64_t)first * 128;
            bytes[x] = left >= (FEW ? in_a ? G::BM : G::BN : 8) ? F8_ALL : left > 0 ? (uint32_t)(left * ld) : 0;
        }
        static_assert(FEW || G::BM == G::BN, "rows of a load in their operand's tile");
#pragma unroll
        for (int j = 0; j < (FEW ? G::LOADS : 2); ++j) {
            const int r = 8 * (w * G::LOADS + j) + lane / 8;
            const bool in_a = 8 * (w * G::LOADS + j) < G::BM;
            off[j] = (uint32_t)(!FEW ? lane / 8 : in_a ? r : r - G::BM) * (uint32_t)f8_pick(in_a, g.lda, g.ldb) +
                     16 * ((lane & 7) ^ f8_swz(r));
        }
#pragma unroll
        for (int x = 0; x < 2; ++x)
            past[x] = 16 * ((lane & 7) ^ f8_swz(8 * (w * G::LOADS + x) + lane / 8)) >= tail;
        if constexpr (SCALED) {
            sblock = w % P::NSC;
            const int si = 64 * sblock + lane;
            if (64 * (int)sblock < G::BM) {
                sbase = g.SA + m0;
                sstep = g.ldsa;
                soff = 4u * (uint32_t)min(si / G::WM * G::WM + 16 * (si % G::FM) + si % G::WM / G::FM, g.M - 1 - m0);
            } else if constexpr (ROWB) {
                sbase = g.SB + n0;
                sstep = g.ldsb;
                soff = 4u * (uint32_t)min(si - G::BM, g.N - 1 - n0);
            } else {
                sbase = g.SB + (int64_t)(n0 / 128) * g.ldsb;
                sstep = 1;
                soff = 4u * (uint32_t)(min(n0 + 4 * (si - G::BM), g.N - 1) / 128 - n0 / 128) * (uint32_t)g.ldsb;
            }
            sbase += first * sstep;
        }
    }
    __device__ __forceinline__ uint8_t *stage(int kb) const { return smem + (kb % S) * P::STAGE; }
    __device__ __forceinline__ uint8_t *scales(int kb) const
    {
        return smem + S * P::STAGE + (kb % P::SLOTS) * (P::SCALES * 4);
    }
    // Load j of stage kb (j = LOADS: its scales).  Stages past the last deliver
    // zeros, so that every step makes the same loads.
    __device__ __forceinline__ void fetch(int kb, int w, int j) const
    {
        if (SCALED && j == G::LOADS)
            f8_load_lds4(sbase + kb * sstep, kb < nk ? F8_ALL : 0, soff, scales(kb) + 256 * sblock);
        else {
            const bool second = FEW && MIXED && 8 * (w * G::LOADS + j) >= G::BM;
            const int x = FEW ? 0 : j, y = BASES > 1 && FEW ? 1 : x;
            const uint8_t *p = f8_pick(second, base[y], base[x]);
            const uint32_t n = f8_pick(second, bytes[y], bytes[x]);
            f8_load_lds16(f8_rsrc(FEW ? p : p + (int64_t)kb * 128, kb < nk ? n : 0),
                          kb == nk - 1 && past[j % 2] ? F8_PAST : off[FEW ? j : j % 2], FEW && kb < nk ? kb * 128 : 0,
                          stage(kb) + (w * G::LOADS + j) * 1024);
        }
    }
    // The bytes past K of the chunk that holds the last values of a row: zeros.
    __device__ __forceinline__ void mask_tail() const
    {
        for (int r = threadIdx.x; r < G::ROWS; r += G::NT) {
            f8_i32x4 *p = reinterpret_cast<f8_i32x4 *>(stage(nk - 1) + r * 128 + 16 * ((tail / 16) ^ f8_swz(r)));
            *p = keep16(*p, tail % 16);
        }
        __syncthreads();
    }
};

// Pipeline.  At the start of a step the fragments of the B rows and of the first A
// rows are in registers.  Each row of blocks reads the next A rows under its
// products.  In the last row every wavefront has read all of this stage: there the
// wavefronts meet, the stage S ahead is requested into its place, a load per
// product (EARLY of them there and the others under the next step's first rows;
// all of them under those 470 against 452 us at 8192^3, three per product 467), and
// the next stage's fragments are read under the last row's products.
template <class G, int S, int FA, int FB, bool ROWB, bool EXACT>
__global__ __launch_bounds__(G::NT) void f8_pipe_kernel(F8GemmArgs g)
{
    typedef F8Pipe<G, S, ROWB, EXACT> P;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[P::BYTES];
    int tm, tn;
    const int tiles = g.tiles_m * g.tiles_n, split = blockIdx.x / tiles;
    f8_map_tile(blockIdx.x % tiles, g.tiles_m, g.tiles_n, tm, tn);
    const int m0 = tm * G::BM, n0 = tn * G::BN;
    const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = w / G::WGN, wn = w % G::WGN;
    const F8Stages<G, S, ROWB, EXACT> in(g, smem, m0, n0, w, split);

    f8_f32x4 acc[G::FM][G::FN];
#pragma unroll
    for (int i = 0; i < G::FM; ++i)
#pragma unroll
        for (int j = 0; j < G::FN; ++j)
            acc[i][j] = f8_f32x4{};

    // Where this lane's two chunks of row l16 of a block of 16 rows lie, and of
    // row 16i + l16 of its wavefront's rows from `first` on.
    const uint32_t lo = l16 * 128 + 16 * (q ^ f8_swz(l16)), hi = lo ^ 64;
    const uint32_t at_a = wm * G::WM * 128, at_b = (G::BM + wn * G::WN) * 128;
    auto read = [&](const uint8_t *st, uint32_t first, int i) {
        return f8_join(*reinterpret_cast<const f8_i32x4 *>(st + first + lo + i * 2048),
                       *reinterpret_cast<const f8_i32x4 *>(st + first + hi + i * 2048));
    };

    poison_lds(smem, P::BYTES);
    for (int st = 0; st < S - 1; ++st) {
#pragma unroll
        for (int j = 0; j <= G::LOADS; ++j)
            in.fetch(st, w, j);
    }
    f8_wait_barrier<(S - 2) * P::LOADS>();
#pragma unroll
    for (int j = 0; j < P::EARLY; ++j)
        in.fetch(S - 1, w, j);
    if (in.nk == 1 && in.tail % 16)
        in.mask_tail();
    Frag<FB, EXACT> fb[G::FN];
#pragma unroll
    for (int j = 0; j < G::FN; ++j)
        fb[j].set(read(smem, at_b, j));
    f8_i32x8 ra[2];                              // the next rows of A
    ra[0] = read(smem, at_a, 0);
    for (int kb = 0; kb < in.nk; ++kb) {
        const uint8_t *st = in.stage(kb), *next = in.stage(kb + 1);
        const float *sca = reinterpret_cast<const float *>(in.scales(kb)) + wm * G::WM + l16 * G::FM;
        const float *scb = reinterpret_cast<const float *>(in.scales(kb)) + G::BM +
                           (ROWB ? wn * G::WN + 4 * q : wn * G::WN / 4);
        // 16 x 16 block e = i * FN + j: its products while block e - LAG is scaled and
        // added (the wait for a product is then covered by the work between).  What the
        // next row needs is read right after a row's first product: the wait that comes
        // before each row then finds reads that are a row old.  The bf16 form has no
        // registers to spare: it reads the scales block by block, and converts the next
        // B fragments one by one when the last row is done with them.
        constexpr int NB = G::FM * G::FN, LAG = EXACT ? 1 : 3;
        float sa[EXACT ? 2 : G::FM], sb = 1.0f;
        f8_f32x4 sbv[EXACT ? 2 : ROWB ? G::FN : 1];
        f8_f32x4 t[LAG + 1];
        Frag<FA, EXACT> fa;
        f8_i32x8 rb;
#pragma unroll
        for (int e = 0; e < NB + LAG; ++e) {
            const int i = e / G::FN, j = e % G::FN;
            if (e < NB) {
                if (j == 0)
                    fa.set(ra[EXACT ? 0 : i & 1]);
                f8_f32x4 &u = t[e % (LAG + 1)];
                if constexpr (EXACT) {
                    __builtin_amdgcn_sched_barrier(0);
                    u = f8_mma_part<0>(fb[j], fa, f8_f32x4{});
                } else {
                    u = f8_mma<FA, FB>(fb[j], fa);
                }
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (EXACT) {
                    if (j == 0)
                        sa[i & 1] = sca[i];
                    if (ROWB)
                        sbv[e & 1] = *reinterpret_cast<const f8_f32x4 *>(scb + 16 * j);
                    else if (e == 0)
                        sb = scb[0];
                } else if (e == 0) {
#pragma unroll
                    for (int x = 0; x < G::FM; ++x)
                        sa[x] = sca[x];
                    if constexpr (ROWB) {
#pragma unroll
                        for (int x = 0; x < G::FN; ++x)
                            sbv[x] = *reinterpret_cast<const f8_f32x4 *>(scb + 16 * x);
                    } else {
                        sb = scb[0];
                    }
                }
                if (j == 0 && i + 1 < G::FM)
                    ra[EXACT ? 0 : (i + 1) & 1] = read(st, at_a, i + 1);
                if (i + 1 < G::FM) {
#pragma unroll
                    for (int x = P::EARLY + e * P::PER; x < P::EARLY + (e + 1) * P::PER && x <= G::LOADS; ++x)
                        in.fetch(kb + S - 1, w, x);
                } else if (j > 0) {
                    in.fetch(kb + S, w, j - 1);
                }
                if (j == 0 && i + 1 == G::FM) {
                    f8_wait_barrier<(S - 2) * P::LOADS>();  // stage kb+1 has landed
                    poison_lds(in.stage(kb + S), P::STAGE);
                    if (kb + 2 == in.nk && in.tail % 16)
                        in.mask_tail();
                    if (EXACT)
                        rb = read(next, at_b, 0);
                    ra[0] = read(next, at_a, 0);
                }
                if (!EXACT && i + 1 == G::FM)
                    fb[j].set(read(next, at_b, j));
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (EXACT) {
                    u = f8_mma_part<1>(fb[j], fa, u);
                    u = f8_mma_part<2>(fb[j], fa, u);
                    u = f8_mma_part<3>(fb[j], fa, u);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            if (e >= LAG) {
                const int pe = e - LAG, pi = pe / G::FN, pj = pe % G::FN;
                const f8_f32x4 &u = t[pe % (LAG + 1)];
                float &a = sa[EXACT ? pi & 1 : pi];
                if (!ROWB && pj == 0)
                    a *= sb;
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    acc[pi][pj][x] = fmaf(u[x], ROWB ? a * sbv[EXACT ? pe & 1 : ROWB ? pj : 0][x] : a, acc[pi][pj][x]);
                // the additions stay here: the compiler would sink them below the
                // branch of the last row, and keep all products in registers till then
                asm volatile("" : "+v"(acc[pi][pj]));
            }
            __builtin_amdgcn_sched_barrier(0);
            if (EXACT && e < NB && i + 1 == G::FM) {
                fb[j].set(rb);
                if (j + 1 < G::FN)
                    rb = read(next, at_b, j + 1);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
    // the stages requested past the last one land before the LDS is used again
    f8_wait_barrier<0>();
    float *buf = reinterpret_cast<float *>(smem) + w * G::OUT;
#pragma unroll
    for (int i = 0; i < G::FM; ++i)
        store_rows<G::FN>(g, buf, m0 + wm * G::WM + 16 * i, n0 + wn * G::WN, acc[i],
                          g.ws ? g.ws + (int64_t)split * g.M * g.N : nullptr);
}

// The same for tiles of few blocks a wavefront, one workgroup to a CU: a step's work
// is then shorter than the way of one fragment from the LDS, so all fragments and
// scales of the next stage are read before this stage's products, into a second set
// of registers.  The wavefronts meet once a step, when each has its set: the stage S
// ahead is requested into the place of the one in the registers.
template <class G, int S, int FA, int FB, bool ROWB, bool EXACT>
__global__ __launch_bounds__(G::NT) void f8_flat_kernel(F8GemmArgs g)
{
    typedef F8Pipe<G, S, ROWB, false> P;
    static_assert((S - 1) * P::LOADS <= 63, "vmcnt range");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[P::BYTES];
    int tm, tn;
    const int tiles = g.tiles_m * g.tiles_n, split = blockIdx.x / tiles;
    f8_map_tile(blockIdx.x % tiles, g.tiles_m, g.tiles_n, tm, tn);
    const int m0 = tm * G::BM, n0 = tn * G::BN;
    const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = w / G::WGN, wn = w % G::WGN;
    const F8Stages<G, S, ROWB, false> in(g, smem, m0, n0, w, split);

    f8_f32x4 acc[G::FM][G::FN];
#pragma unroll
    for (int i = 0; i < G::FM; ++i)
#pragma unroll
        for (int j = 0; j < G::FN; ++j)
            acc[i][j] = f8_f32x4{};

    const uint32_t lo = l16 * 128 + 16 * (q ^ f8_swz(l16)), hi = lo ^ 64;
    struct Set {
        f8_i32x8 a[G::FM], b[G::FN];
        float sa[G::FM], sb;
        f8_f32x4 sbv[ROWB ? G::FN : 1];
    } set[2];
    auto read = [&](Set &x, int kb) {
        const uint8_t *st = in.stage(kb);
        const uint8_t *a = st + wm * G::WM * 128, *b = st + (G::BM + wn * G::WN) * 128;
#pragma unroll
        for (int j = 0; j < G::FN; ++j)
            x.b[j] = f8_join(*reinterpret_cast<const f8_i32x4 *>(b + lo + j * 2048),
                             *reinterpret_cast<const f8_i32x4 *>(b + hi + j * 2048));
#pragma unroll
        for (int i = 0; i < G::FM; ++i)
            x.a[i] = f8_join(*reinterpret_cast<const f8_i32x4 *>(a + lo + i * 2048),
                             *reinterpret_cast<const f8_i32x4 *>(a + hi + i * 2048));
        const float *sc = reinterpret_cast<const float *>(in.scales(kb));
#pragma unroll
        for (int i = 0; i < G::FM; ++i)
            x.sa[i] = sc[wm * G::WM + l16 * G::FM + i];
        if constexpr (ROWB) {
#pragma unroll
            for (int j = 0; j < G::FN; ++j)
                x.sbv[j] = *reinterpret_cast<const f8_f32x4 *>(sc + G::BM + wn * G::WN + 16 * j + 4 * q);
        } else {
            x.sb = sc[G::BM + wn * G::WN / 4];
        }
    };
    auto step = [&](const Set &x, Set &next, int kb) {
        f8_wait_barrier<(S - 2) * P::LOADS>();  // this stage is read, and stage kb+1 has landed
        poison_lds(in.stage(kb), P::STAGE);
        if (kb + 2 == in.nk && in.tail % 16)
            in.mask_tail();
        read(next, kb + 1);
        __builtin_amdgcn_sched_barrier(0);
        Frag<FB, EXACT> fb[G::FN];
        Frag<FA, EXACT> fa;
#pragma unroll
        for (int j = 0; j < G::FN; ++j)
            fb[j].set(x.b[j]);
        constexpr int NB = G::FM * G::FN, LAG = EXACT ? 1 : NB > 4 ? 3 : 2, PER = (P::LOADS + NB - 1) / NB;
        f8_f32x4 t[LAG + 1];
#pragma unroll
        for (int e = 0; e < NB + LAG; ++e) {
            const int i = e / G::FN, j = e % G::FN;
            if (e < NB) {
                if (j == 0)
                    fa.set(x.a[i]);
                t[e % (LAG + 1)] = f8_mma<FA, FB>(fb[j], fa);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int y = e * PER; y < (e + 1) * PER && y <= G::LOADS; ++y)
                    in.fetch(kb + S, w, y);
                __builtin_amdgcn_sched_barrier(0);
            }
            if (e >= LAG) {
                const int pe = e - LAG, pi = pe / G::FN, pj = pe % G::FN;
                const f8_f32x4 &u = t[pe % (LAG + 1)];
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    acc[pi][pj][y] = fmaf(u[y], x.sa[pi] * (ROWB ? x.sbv[ROWB ? pj : 0][y] : x.sb), acc[pi][pj][y]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    poison_lds(smem, P::BYTES);
    for (int st = 0; st < S; ++st)
#pragma unroll
        for (int j = 0; j <= G::LOADS; ++j)
            in.fetch(st, w, j);
    f8_wait_barrier<(S - 1) * P::LOADS>();
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
    float *buf = reinterpret_cast<float *>(smem) + w * G::OUT;
#pragma unroll
    for (int i = 0; i < G::FM; ++i)
        store_rows<G::FN>(g, buf, m0 + wm * G::WM + 16 * i, n0 + wn * G::WN, acc[i],
                          g.ws ? g.ws + (int64_t)split * g.M * g.N : nullptr);
}

template <class G, int S, bool FLAT>
hipError_t launch_pipe(const F8GemmArgs &a, int splits, int fa, int fb, bool row_b, hipStream_t s)
{
    const dim3 grid((unsigned)(a.tiles_m * a.tiles_n * splits)), block(G::NT);
    on_format(fa, [&](auto FA) { on_format(fb, [&](auto FB) { on_bool(row_b, [&](auto ROWB) {
        on_bool(a.c_type == SGEMM_TYPE_F32, [&](auto EX) {
            if constexpr (FLAT)
                f8_flat_kernel<G, S, FA(), FB(), ROWB(), EX()><<<grid, block, 0, s>>>(a);
            else
                f8_pipe_kernel<G, S, FA(), FB(), ROWB(), EX()><<<grid, block, 0, s>>>(a);
        }); }); }); });
    return hipGetLastError();
}

}  // namespace
}  // namespace sgemm
