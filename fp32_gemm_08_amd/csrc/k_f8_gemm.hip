// 8-bit block-scaled product C = alpha * A * B^T + beta * C on the matrix
// cores, which add up one k-block of 128 products; the FP32 factor sA*sB of
// that k-block scales the sum, and a second FP32 sum runs over the k-blocks:
//
//   C[m][n] = alpha * sum_b sA[b][m] * sB[b][n] * (sum_{k in b} qA[m][k] * qB[n][k])
//
// A 16-bit C is computed by v_mfma_f32_16x16x128_f8f6f4.  That instruction
// adds products in groups of 8, each group aligned to its largest product with
// 13 bits kept below it (measured: 2^16 + 8 keeps the 8, 2^16 + 7 loses the 7;
// on normally distributed operands the sum of 128 is off by 1.5e-5 of its
// size), far below a 16-bit C's half step of 2^-9 or 2^-12, at twice the rate
// of the 16-bit instructions.  An FP32 C is meant to hold more than that (a
// gradient that is accumulated over many calls): its 8-bit operands are turned
// into bf16, which holds every e4m3 and e5m2 value, and go through
// v_mfma_f32_16x16x32_bf16, whose sums are FP32 (1e-8 on the same operands).
//
// The instructions take rows of B as their first operand and rows of A as their
// second, so that lane l holds C[m = l % 16][n = 4*(l/16) .. +3]: four
// consecutive columns of one row, one store, and one factor where a k-block's
// B scale is the same for 128 columns.  Lane l supplies 32 values of row
// l % 16 of each operand, the 16-byte chunks l/16 and 4 + l/16 of its 128
// (which 32 is free as long as both operands agree: the sum runs over all).
#include "f8_mma.h"

namespace sgemm {
namespace {

typedef __attribute__((address_space(3))) void f8_lds;

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
template <int FN>
__device__ __forceinline__ void store_rows(const F8GemmArgs &g, float *buf, int m, int n, const f8_f32x4 (&acc)[FN])
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
        if (g.c_type == SGEMM_TYPE_F32)
            put8<float>(g, m + r, n + c, v);
        else if (g.c_type == SGEMM_TYPE_BF16)
            put8<__bf16>(g, m + r, n + c, v);
        else
            put8<_Float16>(g, m + r, n + c, v);
    }
}

// ------------------------------------------------------------- tiles

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

// Simple form: stage a k-block through registers, multiply it, repeat.
template <class G, int FA, int FB, bool ROWB, bool ALIGNED, bool EXACT>
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

    const int nkb = (int)(((int64_t)g.K + 127) / 128);
    for (int kb = 0; kb < nkb; ++kb) {
        poison_lds(smem, G::STAGE);
        // rows 0 .. BM-1 of a stage are A's, the others B's; rows past the
        // matrix repeat its last one (their results are not stored)
        for (int e = threadIdx.x; e < G::ROWS * 8; e += G::NT) {
            const int r = e >> 3, c = e & 7;
            const int64_t k = (int64_t)kb * 128 + 16 * c;
            const int valid = (int)min<int64_t>(g.K - k, 16);
            const uint8_t *p = r < G::BM ? g.A + (int64_t)min(m0 + r, g.M - 1) * g.lda + k
                                         : g.B + (int64_t)min(n0 + r - G::BM, g.N - 1) * g.ldb + k;
            const f8_i32x4 x = ALIGNED ? load16_aligned(p, valid) : load16_any(p, valid);
            *reinterpret_cast<f8_i32x4 *>(smem + r * 128 + 16 * (c ^ f8_swz(r))) = x;
        }
        for (int r = threadIdx.x; r < G::BM + (ROWB ? G::BN : 0); r += G::NT)
            sc[r] = r < G::BM ? g.SA[kb * g.ldsa + min(m0 + r, g.M - 1)]
                              : g.SB[kb * g.ldsb + min(n0 + r - G::BM, g.N - 1)];
        __syncthreads();
        const float sb = ROWB ? 0.0f : g.SB[(int64_t)(min(n0 + wn * G::WN, g.N - 1) / 128) * g.ldsb + kb];
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

// Pipelined form, for operands whose rows start on 16-byte boundaries: S stages
// rotate, filled by direct global -> LDS loads.
template <class G, int S_, bool ROWB>
struct F8Pipe {
    static constexpr int S = S_;
    static constexpr int SCALES = G::BM + (ROWB ? G::BN : 64);  // floats of a stage
    static constexpr int NSC = SCALES / 64;                     // loads that fetch them
    static constexpr int STAGE = G::ROWS * 128 + SCALES * 4;
    static constexpr int LOADS = G::LOADS + 1;                  // per wavefront and stage
    static_assert(NSC <= G::NW && SCALES % 64 == 0, "one scale load per wavefront fetches all");
    static_assert(G::LOADS < (G::FM - 1) * G::FN, "a step's loads come before its last row");
    static_assert(S * STAGE <= 160 * 1024 && (S - 2) * LOADS <= 63, "LDS size, vmcnt range");
};

// Direct global -> LDS loads of 16 (or 4) bytes per lane from `base` + the lane's
// offset, lane i landing at byte 16 * i (or 4 * i).  They are buffer loads: the
// base stays in scalar registers, and offsets from `bytes` on deliver zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t f8_rsrc(const void *base, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, bytes, 0x00020000);
}
__device__ __forceinline__ void f8_load_lds16(const void *base, uint32_t bytes, uint32_t off, uint8_t *lds)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(f8_rsrc(base, bytes), (f8_lds *)lds, 16, off, 0, 0, 0);
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

// What a wavefront loads of each stage.
template <class G, int S, bool ROWB>
struct F8Stages {
    typedef F8Pipe<G, S, ROWB> P;
    uint8_t *smem;
    // Operand rows: load j has the 8 rows from 8 * (w * LOADS + j) of the stage on,
    // lane l row l/8, chunk (l % 8) ^ swizzle of that row.  The base of the 8 rows is
    // uniform and the swizzle repeats every 16 rows, so the lane's offset is one of
    // two.  Rows past the matrix and chunks past K deliver zeros by the range check
    // (rows are 128 bytes or more apart, and 8 of them lie within 2^32 bytes: the
    // caller's conditions).
    const uint8_t *base[G::LOADS];
    uint32_t bytes[G::LOADS];
    uint32_t off[2];
    bool past[2];                   // the lane's chunk is past K in the last stage
    // This lane's scale: those of A's rows in the order (row % 16, row / 16) of a
    // wavefront's rows, so that a lane reads its own together; those of B's
    // columns in order, or of each fourth column.
    const float *sbase;
    int64_t sstep;
    uint32_t soff, sblock;
    int nk, tail;                   // stages, values of the last stage's rows

    __device__ __forceinline__ F8Stages(const F8GemmArgs &g, uint8_t *lds, int m0, int n0, int w) : smem(lds)
    {
        const int lane = threadIdx.x & 63;
        nk = (int)(((int64_t)g.K + 127) / 128);
        tail = g.K - (nk - 1) * 128;
#pragma unroll
        for (int j = 0; j < G::LOADS; ++j) {
            const int r = 8 * (w * G::LOADS + j);
            const bool in_a = r < G::BM;
            const int row = in_a ? m0 + r : n0 + r - G::BM, left = (in_a ? g.M : g.N) - row;
            const int64_t ld = in_a ? g.lda : g.ldb;
            base[j] = f8_pick(in_a, g.A, g.B) + (left > 0 ? row * ld : 0);
            bytes[j] = left >= 8 ? F8_ALL : left > 0 ? (uint32_t)(left * ld) : 0;
        }
        // a wavefront's loads of both operands (LOADS of 6) would need two offsets each
        static_assert(G::BM / 8 % G::LOADS == 0, "a wavefront's rows are of one operand");
        const int64_t ld = 8 * w * G::LOADS < G::BM ? g.lda : g.ldb;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int c = (lane & 7) ^ f8_swz(8 * (w * G::LOADS + x) + lane / 8);
            off[x] = (uint32_t)(lane / 8) * (uint32_t)ld + 16 * c;
            past[x] = 16 * c >= tail;
        }
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
    }
    __device__ __forceinline__ uint8_t *stage(int kb) const { return smem + (kb % S) * P::STAGE; }
    // Load j of stage kb (j = LOADS: its scales).  Stages past the last deliver
    // zeros, so that every step makes the same loads.
    __device__ __forceinline__ void fetch(int kb, int w, int j) const
    {
        if (j == G::LOADS)
            f8_load_lds4(sbase + kb * sstep, kb < nk ? F8_ALL : 0, soff, stage(kb) + G::ROWS * 128 + 256 * sblock);
        else
            f8_load_lds16(base[j] + (int64_t)kb * 128, kb < nk ? bytes[j] : 0,
                          kb == nk - 1 && past[j % 2] ? F8_PAST : off[j % 2], stage(kb) + (w * G::LOADS + j) * 1024);
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
    typedef F8Pipe<G, S, ROWB> P;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[S * P::STAGE];
    int tm, tn;
    f8_map_tile(blockIdx.x, g.tiles_m, g.tiles_n, tm, tn);
    const int m0 = tm * G::BM, n0 = tn * G::BN;
    const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = w / G::WGN, wn = w % G::WGN;
    const F8Stages<G, S, ROWB> in(g, smem, m0, n0, w);

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

    for (int st = 0; st < S - 1; ++st) {
        poison_lds(in.stage(st), P::STAGE);
#pragma unroll
        for (int j = 0; j <= G::LOADS; ++j)
            in.fetch(st, w, j);
    }
    f8_wait_barrier<(S - 2) * P::LOADS>();
#pragma unroll
    for (int j = 0; j < G::FN - 1; ++j)
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
        const float *sca = reinterpret_cast<const float *>(st + G::ROWS * 128) + wm * G::WM + l16 * G::FM;
        const float *scb = reinterpret_cast<const float *>(st + G::ROWS * 128) + G::BM +
                           (ROWB ? wn * G::WN + 4 * q : wn * G::WN / 4);
        poison_lds(in.stage(kb + S - 1), P::STAGE);
        // 16 x 16 block e = i * FN + j: its products while block e - LAG is scaled and
        // added (the wait for a product is then covered by the work between).  What the
        // next row needs is read right after a row's first product: the wait that comes
        // before each row then finds reads that are a row old.  The bf16 form has no
        // registers to spare: it reads the scales block by block, and converts the next
        // B fragments one by one when the last row is done with them.
        constexpr int NB = G::FM * G::FN, LAG = EXACT ? 1 : 3, EARLY = G::FN - 1;
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
                if (EARLY + e <= G::LOADS)
                    in.fetch(kb + S - 1, w, EARLY + e);
                if (j > 0 && i + 1 == G::FM)
                    in.fetch(kb + S, w, j - 1);
                if (j == 0 && i + 1 == G::FM) {
                    f8_wait_barrier<(S - 2) * P::LOADS>();  // stage kb+1 has landed
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
        store_rows<G::FN>(g, buf, m0 + wm * G::WM + 16 * i, n0 + wn * G::WN, acc[i]);
}

template <typename T>
__global__ __launch_bounds__(256) void f8_scale_kernel(T *C, int64_t ldc, int cols, float beta)
{
    const int64_t row = blockIdx.x;
    for (int64_t c = threadIdx.x; c < cols; c += 256)
        C[row * ldc + c] = (T)(beta != 0.0f ? beta * (float)C[row * ldc + c] : 0.0f);
}

typedef F8Geo<64, 64, 2, 2> GS;
typedef F8Geo<128, 128, 2, 2> GM;
typedef F8Geo<256, 256, 2, 4> GL;

template <class G>
void launch_tile(const F8GemmArgs &a, int fa, int fb, bool row_b, bool aligned, hipStream_t s)
{
    const dim3 grid((unsigned)(a.tiles_m * a.tiles_n)), block(G::NT);
    on_format(fa, [&](auto FA) { on_format(fb, [&](auto FB) { on_bool(row_b, [&](auto ROWB) {
        on_bool(aligned, [&](auto AL) { on_bool(a.c_type == SGEMM_TYPE_F32, [&](auto EX) {
            f8_tile_kernel<G, FA(), FB(), ROWB(), AL(), EX()><<<grid, block, 0, s>>>(a);
        }); }); }); }); });
}

template <class G, int S>
void launch_pipe(const F8GemmArgs &a, int fa, int fb, bool row_b, hipStream_t s)
{
    const dim3 grid((unsigned)(a.tiles_m * a.tiles_n)), block(G::NT);
    on_format(fa, [&](auto FA) { on_format(fb, [&](auto FB) { on_bool(row_b, [&](auto ROWB) {
        on_bool(a.c_type == SGEMM_TYPE_F32, [&](auto EX) {
            f8_pipe_kernel<G, S, FA(), FB(), ROWB(), EX()><<<grid, block, 0, s>>>(a);
        }); }); }); });
}

}  // namespace

F8GemmPlan f8_gemm_plan(bool row_b, int64_t M, int64_t N, int64_t K, bool aligned)
{
    (void)K;
    F8GemmPlan p;
    int64_t bm = GS::BM, bn = GS::BN;
    p.kid = KID_F8_S;
    if (aligned && M <= 64) {
        p.kid = KID_F8_SKINNY;
        bm = 64, bn = f8_skinny_cols(row_b, N);
    } else if (aligned && M * N >= (int64_t)256 * 256 * 128) {
        p.kid = KID_F8_L;
        bm = GL::BM, bn = GL::BN;
    } else if (aligned && M > 64 && N > 64) {
        p.kid = KID_F8_M;
        bm = GM::BM, bn = GM::BN;
    }
    p.tiles_m = (M + bm - 1) / bm;
    p.tiles_n = (N + bn - 1) / bn;
    return p;
}

hipError_t launch_f8_gemm(F8GemmArgs a, const F8GemmPlan &p, int format_a, int format_b, bool row_b, bool aligned,
                          hipStream_t s)
{
    a.tiles_m = (int)p.tiles_m;
    a.tiles_n = (int)p.tiles_n;
    if (p.kid == KID_F8_SKINNY)
        return launch_f8_skinny(a, format_a, format_b, row_b, s);
    if (p.kid == KID_F8_L)
        launch_pipe<GL, 2>(a, format_a, format_b, row_b, s);
    else if (p.kid == KID_F8_M)
        launch_pipe<GM, 4>(a, format_a, format_b, row_b, s);
    else
        launch_tile<GS>(a, format_a, format_b, row_b, aligned, s);
    return hipGetLastError();
}

hipError_t launch_f8_scale(void *C, int64_t ldc, int rows, int cols, int c_type, float beta, hipStream_t s)
{
    if (c_type == SGEMM_TYPE_F32)
        f8_scale_kernel<<<(unsigned)rows, 256, 0, s>>>(static_cast<float *>(C), ldc, cols, beta);
    else if (c_type == SGEMM_TYPE_FP16)
        f8_scale_kernel<<<(unsigned)rows, 256, 0, s>>>(static_cast<_Float16 *>(C), ldc, cols, beta);
    else
        f8_scale_kernel<<<(unsigned)rows, 256, 0, s>>>(static_cast<__bf16 *>(C), ldc, cols, beta);
    return hipGetLastError();
}

}  // namespace sgemm
