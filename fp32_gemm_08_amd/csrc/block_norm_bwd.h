// Backward pass of the norms around a block.  With n = h * rstd, m = o * rstd_post (or o)
// and g = dy * w:
//
//     d = rstd * (g - n * mean(g n)) + dh          dx = alpha * d
//     p = gate * d * w_post                        do = rstd_post * (p - m * mean(p m))
//     dw = sum dy n     t = sum over the rows of a gate of d m
//     dw_post = sum over gates of gate * t         dgate = w_post * t
//
// so one sum t serves both of the last.  A walker (a workgroup, or the 16 to 64 lanes
// that hold a row) takes rows one after another and keeps its columns' sums; a second kernel
// adds what the workgroups left, in a fixed order.
//
// Bound by memory: 16384 x 4096 bf16, h and o in 8 bits, 8 gates 136 to 142 us with the second
// kernel (6.5 us of them), 4.9 TB/s (fp16 145, fp32 229, from bf16 159, a gate for each row
// 290); from 238 with rows taken in runs and their loads not requested ahead.  Rows of 4095 148
// (184 from bf16).  Above 8192 columns the sums of a lane's columns no longer fit its registers:
// 4096 x 16384 267 us, 2048 x 32768, where a row does not either, 1330.  1000 x 1017 fp32 14.0,
// two launches.
#pragma once
#include "norm_internal.h"
#include "norm_rows.h"

namespace sgemm {
namespace {

// Where h and o come from: rows of T, or e4m3 with a scale per block of 128.
template <typename T, bool KEPT> struct Source;
template <typename T> struct Source<T, false> {
    typedef typename Elt<T>::Raw Raw;
    static __device__ __forceinline__ void load(Raw &r, const void *p, int64_t ld, const float *, int64_t, int64_t row,
                                                int c, int cols)
    {
        r = row_raw8<true>(static_cast<const T *>(p) + row * ld, c, cols);
    }
    // (rows of at least 8; fix() before the values are used)
    static __device__ __forceinline__ void load_any(Raw &r, const void *p, int64_t ld, const float *, int64_t, int64_t row,
                                                    int c, int cols)
    {
        r = row_any8<true>(static_cast<const T *>(p) + row * ld, c, cols);
    }
    static __device__ __forceinline__ void fix(Raw &r, int past) { row_fix8<T>(r, past); }
    static __device__ __forceinline__ void values(const Raw &r, float (&v)[8])
    {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = (float)r[j];
    }
};
template <typename T> struct Source<T, true> {
    struct Raw {
        f8_u32x2 q;
        float s;
    };
    static __device__ __forceinline__ void load(Raw &r, const void *p, int64_t ld, const float *S, int64_t lds,
                                                int64_t row, int c, int cols)
    {
        r.q = row_raw8b<true>(static_cast<const uint8_t *>(p) + row * ld, c, cols);
        r.s = c < cols ? S[(int64_t)(c / F8_BLOCK) * lds + row] : 0.0f;
    }
    static __device__ __forceinline__ void load_any(Raw &r, const void *p, int64_t ld, const float *S, int64_t lds,
                                                    int64_t row, int c, int cols)
    {
        r.q = row_any8b<true>(static_cast<const uint8_t *>(p) + row * ld, c, cols);
        r.s = S[(int64_t)(min(c, cols - 1) / F8_BLOCK) * lds + row];
    }
    static __device__ __forceinline__ void fix(Raw &r, int past)
    {
        row_fix8b(r.q, past);
        if (past >= 8)
            r.s = 0.0f;
    }
    static __device__ __forceinline__ void values(const Raw &r, float (&v)[8])
    {
        f8_unpack8<0>(r.q, v);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] *= r.s;
    }
};

// A row's vector of weights, 1 where there is none.
template <typename T>
__device__ __forceinline__ void weights8(const void *W, int64_t at, int w_f32, int c, int cols, float (&v)[8])
{
    if (W) {
        load_w8<T>(static_cast<const uint8_t *>(W) + at * (w_f32 ? 4 : (int)sizeof(T)), w_f32, c, cols, v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = 1.0f;
    }
}

// The rows of a walker.  One gate a walker: `team` workgroups share a gate's rows and take
// them in turn, so that all walkers of a gate are at neighbouring rows at a time (rows in
// runs of a walker's own took 154 where this took 138 us, 16384 x 4096 bf16), and workgroups of
// one XCD at the nearest, since the scales of 32 consecutive rows share a line.  SEVERAL:
// `chunk` consecutive rows.
template <bool SEVERAL, int ROWS> struct BlockNormWalk {
    int group;              // of the workgroup, in the order of the sums
    int gate;               // the first row's
    int64_t walker, first, end;
    int step;
    __device__ __forceinline__ BlockNormWalk(const BlockNormBwdArgs &g, int own)
    {
        const int n = g.groups;
        group = n % 8 == 0 ? (int)(blockIdx.x % 8) * (n / 8) + (int)(blockIdx.x / 8) : (int)blockIdx.x;
        walker = (int64_t)group * ROWS + own;
        if constexpr (SEVERAL) {
            first = walker * g.chunk;
            end = min<int64_t>(g.rows, first + g.chunk);
            step = 1;
            gate = (int)((uint32_t)min<int64_t>(first, g.rows - 1) / (uint32_t)g.gate_rows);
        } else {
            gate = group / g.team;
            const int64_t begin = (int64_t)gate * g.gate_rows;
            first = begin + (int64_t)(group - gate * g.team) * ROWS + own;
            end = min<int64_t>(g.rows, begin + g.gate_rows);
            step = g.team * ROWS;
        }
    }
};

// A workgroup's sums of its columns: of its rows of lanes in order, through `sums`.
template <int NT, int L, int V>
__device__ __forceinline__ void block_norm_put_sums(float *out, float *sums, int lane, int own, int cols,
                                                    const float (*v)[8])
{
    constexpr int ROWS = NT / L;
    if constexpr (ROWS == 1) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (8 * (lane + L * i) < cols)
                row_store8(out, 8 * (lane + L * i), cols, v[i]);
    } else {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                sums[(own * 8 + j) * (V * L) + L * i + lane] = v[i][j];
        __syncthreads();
        for (int c = threadIdx.x; c < cols; c += NT) {
            float s = 0.0f;
#pragma unroll
            for (int r = 0; r < ROWS; ++r)
                s += sums[(r * 8 + c % 8) * (V * L) + c / 8];
            out[c] = s;
        }
    }
}

// What a work-item holds of a row: V pieces of 8 consecutive columns.  With one piece its
// sums of dw and t, w and gate * w_post stay in registers; with more the weights are read
// again for every row, from the L2, and with two the sums are in the LDS (1024 work-items
// have 128 registers each).  AHEAD: the next row's values are requested before this row's
// are used.  SEVERAL: a walker's rows may have several gates; dw_post, which then changes
// once per gate, is kept in the LDS, or (two pieces) in the workgroup's place in the
// workspace, by the work-item that has its columns.
template <typename T, int NT, int L, int V, bool AHEAD, bool KEPT, bool SEVERAL>
__global__ __launch_bounds__(NT) void block_norm_bwd_kernel(BlockNormBwdArgs g)
{
    typedef typename Elt<T>::Raw Raw;
    typedef Source<T, KEPT> Src;
    constexpr int ROWS = NT / L;
    constexpr bool HOLD = V == 1, FAR = V == 2;
    __shared__ float slot[4][NT / 64];
    __shared__ float sums[FAR ? 2 * NT * 8 * V : SEVERAL || ROWS > 1 ? NT * 8 * V : 1];
    const int lane = threadIdx.x % L, own = ROWS == 1 ? 0 : threadIdx.x / L;
    const bool read_o = g.O != nullptr, out_o = g.DO || g.DWP || g.DG;
    const BlockNormWalk<SEVERAL, ROWS> walk(g, own);
    const int64_t walker = walk.walker, r0 = walk.first, r1 = walk.end;
    auto col = [&](int i) { return 8 * (lane + L * i); };
    auto held = [&](int i, int j) -> float & { return sums[(j * V + i) * NT + threadIdx.x]; };
    float *place = g.ws + ((int64_t)g.groups + walk.group) * g.cols;  // (two pieces) of dw_post

    int gr = walk.gate;
    int64_t gate_end = (int64_t)(gr + 1) * g.gate_rows;
    auto gate_weight = [&](int i, float (&v)[8]) {  // gate * w_post
        float wp[8];
        weights8<T>(g.G, gr * g.ldg, g.w_f32, col(i), g.cols, v);
        weights8<T>(g.WP, 0, g.w_f32, col(i), g.cols, wp);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] *= wp[j];
    };
    struct Row {
        Raw dy[V], dh[V];
        typename Src::Raw h[V], o[V];
        float rstd, rstd_post;
    } a, b;
    auto request = [&](int64_t row, Row &to) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = col(i);
            if (g.DY) {
                to.dy[i] = row_raw8<true>(static_cast<const T *>(g.DY) + row * g.lddy, c, g.cols);
                Src::load(to.h[i], g.H, g.ldh, g.SH, g.ldsh, row, c, g.cols);
            }
            if (g.DH)
                to.dh[i] = row_raw8<true>(static_cast<const T *>(g.DH) + row * g.lddh, c, g.cols);
            if (read_o)
                Src::load(to.o[i], g.O, g.ldo, g.SO, g.ldso, row, c, g.cols);
        }
        to.rstd = g.DY ? g.rstd[row] : 0.0f;
        to.rstd_post = g.WP ? g.rstd_post[row] : 1.0f;
    };
    if (AHEAD && r0 < r1)
        request(r0, b);
    float hw[HOLD ? V : 1][8], hgw[HOLD ? V : 1][8], rdw[FAR ? 1 : V][8], rt[FAR ? 1 : V][8];
    auto dw = [&](int i, int j) -> float & { return FAR ? sums[(j * V + i) * NT + threadIdx.x] : rdw[FAR ? 0 : i][j]; };
    auto t = [&](int i, int j) -> float & { return FAR ? sums[((8 + j) * V + i) * NT + threadIdx.x] : rt[FAR ? 0 : i][j]; };
    if constexpr (HOLD) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            weights8<T>(g.W, 0, g.w_f32, col(i), g.cols, hw[i]);
            gate_weight(i, hgw[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            dw(i, j) = t(i, j) = 0.0f;
            if (SEVERAL && !FAR)
                held(i, j) = 0.0f;
        }
        if (SEVERAL && FAR && g.DWP && col(i) < g.cols) {
            const float zero[8] = {};
            row_store8(place, col(i), g.cols, zero);
        }
    }
    int turn = 0;
    for (int64_t row = r0; row < r1; row += walk.step, turn ^= 1) {
        if constexpr (AHEAD) {
            a = b;
            if (row + walk.step < r1)
                request(row + walk.step, b);
        } else {
            request(row, a);
        }
        float mean = 0.0f;
        if (g.DY) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float h[8], w[8];
                Src::values(a.h[i], h);
                if constexpr (!HOLD)
                    weights8<T>(g.W, 0, g.w_f32, col(i), g.cols, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float dy = (float)a.dy[i][j], n = h[j] * a.rstd;
                    sum = fmaf(dy * (HOLD ? hw[HOLD ? i : 0][j] : w[j]), n, sum);
                    dw(i, j) = fmaf(dy, n, dw(i, j));
                }
            }
            mean = row_sum<NT, L>(sum, slot[turn]) / (float)g.cols;
        }
        float p[V][8], sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float h[8], o[8], dx[8], w[8], gw[8];
            if (g.DY)
                Src::values(a.h[i], h);
            if (read_o)
                Src::values(a.o[i], o);
            if constexpr (!HOLD) {
                if (g.DY)
                    weights8<T>(g.W, 0, g.w_f32, col(i), g.cols, w);
                if (out_o)
                    gate_weight(i, gw);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float d = g.DY ? a.rstd * ((float)a.dy[i][j] * (HOLD ? hw[HOLD ? i : 0][j] : w[j]) - h[j] * a.rstd * mean) : 0.0f;
                if (g.DH)
                    d += (float)a.dh[i][j];
                dx[j] = g.alpha * d;
                if (out_o)
                    p[i][j] = d * (HOLD ? hgw[HOLD ? i : 0][j] : gw[j]);
                if (read_o) {
                    const float m = o[j] * a.rstd_post;
                    sum = fmaf(p[i][j], m, sum);
                    t(i, j) = fmaf(d, m, t(i, j));
                }
            }
            if (g.DX && col(i) < g.cols)
                row_store8(static_cast<T *>(g.DX) + row * g.lddx, col(i), g.cols, dx);
        }
        if (g.DO) {
            mean = g.WP ? row_sum<NT, L>(sum, slot[2 + turn]) / (float)g.cols : 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (col(i) >= g.cols)
                    continue;
                if (g.WP) {
                    float o[8];
                    Src::values(a.o[i], o);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        p[i][j] = a.rstd_post * (p[i][j] - o[j] * a.rstd_post * mean);
                }
                row_store8(static_cast<T *>(g.DO) + row * g.lddo, col(i), g.cols, p[i]);
            }
        }
        if constexpr (SEVERAL) {
            if (row + 1 == r1 || row + 1 == gate_end) {
                const int64_t first = gate_end - g.gate_rows;
                const bool whole = first >= r0 && (row + 1 == gate_end || row + 1 == g.rows);
                float *out = !g.DG ? nullptr
                             : whole ? g.DG + gr * g.lddg
                                     : g.ws + (2 * (int64_t)g.groups + 2 * walker + (first > r0)) * g.cols;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float v[8], sum_t[8];
                    weights8<T>(g.G, gr * g.ldg, g.w_f32, col(i), g.cols, v);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        sum_t[j] = t(i, j);
                        t(i, j) = 0.0f;
                    }
                    if constexpr (FAR) {
                        if (g.DWP && col(i) < g.cols) {
                            float old[8];
                            row_load8<false>(place, col(i), g.cols, old);
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                old[j] = fmaf(v[j], sum_t[j], old[j]);
                            row_store8(place, col(i), g.cols, old);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            held(i, j) = fmaf(v[j], sum_t[j], held(i, j));
                    }
                    if (out && whole) {
                        weights8<T>(g.WP, 0, g.w_f32, col(i), g.cols, v);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            sum_t[j] *= v[j];
                    }
                    if (out && col(i) < g.cols)
                        row_store8(out, col(i), g.cols, sum_t);
                }
                if (row + 1 < r1) {
                    ++gr;
                    gate_end += g.gate_rows;
                    if constexpr (HOLD) {
#pragma unroll
                        for (int i = 0; i < V; ++i)
                            gate_weight(i, hgw[i]);
                    }
                }
            }
        }
    }
    // the workgroup's sums: of dy n, and of d m or gate d m
    if constexpr (FAR) {
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            if (k == 0 ? !g.DW : SEVERAL || (!g.DWP && (k == 2 || !g.DG)) || (k == 2 && g.team == g.groups))
                continue;
            float *out = g.ws + ((int64_t)k * g.groups + walk.group) * g.cols;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float v[8];
                weights8<T>(k == 2 ? g.G : nullptr, gr * g.ldg, g.w_f32, col(i), g.cols, v);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] *= k == 0 ? dw(i, j) : t(i, j);
                if (col(i) < g.cols)
                    row_store8(out, col(i), g.cols, v);
            }
        }
    } else {
        if constexpr (SEVERAL) {
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    rt[FAR ? 0 : i][j] = held(i, j);
        }
        if (g.DW)
            block_norm_put_sums<NT, L, V>(g.ws + (int64_t)walk.group * g.cols, sums, lane, own, g.cols, rdw);
        if (SEVERAL ? g.DWP != nullptr : g.DWP || g.DG)
            block_norm_put_sums<NT, L, V>(place, sums, lane, own, g.cols, rt);
        if (!SEVERAL && g.DWP && g.team < g.groups) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float v[8];
                weights8<T>(g.G, gr * g.ldg, g.w_f32, col(i), g.cols, v);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    rt[FAR ? 0 : i][j] *= v[j];
            }
            block_norm_put_sums<NT, L, V>(place + (int64_t)g.groups * g.cols, sums, lane, own, g.cols, rt);
        }
    }
}

// The same with dy, dh, dx and do, one piece a work-item and one gate a walker: few
// conditions in the loop, the next row's values requested as soon as this row's are
// converted, and n, g, m and p kept from one pass over the row to the next.  TAIL: the row's
// last piece may be shorter (rows of at least 8); its wavefront alone moves what it loaded
// (moved before the next row is requested, as in the other kernel, that request waits for
// memory: 16384 x 4095 330 us).
template <typename T, int NT, int L, bool KEPT, bool POST, bool TAIL>
__global__ __launch_bounds__(NT) void block_norm_bwd_all_kernel(BlockNormBwdArgs g)
{
    typedef typename Elt<T>::Raw Raw;
    typedef Source<T, KEPT> Src;
    constexpr int ROWS = NT / L;
    __shared__ float slot[4][NT / 64];
    __shared__ float sums[ROWS > 1 ? NT * 8 : 1];
    const int lane = threadIdx.x % L, own = ROWS == 1 ? 0 : threadIdx.x / L;
    const BlockNormWalk<false, ROWS> walk(g, own);
    const bool live = 8 * lane < g.cols, read_o = POST || g.O;
    // work-items past the row's end take its first piece and add zeros, or (TAIL) have zeros
    const int c = live || TAIL ? 8 * lane : 0, cols = TAIL ? g.cols : c + 8;
    const int past = c + 8 - cols;
    const bool moves = TAIL && __ballot(past > 0) != 0;
    struct Row {
        Raw dy, dh;
        typename Src::Raw h, o;
        float rstd, rstd_post;
    } b;
    auto request = [&](int64_t row) {
        b.dy = row_any8<true>(static_cast<const T *>(g.DY) + row * g.lddy, c, cols);
        Src::load_any(b.h, g.H, g.ldh, g.SH, g.ldsh, row, c, cols);
        b.dh = row_any8<true>(static_cast<const T *>(g.DH) + row * g.lddh, c, cols);
        if (read_o)
            Src::load_any(b.o, g.O, g.ldo, g.SO, g.ldso, row, c, cols);
        b.rstd = g.rstd[row];
        b.rstd_post = POST ? g.rstd_post[row] : 1.0f;
    };
    if (walk.first < walk.end)
        request(walk.first);
    float w[8], gw[8], wp[8], dw[1][8], t[1][8];
    weights8<T>(g.W, 0, g.w_f32, c, g.cols, w);
    weights8<T>(g.G, walk.gate * g.ldg, g.w_f32, c, g.cols, gw);
    weights8<T>(POST ? g.WP : nullptr, 0, g.w_f32, c, g.cols, wp);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        gw[j] *= wp[j];
        dw[0][j] = t[0][j] = 0.0f;
    }
    const float per_col = 1.0f / (float)g.cols;
    int turn = 0;
    for (int64_t row = walk.first; row < walk.end; row += walk.step, turn ^= 1) {
        const float rstd = b.rstd, rp = b.rstd_post;
        float n[8], gy[8], m[8], p[8], dh[8], sum = 0.0f;
        if (moves) {
            row_fix8<T>(b.dy, past);
            row_fix8<T>(b.dh, past);
            Src::fix(b.h, past);
            if (read_o)
                Src::fix(b.o, past);
        }
        Src::values(b.h, n);
        if (read_o)
            Src::values(b.o, m);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float dy = (float)b.dy[j];
            n[j] *= rstd;
            if (POST)
                m[j] *= rp;
            dh[j] = (float)b.dh[j];
            gy[j] = dy * w[j];
            sum = fmaf(gy[j], n[j], sum);
            dw[0][j] = fmaf(dy, n[j], dw[0][j]);
        }
        if (row + walk.step < walk.end)
            request(row + walk.step);
        const float mean = row_sum<NT, L>(live ? sum : 0.0f, slot[turn]) * per_col;
        float dx[8];
        sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float d = fmaf(rstd, fmaf(-mean, n[j], gy[j]), dh[j]);
            dx[j] = g.alpha * d;
            p[j] = d * gw[j];
            if (POST)
                sum = fmaf(p[j], m[j], sum);
            if (read_o)
                t[0][j] = fmaf(d, m[j], t[0][j]);
        }
        if (live)
            row_store8(static_cast<T *>(g.DX) + row * g.lddx, c, cols, dx);
        if constexpr (POST) {
            const float back = row_sum<NT, L>(live ? sum : 0.0f, slot[2 + turn]) * per_col * rp;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                p[j] = fmaf(rp, p[j], -back * m[j]);
        }
        if (live)
            row_store8(static_cast<T *>(g.DO) + row * g.lddo, c, cols, p);
    }
    if (g.DW)
        block_norm_put_sums<NT, L, 1>(g.ws + (int64_t)walk.group * g.cols, sums, lane, own, g.cols, dw);
    if (g.DWP || g.DG)
        block_norm_put_sums<NT, L, 1>(g.ws + ((int64_t)g.groups + walk.group) * g.cols, sums, lane, own, g.cols, t);
    if (g.DWP && g.team < g.groups) {
        weights8<T>(g.G, walk.gate * g.ldg, g.w_f32, c, g.cols, gw);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            t[0][j] *= gw[j];
        block_norm_put_sums<NT, L, 1>(g.ws + (2 * (int64_t)g.groups + walk.group) * g.cols, sums, lane, own, g.cols, t);
    }
}

// Work-items of a workgroup and of a row, and pieces per work-item: one piece up to 8192
// columns.
template <typename T, typename F>
void bwd_by_cols(int cols, F f)
{
    if (cols <= 128)
        f.template run<T, 256, 16, 1>();
    else if (cols <= 256)
        f.template run<T, 256, 32, 1>();
    else if (cols <= 512)
        f.template run<T, 256, 64, 1>();
    else if (cols <= 1024)
        f.template run<T, 128, 128, 1>();
    else if (cols <= 2048)
        f.template run<T, 256, 256, 1>();
    else if (cols <= 4096)
        f.template run<T, 512, 512, 1>();
    else if (cols <= 8192)
        f.template run<T, 1024, 1024, 1>();
    else if (cols <= 16384)
        f.template run<T, 1024, 1024, 2>();
    else
        f.template run<T, 1024, 1024, 4>();
}

template <bool KEPT> struct Bwd {
    const BlockNormBwdArgs &a;
    hipStream_t s;
    template <typename T, int NT, int L, int V, bool SEVERAL> void go()
    {
        if constexpr (V == 1 && !SEVERAL) {
            if (a.DY && a.DH && a.DX && a.DO && a.cols >= 8) {
                const dim3 grid((unsigned)a.groups), block(NT);
                const bool whole = a.cols % 8 == 0;
                if (a.WP && whole)
                    block_norm_bwd_all_kernel<T, NT, L, KEPT, true, false><<<grid, block, 0, s>>>(a);
                else if (a.WP)
                    block_norm_bwd_all_kernel<T, NT, L, KEPT, true, true><<<grid, block, 0, s>>>(a);
                else if (whole)
                    block_norm_bwd_all_kernel<T, NT, L, KEPT, false, false><<<grid, block, 0, s>>>(a);
                else
                    block_norm_bwd_all_kernel<T, NT, L, KEPT, false, true><<<grid, block, 0, s>>>(a);
                return;
            }
        }
        constexpr bool AHEAD = V == 1 && NT < 1024;
        block_norm_bwd_kernel<T, NT, L, V, AHEAD, KEPT, SEVERAL><<<(unsigned)a.groups, NT, 0, s>>>(a);
    }
    template <typename T, int NT, int L, int V> void run()
    {
        a.team ? go<T, NT, L, V, false>() : go<T, NT, L, V, true>();
    }
};

}  // namespace

// The kernels of each type of row, from kept values or not, are compiled in a file of their own.
template <typename T, bool KEPT> void launch_block_norm_bwd_from(const BlockNormBwdArgs &a, hipStream_t s);
template <typename T> void launch_block_norm_bwd_rows(const BlockNormBwdArgs &a, bool kept, hipStream_t s)
{
    kept ? launch_block_norm_bwd_from<T, true>(a, s) : launch_block_norm_bwd_from<T, false>(a, s);
}

}  // namespace sgemm
