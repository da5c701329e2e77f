// Backward pass of the norms around a block.  With n = h * rstd, m = o * rstd_post (or o)
// and g = dy * w:
//
//     d = rstd * (g - n * mean(g n)) + dh          dx = alpha * d
//     p = gate * d * w_post                        do = rstd_post * (p - m * mean(p m))
//     dw = sum dy n     t = sum over the rows of a gate of d m
//     dw_post = sum over gates of gate * t         dgate = w_post * t
//
// so one sum t serves both of the last.  A walker (a workgroup, or the 16 to 64 lanes
// that hold a row) takes consecutive rows and keeps its columns' sums in registers; a
// second kernel adds what the walkers left, in a fixed order.  Consecutive rows, since
// the scales of 32 consecutive rows' blocks share a line.
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

// What a work-item holds of a row: V pieces of 8 consecutive columns.  Its sums of dw and
// t, and with one piece also w and gate * w_post, stay in registers: with these, two rows
// of 16-bit values and the working values one piece fits the 128 registers of 16
// wavefronts per CU.  More pieces read the weights again for every row, from the L2.
// dw_post, which changes once per row of the gate, is kept in the LDS.
// AHEAD: the next row's values are requested before this row's are used.  SEVERAL: the
// gate has more rows than one.
template <typename T, int NT, int L, int V, bool AHEAD, bool KEPT, bool SEVERAL>
__global__ __launch_bounds__(NT) void block_norm_bwd_kernel(BlockNormBwdArgs g)
{
    typedef typename Elt<T>::Raw Raw;
    typedef Source<T, KEPT> Src;
    constexpr int ROWS = NT / L;
    constexpr bool HOLD = V == 1;
    __shared__ float slot[4][NT / 64];
    __shared__ float sums[SEVERAL || ROWS > 1 ? NT * 8 * V : 1];
    const int lane = threadIdx.x % L, own = ROWS == 1 ? 0 : threadIdx.x / L;
    const bool read_o = g.O != nullptr, out_o = g.DO || g.DWP || g.DG;
    const int64_t walker = (int64_t)blockIdx.x * ROWS + own, r0 = walker * g.chunk;
    const int64_t r1 = min<int64_t>(g.rows, r0 + g.chunk);
    auto col = [&](int i) { return 8 * (lane + L * i); };
    auto held = [&](int i, int j) -> float & { return sums[(j * V + i) * NT + threadIdx.x]; };

    int gr = SEVERAL ? (int)((uint32_t)min<int64_t>(r0, g.rows - 1) / (uint32_t)g.gate_rows) : 0;  // the gate's row
    int64_t gate_end = SEVERAL ? (int64_t)(gr + 1) * g.gate_rows : g.rows;
    auto gate_weight = [&](int i, float (&v)[8]) {  // gate * w_post
        float wp[8];
        weights8<T>(g.G, gr * g.ldg, g.w_f32, col(i), g.cols, v);
        weights8<T>(g.WP, 0, g.w_f32, col(i), g.cols, wp);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] *= wp[j];
    };
    float hw[HOLD ? V : 1][8], hgw[HOLD ? V : 1][8], dw[V][8], t[V][8];
    if constexpr (HOLD) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            weights8<T>(g.W, 0, g.w_f32, col(i), g.cols, hw[i]);
            gate_weight(i, hgw[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            dw[i][j] = t[i][j] = 0.0f;
            if (SEVERAL)
                held(i, j) = 0.0f;
        }
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
    int turn = 0;
    for (int64_t row = r0; row < r1; ++row, turn ^= 1) {
        if constexpr (AHEAD) {
            a = b;
            if (row + 1 < r1)
                request(row + 1, b);
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
                    dw[i][j] = fmaf(dy, n, dw[i][j]);
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
                    t[i][j] = fmaf(d, m, t[i][j]);
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
                    float v[8];
                    weights8<T>(g.G, gr * g.ldg, g.w_f32, col(i), g.cols, v);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        held(i, j) = fmaf(v[j], t[i][j], held(i, j));
                    if (out && whole) {
                        weights8<T>(g.WP, 0, g.w_f32, col(i), g.cols, v);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            t[i][j] *= v[j];
                    }
                    if (out && col(i) < g.cols)
                        row_store8(out, col(i), g.cols, t[i]);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        t[i][j] = 0.0f;
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
    // the workgroup's sums: of d m or gate d m, and of dy n
    if constexpr (SEVERAL) {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                t[i][j] = held(i, j);
    }
    if (g.DW)
        block_norm_put_sums<NT, L, V>(g.ws + (int64_t)blockIdx.x * g.cols, sums, lane, own, g.cols, dw);
    if (SEVERAL ? g.DWP != nullptr : g.DWP || g.DG)
        block_norm_put_sums<NT, L, V>(g.ws + ((int64_t)g.groups + blockIdx.x) * g.cols, sums, lane, own, g.cols, t);
}

// The same for whole pieces (cols a multiple of 8) with every operand and DX and DO there,
// one piece a work-item: no conditions in the loop, the next row's values requested as soon
// as this row's are converted, and n, g, m and p kept from one pass over the row to the next.
template <typename T, int NT, int L, bool KEPT, bool SEVERAL>
__global__ __launch_bounds__(NT) void block_norm_bwd_whole_kernel(BlockNormBwdArgs g)
{
    typedef typename Elt<T>::Raw Raw;
    typedef Source<T, KEPT> Src;
    constexpr int ROWS = NT / L;
    __shared__ float slot[4][NT / 64];
    __shared__ float sums[SEVERAL || ROWS > 1 ? NT * 8 : 1];
    const int lane = threadIdx.x % L, own = ROWS == 1 ? 0 : threadIdx.x / L;
    const int64_t walker = (int64_t)blockIdx.x * ROWS + own, r0 = walker * g.chunk;
    const int64_t r1 = min<int64_t>(g.rows, r0 + g.chunk);
    const bool live = 8 * lane < g.cols;
    const int c = live ? 8 * lane : 0;      // (work-items past the row's end take its first piece, and add zeros)
    auto held = [&](int j) -> float & { return sums[j * NT + threadIdx.x]; };

    int gr = SEVERAL ? (int)((uint32_t)min<int64_t>(r0, g.rows - 1) / (uint32_t)g.gate_rows) : 0;  // the gate's row
    int64_t gate_end = SEVERAL ? (int64_t)(gr + 1) * g.gate_rows : g.rows;
    float w[8], gw[8], dw[8], t[8];
    auto gate_weight = [&] {  // gate * w_post
        float wp[8];
        weights8<T>(g.G, gr * g.ldg, g.w_f32, c, g.cols, gw);
        weights8<T>(g.WP, 0, g.w_f32, c, g.cols, wp);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            gw[j] *= wp[j];
    };
    weights8<T>(g.W, 0, g.w_f32, c, g.cols, w);
    gate_weight();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        dw[j] = t[j] = 0.0f;
        if (SEVERAL)
            held(j) = 0.0f;
    }
    struct Row {
        Raw dy, dh;
        typename Src::Raw h, o;
        float rstd, rstd_post;
    } b;
    auto request = [&](int64_t row) {
        b.dy = Elt<T>::template raw8<true>(static_cast<const T *>(g.DY) + row * g.lddy + c);
        Src::load(b.h, g.H, g.ldh, g.SH, g.ldsh, row, c, c + 8);
        b.dh = Elt<T>::template raw8<true>(static_cast<const T *>(g.DH) + row * g.lddh + c);
        Src::load(b.o, g.O, g.ldo, g.SO, g.ldso, row, c, c + 8);
        b.rstd = g.rstd[row];
        b.rstd_post = g.rstd_post[row];
    };
    if (r0 < r1)
        request(r0);
    const float per_col = 1.0f / (float)g.cols;
    int turn = 0;
    for (int64_t row = r0; row < r1; ++row, turn ^= 1) {
        const float rstd = b.rstd, rp = b.rstd_post;
        float n[8], gy[8], m[8], p[8], dh[8], sum = 0.0f;
        Src::values(b.h, n);
        Src::values(b.o, m);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float dy = (float)b.dy[j];
            n[j] *= rstd;
            m[j] *= rp;
            dh[j] = (float)b.dh[j];
            gy[j] = dy * w[j];
            sum = fmaf(gy[j], n[j], sum);
            dw[j] = fmaf(dy, n[j], dw[j]);
        }
        if (row + 1 < r1)
            request(row + 1);
        const float mean = row_sum<NT, L>(live ? sum : 0.0f, slot[turn]) * per_col;
        float dx[8];
        sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float d = fmaf(rstd, fmaf(-mean, n[j], gy[j]), dh[j]);
            dx[j] = g.alpha * d;
            p[j] = d * gw[j];
            sum = fmaf(p[j], m[j], sum);
            t[j] = fmaf(d, m[j], t[j]);
        }
        if (live)
            Elt<T>::store8(static_cast<T *>(g.DX) + row * g.lddx + c, dx);
        const float back = row_sum<NT, L>(live ? sum : 0.0f, slot[2 + turn]) * per_col * rp;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            p[j] = fmaf(rp, p[j], -back * m[j]);
        if (live)
            Elt<T>::store8(static_cast<T *>(g.DO) + row * g.lddo + c, p);
        if constexpr (SEVERAL) {
            if (row + 1 == r1 || row + 1 == gate_end) {
                const int64_t first = gate_end - g.gate_rows;
                const bool whole = first >= r0 && (row + 1 == gate_end || row + 1 == g.rows);
                float *out = !g.DG ? nullptr
                             : whole ? g.DG + gr * g.lddg
                                     : g.ws + (2 * (int64_t)g.groups + 2 * walker + (first > r0)) * g.cols;
                float v[8];
                weights8<T>(g.G, gr * g.ldg, g.w_f32, c, g.cols, v);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    held(j) = fmaf(v[j], t[j], held(j));
                if (out && whole) {
                    weights8<T>(g.WP, 0, g.w_f32, c, g.cols, v);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        t[j] *= v[j];
                }
                if (out && live)
                    Elt<float>::store8(out + c, t);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    t[j] = 0.0f;
                if (row + 1 < r1) {
                    ++gr;
                    gate_end += g.gate_rows;
                    gate_weight();
                }
            }
        }
    }
    if constexpr (SEVERAL) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            t[j] = held(j);
    }
    if (g.DW)
        block_norm_put_sums<NT, L, 1>(g.ws + (int64_t)blockIdx.x * g.cols, sums, lane, own, g.cols, &dw);
    if (SEVERAL ? g.DWP != nullptr : g.DWP || g.DG)
        block_norm_put_sums<NT, L, 1>(g.ws + ((int64_t)g.groups + blockIdx.x) * g.cols, sums, lane, own, g.cols, &t);
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
        f.template run<T, 512, 512, 2>();
    else if (cols <= 16384)
        f.template run<T, 512, 512, 4>();
    else
        f.template run<T, 1024, 1024, 4>();
}

struct Bwd {
    const BlockNormBwdArgs &a;
    bool kept, several;
    hipStream_t s;
    template <typename T, int NT, int L, int V, bool KEPT, bool SEVERAL> void go()
    {
        if constexpr (V == 1) {
            if (a.cols % 8 == 0 && a.DY && a.DH && a.DX && a.DO && a.WP) {
                block_norm_bwd_whole_kernel<T, NT, L, KEPT, SEVERAL><<<(unsigned)a.groups, NT, 0, s>>>(a);
                return;
            }
        }
        constexpr bool AHEAD = V == 2 && sizeof(T) == 2;
        block_norm_bwd_kernel<T, NT, L, V, AHEAD, KEPT, SEVERAL><<<(unsigned)a.groups, NT, 0, s>>>(a);
    }
    template <typename T, int NT, int L, int V> void run()
    {
        kept ? several ? go<T, NT, L, V, true, true>() : go<T, NT, L, V, true, false>()
             : several ? go<T, NT, L, V, false, true>() : go<T, NT, L, V, false, false>();
    }
};

}  // namespace

// The kernels of each type of row are compiled in a file of their own.
template <typename T> void launch_block_norm_bwd_rows(const BlockNormBwdArgs &a, bool kept, bool several, hipStream_t s);

}  // namespace sgemm
