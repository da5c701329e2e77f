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

// AHEAD: the next row's values are requested before this row's are used.  SEVERAL: the
// gate has more rows than one.
template <typename T, int NT, int L, int V, bool AHEAD, bool KEPT, bool SEVERAL>
__global__ __launch_bounds__(NT) void block_norm_bwd_kernel(BlockNormBwdArgs g)
{
    typedef typename Elt<T>::Raw Raw;
    typedef Source<T, KEPT> Src;
    constexpr int ROWS = NT / L;
    __shared__ float slot[4][NT / 64];
    __shared__ float sums[ROWS > 1 ? NT * 8 * V : 1];
    const int lane = threadIdx.x % L, own = threadIdx.x / L;
    const bool read_o = g.O != nullptr, out_o = g.DO || g.DWP || g.DG;
    const int64_t walker = (int64_t)blockIdx.x * ROWS + own, r0 = walker * g.chunk;
    const int64_t r1 = min<int64_t>(g.rows, r0 + g.chunk);

    float w[V][8], wp[V][8], gate[V][8], dw[V][8], t[V][8], dwp[SEVERAL ? V : 1][8];
    int gr = SEVERAL ? (int)((uint32_t)min<int64_t>(r0, g.rows - 1) / (uint32_t)g.gate_rows) : 0;  // the gate's row
    int64_t gate_end = SEVERAL ? (int64_t)(gr + 1) * g.gate_rows : g.rows;
    auto load_gate = [&] {
#pragma unroll
        for (int i = 0; i < V; ++i)
            weights8<T>(g.G, gr * g.ldg, g.w_f32, 8 * (lane + L * i), g.cols, gate[i]);
    };
    load_gate();
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = 8 * (lane + L * i);
        weights8<T>(g.W, 0, g.w_f32, c, g.cols, w[i]);
        weights8<T>(g.WP, 0, g.w_f32, c, g.cols, wp[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            dw[i][j] = t[i][j] = 0.0f;
            if (SEVERAL)
                dwp[i][j] = 0.0f;
        }
    }
    struct Row {
        Raw dy[V], dh[V];
        typename Src::Raw h[V], o[V];
        float rstd, rstd_post;
    } a, b;
    auto request = [&](int64_t row, Row &to) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = 8 * (lane + L * i);
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
                float h[8];
                Src::values(a.h[i], h);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float dy = (float)a.dy[i][j], n = h[j] * a.rstd;
                    sum = fmaf(dy * w[i][j], n, sum);
                    dw[i][j] = fmaf(dy, n, dw[i][j]);
                }
            }
            mean = row_sum<NT, L>(sum, slot[turn]) / (float)g.cols;
        }
        float p[V][8], sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = 8 * (lane + L * i);
            float h[8], o[8], dx[8];
            if (g.DY)
                Src::values(a.h[i], h);
            if (read_o)
                Src::values(a.o[i], o);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float d = g.DY ? a.rstd * ((float)a.dy[i][j] * w[i][j] - h[j] * a.rstd * mean) : 0.0f;
                if (g.DH)
                    d += (float)a.dh[i][j];
                dx[j] = g.alpha * d;
                p[i][j] = gate[i][j] * d * wp[i][j];
                if (read_o) {
                    const float m = o[j] * a.rstd_post;
                    sum = fmaf(p[i][j], m, sum);
                    t[i][j] = fmaf(d, m, t[i][j]);
                }
            }
            if (g.DX && c < g.cols)
                row_store8(static_cast<T *>(g.DX) + row * g.lddx, c, g.cols, dx);
        }
        if (out_o) {
            mean = g.WP ? row_sum<NT, L>(sum, slot[2 + turn]) / (float)g.cols : 0.0f;
            if (g.DO) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int c = 8 * (lane + L * i);
                    if (c >= g.cols)
                        continue;
                    float o[8];
                    if (read_o)
                        Src::values(a.o[i], o);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        p[i][j] = g.WP ? a.rstd_post * (p[i][j] - o[j] * a.rstd_post * mean) : p[i][j];
                    row_store8(static_cast<T *>(g.DO) + row * g.lddo, c, g.cols, p[i]);
                }
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
                    const int c = 8 * (lane + L * i);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        dwp[i][j] = fmaf(gate[i][j], t[i][j], dwp[i][j]);
                        if (whole)
                            t[i][j] *= wp[i][j];
                    }
                    if (out && c < g.cols)
                        row_store8(out, c, g.cols, t[i]);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        t[i][j] = 0.0f;
                }
                if (row + 1 < r1) {
                    ++gr;
                    gate_end += g.gate_rows;
                    load_gate();
                }
            }
        }
    }
    // the workgroup's sums: of dy n, and of d m or gate d m
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (!(k == 0 ? g.DW : SEVERAL ? g.DWP : g.DWP || g.DG ? g.ws : nullptr))
            continue;
        float *out = g.ws + ((int64_t)k * g.groups + blockIdx.x) * g.cols;
        if constexpr (ROWS == 1) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = 8 * (lane + L * i);
                if (c < g.cols)
                    row_store8(out, c, g.cols, k == 0 ? dw[i] : SEVERAL ? dwp[i] : t[i]);
            }
        } else {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    sums[(own * 8 + j) * (V * L) + L * i + lane] = k == 0 ? dw[i][j] : SEVERAL ? dwp[i][j] : t[i][j];
            __syncthreads();
            for (int c = threadIdx.x; c < g.cols; c += NT) {
                float s = 0.0f;
#pragma unroll
                for (int r = 0; r < ROWS; ++r)
                    s += sums[(r * 8 + c % 8) * (V * L) + c / 8];
                out[c] = s;
            }
        }
    }
}

struct Bwd {
    const BlockNormBwdArgs &a;
    bool kept, several;
    hipStream_t s;
    template <typename T, int NT, int L, int V, bool KEPT, bool SEVERAL> void go()
    {
        block_norm_bwd_kernel<T, NT, L, V, false, KEPT, SEVERAL><<<(unsigned)a.groups, NT, 0, s>>>(a);
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
