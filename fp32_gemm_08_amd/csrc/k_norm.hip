// Root-mean-square norm with the residual's addition and an 8-bit output, and
// its backward pass.
//
// L work-items hold a row, each V pieces of 8 consecutive columns in registers,
// so each row is read once: a workgroup takes one row (L = NT) or, of rows of up
// to 512 columns, NT / L at a time (16, 32 or 64 lanes a row).  16 consecutive
// lanes hold one block of 128 columns, whose maximum is four lane permutations.
//
// Backward: with n = h * rstd and g = dy * w,
//     dx = rstd * (g - n * mean(g n)) + dh,      dw = sum over rows of dy n.
// A workgroup walks the rows, a stride of all workgroups' rows apart; each
// work-item keeps the sums of dw for its columns in registers, and a second
// kernel adds the workgroups' sums in a fixed order.
#include "norm_rows.h"

#include <algorithm>

namespace sgemm {
namespace {

template <typename T, int NT, int L, int V>
__global__ __launch_bounds__(NT) void rmsnorm_kernel(NormArgs g)
{
    __shared__ float slot[NT / 64];
    const int lane = threadIdx.x % L;                                    // of the row's
    const int64_t row = (int64_t)blockIdx.x * (NT / L) + threadIdx.x / L;
    if (row >= g.rows)
        return;  // whole rows of lanes, and only where no row needs the workgroup
    const T *x = static_cast<const T *>(g.X) + row * g.ldx;
    float h[V][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = 8 * (lane + L * i);
        row_load8<true>(x, c, g.cols, h[i]);
        if (g.R) {
            float r[8];
            row_load8<true>(static_cast<const T *>(g.R) + row * g.ldr, c, g.cols, r);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                h[i][j] += r[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            ss = fmaf(h[i][j], h[i][j], ss);
        if (g.H && c < g.cols)
            row_store8(static_cast<T *>(g.H) + row * g.ldh, c, g.cols, h[i]);
    }
    ss = row_sum<NT, L>(ss, slot);
    const float rstd = 1.0f / sqrtf(ss / (float)g.cols + g.eps);
    if (g.rstd && lane == 0)
        g.rstd[row] = rstd;
    if (!g.Y && !g.Q)
        return;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = 8 * (lane + L * i);
        float w[8], y[8];
        load_w8<T>(g.W, g.w_f32, c, g.cols, w);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            y[j] = c + j < g.cols ? h[i][j] * rstd * w[j] : 0.0f;
        if (g.Y && c < g.cols)
            row_store8(static_cast<T *>(g.Y) + row * g.ldy, c, g.cols, y);
        if (g.Q) {
            float inv, scale;
            block_scale<0>(max16(abs_max8(y)), inv, scale);
            if (c < g.cols) {
                const uint32_t lo = f8_pack4<0>(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
                const uint32_t hi = f8_pack4<0>(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv);
                row_store8b(g.Q + row * g.ldq, c, g.cols, lo, hi);
                if ((threadIdx.x & 15) == 0)
                    g.S[(int64_t)(c / F8_BLOCK) * g.lds + row] = scale;
            }
        }
    }
}

// AHEAD: the next row's values are requested before this row's are used.
template <typename T, int NT, int L, int V, bool AHEAD>
__global__ __launch_bounds__(NT) void rmsnorm_bwd_kernel(NormBwdArgs g)
{
    typedef typename Elt<T>::Raw Raw;
    constexpr int ROWS = NT / L;
    __shared__ float slot[2][NT / 64];
    __shared__ float sums[ROWS > 1 ? NT * 8 * V : 1];
    const int lane = threadIdx.x % L, own = threadIdx.x / L;
    float dw[V][8], w[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        load_w8<T>(g.W, g.w_f32, 8 * (lane + L * i), g.cols, w[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            dw[i][j] = 0.0f;
    }
    Raw dy[V], h[V], dh[V];
    Raw ady[AHEAD ? V : 1], ah[AHEAD ? V : 1], adh[AHEAD ? V : 1];  // the next row's
    auto request = [&](int64_t row, Raw *to_dy, Raw *to_h, Raw *to_dh) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = 8 * (lane + L * i);
            to_dy[i] = row_raw8<true>(static_cast<const T *>(g.DY) + row * g.lddy, c, g.cols);
            to_h[i] = row_raw8<true>(static_cast<const T *>(g.H) + row * g.ldh, c, g.cols);
            if (g.DH)
                to_dh[i] = row_raw8<true>(static_cast<const T *>(g.DH) + row * g.lddh, c, g.cols);
        }
    };
    const int64_t step = (int64_t)g.groups * ROWS;
    int64_t row = (int64_t)blockIdx.x * ROWS + own;
    if (AHEAD && row < g.rows)
        request(row, ady, ah, adh);
    for (int turn = 0; row < g.rows; row += step, turn ^= 1) {
        const float rstd = g.rstd[row];
        if constexpr (AHEAD) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                dy[i] = ady[i];
                h[i] = ah[i];
                dh[i] = adh[i];
            }
            if (row + step < g.rows)
                request(row + step, ady, ah, adh);
        } else {
            request(row, dy, h, dh);
        }
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float d = (float)dy[i][j], n = (float)h[i][j] * rstd;
                sum = fmaf(d * w[i][j], n, sum);
                dw[i][j] = fmaf(d, n, dw[i][j]);
            }
        }
        const float mean = row_sum<NT, L>(sum, slot[turn]) / (float)g.cols;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = 8 * (lane + L * i);
            if (c >= g.cols)
                continue;
            float dx[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dx[j] = rstd * ((float)dy[i][j] * w[i][j] - (float)h[i][j] * rstd * mean);
                if (g.DH)
                    dx[j] += (float)dh[i][j];
            }
            row_store8(static_cast<T *>(g.DX) + row * g.lddx, c, g.cols, dx);
        }
    }
    if (!g.DW)
        return;
    float *out = g.ws + (int64_t)blockIdx.x * g.cols;
    if constexpr (ROWS == 1) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = 8 * (lane + L * i);
            if (c < g.cols)
                row_store8(out, c, g.cols, dw[i]);
        }
    } else {
        // the workgroup's rows of lanes, in order
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                sums[(own * 8 + j) * (V * L) + L * i + lane] = dw[i][j];
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

// dw[c] = sum over the workgroups' partial sums, 32 columns and 32 strips of
// partial sums per workgroup, in a fixed order; 8 loads of a strip at a time,
// which is what its time is made of.
__global__ __launch_bounds__(1024) void rmsnorm_dw_kernel(const float *ws, int groups, int cols, float *dw)
{
    __shared__ float part[32][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + x;
    float s = 0.0f;
    if (c < cols)
        for (int i = y; i < groups; i += 8 * 32) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = i + 32 * j < groups ? ws[(int64_t)(i + 32 * j) * cols + c] : 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                s += v[j];
        }
    part[y][x] = s;
    __syncthreads();
    if (y == 0 && c < cols) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            s += part[i][x];
        dw[c] = s;
    }
}

struct Fwd {
    const NormArgs &a;
    hipStream_t s;
    template <typename T, int NT, int L, int V> void run()
    {
        rmsnorm_kernel<T, NT, L, V><<<(unsigned)ceil_div(a.rows, NT / L), NT, 0, s>>>(a);
    }
};
// Work-items of that launch.
struct Items {
    int64_t rows;
    int64_t *out;
    template <typename T, int NT, int L, int V> void run() { *out = ceil_div(rows, NT / L) * NT; }
};
struct Bwd {
    const NormBwdArgs &a;
    hipStream_t s;
    template <typename T, int NT, int L, int V> void run()
    {
        // 1024 work-items have 128 registers each, which is too few above 8192 columns.  With
        // two pieces the next row is held in 16 bits only (190 registers are spilled of bf16
        // rows, 169 of fp16; of 32-bit rows 6, without it); with four 660 and more are spilled
        // either way.  Measured: 8192 x 8192 bf16, nothing spilled, 101 us (5.3 TB/s); 4096 x
        // 16384 bf16 123 (4.4); 2048 x 32768 bf16 293 (1.8), fp32 430 (2.5).
        constexpr bool AHEAD = NT < 1024 || (V == 2 && sizeof(T) == 2);
        rmsnorm_bwd_kernel<T, NT, L, V, AHEAD><<<(unsigned)a.groups, NT, 0, s>>>(a);
    }
};
// Workgroups of the backward pass: 12 wavefronts per CU, 8 of those that hold two
// pieces a lane (measured in us with 512 / 768 / 1024 / 2048 workgroups of 256, bf16:
// 65536 x 300 81 / 62 / 53 / 56, 65536 x 128 16.4 / 16.4 / 17.1 / 20.3, 32768 x 2048
// 116 / 100 / 107 / 116; two pieces: 16384 x 4096 106 / 110 / 115 / 118).  Of few
// rows, one row for each: 11.9 us on 1000 rows, 14.8 with 8 rows to a workgroup.
struct Groups {
    int64_t rows;
    int64_t *out;
    template <typename T, int NT, int L, int V> void run()
    {
        constexpr int64_t ROWS = NT / L, MOST = NT >= 512 ? 256 : V == 1 ? 768 : 512;
        *out = std::min((rows + ROWS - 1) / ROWS, MOST);
    }
};

}  // namespace

hipError_t launch_rmsnorm(const NormArgs &a, int type, hipStream_t s)
{
    by_type(type, a.cols, Fwd{a, s});
    return hipGetLastError();
}

int64_t rmsnorm_work_items(int64_t rows, int64_t cols)
{
    int64_t n = 0;
    by_cols<float>((int)cols, Items{rows, &n});
    return n;
}

int64_t rmsnorm_bwd_groups(int64_t rows, int64_t cols)
{
    int64_t n = 0;
    by_cols<float>((int)cols, Groups{rows, &n});
    return n;
}

hipError_t launch_rmsnorm_bwd(const NormBwdArgs &a, int type, hipStream_t s)
{
    if (a.groups > 0) {
        by_type(type, a.cols, Bwd{a, s});
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    if (a.DW)
        rmsnorm_dw_kernel<<<(unsigned)((a.cols + 31) / 32), 1024, 0, s>>>(a.ws, a.groups, a.cols, a.DW);
    return hipGetLastError();
}

}  // namespace sgemm
