// Root-mean-square norm with the residual's addition and an 8-bit output, and
// its backward pass.
//
// Forward: a workgroup of NT work-items per row, each holding V pieces of 8
// consecutive columns in registers between the sum of squares and the output,
// so each row is read once.  16 consecutive lanes hold one block of 128
// columns, whose maximum is four lane permutations.
//
// Backward: with n = h * rstd and g = dy * w,
//     dx = rstd * (g - n * mean(g n)) + dh,      dw = sum over rows of dy n.
// A workgroup walks the rows blockIdx.x, blockIdx.x + groups, ...; each
// work-item keeps the sums of dw for its columns in registers, and a second
// kernel adds the workgroups' sums in a fixed order.
#include "f8_types.h"

namespace sgemm {
namespace {

// Sum of `v` over the workgroup, in every work-item.  `slot` has NT/64 floats
// that no other sum uses at the same time.
template <int NT>
__device__ __forceinline__ float group_sum(float v, float *slot)
{
    v = wave_sum(v);
    if constexpr (NT > 64) {
        if ((threadIdx.x & 63) == 0)
            slot[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < NT / 64; ++i)
            v += slot[i];
    }
    return v;
}

template <typename T>
__device__ __forceinline__ void load_w8(const void *W, int w_f32, int c, int cols, float (&v)[8])
{
    if (w_f32)
        row_load8(static_cast<const float *>(W), c, cols, v);
    else
        row_load8(static_cast<const T *>(W), c, cols, v);
}

template <typename T, int NT, int V>
__global__ __launch_bounds__(NT) void rmsnorm_kernel(NormArgs g)
{
    __shared__ float slot[NT / 64];
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(g.X) + row * g.ldx;
    float h[V][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = 8 * (threadIdx.x + NT * i);
        row_load8(x, c, g.cols, h[i]);
        if (g.R) {
            float r[8];
            row_load8(static_cast<const T *>(g.R) + row * g.ldr, c, g.cols, r);
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
    ss = group_sum<NT>(ss, slot);
    const float rstd = 1.0f / sqrtf(ss / (float)g.cols + g.eps);
    if (g.rstd && threadIdx.x == 0)
        g.rstd[row] = rstd;
    if (!g.Y && !g.Q)
        return;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = 8 * (threadIdx.x + NT * i);
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

template <typename T, int NT, int V>
__global__ __launch_bounds__(NT) void rmsnorm_bwd_kernel(NormBwdArgs g)
{
    __shared__ float slot[2][NT / 64];
    float dw[V][8], w[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        load_w8<T>(g.W, g.w_f32, 8 * (threadIdx.x + NT * i), g.cols, w[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            dw[i][j] = 0.0f;
    }
    int turn = 0;
    for (int64_t row = blockIdx.x; row < g.rows; row += g.groups, turn ^= 1) {
        const float rstd = g.rstd[row];
        float dy[V][8], n[V][8];
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = 8 * (threadIdx.x + NT * i);
            row_load8(static_cast<const T *>(g.DY) + row * g.lddy, c, g.cols, dy[i]);
            row_load8(static_cast<const T *>(g.H) + row * g.ldh, c, g.cols, n[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                n[i][j] *= rstd;
                sum = fmaf(dy[i][j] * w[i][j], n[i][j], sum);
                dw[i][j] = fmaf(dy[i][j], n[i][j], dw[i][j]);
            }
        }
        const float mean = group_sum<NT>(sum, slot[turn]) / (float)g.cols;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = 8 * (threadIdx.x + NT * i);
            if (c >= g.cols)
                continue;
            float dx[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                dx[j] = rstd * (dy[i][j] * w[i][j] - n[i][j] * mean);
            if (g.DH) {
                float dh[8];
                row_load8(static_cast<const T *>(g.DH) + row * g.lddh, c, g.cols, dh);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    dx[j] += dh[j];
            }
            row_store8(static_cast<T *>(g.DX) + row * g.lddx, c, g.cols, dx);
        }
    }
    if (g.DW) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = 8 * (threadIdx.x + NT * i);
            if (c < g.cols)
                row_store8(g.ws + (int64_t)blockIdx.x * g.cols, c, g.cols, dw[i]);
        }
    }
}

// dw[c] = sum over the workgroups' partial sums, 32 columns and 32 strips of
// partial sums per workgroup, in a fixed order.
__global__ __launch_bounds__(1024) void rmsnorm_dw_kernel(const float *ws, int groups, int cols, float *dw)
{
    __shared__ float part[32][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + x;
    float s = 0.0f;
    if (c < cols)
        for (int i = y; i < groups; i += 32)
            s += ws[(int64_t)i * cols + c];
    part[y][x] = s;
    __syncthreads();
    if (y == 0 && c < cols) {
        s = 0.0f;
        for (int i = 0; i < 32; ++i)
            s += part[i][x];
        dw[c] = s;
    }
}

// Work-items per row and pieces per work-item that cover `cols`.
template <typename T, typename F>
void by_cols(int cols, F f)
{
    if (cols <= 512)
        f.template run<T, 64, 1>();
    else if (cols <= 1024)
        f.template run<T, 128, 1>();
    else if (cols <= 2048)
        f.template run<T, 256, 1>();
    else if (cols <= 4096)
        f.template run<T, 256, 2>();
    else if (cols <= 8192)
        f.template run<T, 512, 2>();
    else if (cols <= 16384)
        f.template run<T, 1024, 2>();
    else
        f.template run<T, 1024, 4>();
}

struct Fwd {
    const NormArgs &a;
    hipStream_t s;
    template <typename T, int NT, int V> void run() { rmsnorm_kernel<T, NT, V><<<(unsigned)a.rows, NT, 0, s>>>(a); }
};
struct Bwd {
    const NormBwdArgs &a;
    hipStream_t s;
    template <typename T, int NT, int V> void run()
    {
        rmsnorm_bwd_kernel<T, NT, V><<<(unsigned)a.groups, NT, 0, s>>>(a);
    }
};

template <typename F>
void by_type(int type, int cols, F f)
{
    if (type == SGEMM_TYPE_F32)
        by_cols<float>(cols, f);
    else if (type == SGEMM_TYPE_FP16)
        by_cols<_Float16>(cols, f);
    else
        by_cols<__bf16>(cols, f);
}

}  // namespace

hipError_t launch_rmsnorm(const NormArgs &a, int type, hipStream_t s)
{
    by_type(type, a.cols, Fwd{a, s});
    return hipGetLastError();
}

int64_t rmsnorm_bwd_groups(int64_t rows, int64_t cols)
{
    (void)cols;
    return rows < 1024 ? rows : 1024;
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
