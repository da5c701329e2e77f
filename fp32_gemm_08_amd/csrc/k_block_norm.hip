// The norms after and before a block, with the block's gate and the residual's scale:
//
//     z = o * rstd_post * w_post      h = alpha * x + gate * z      y = h * rstd * w
//
// L work-items hold a row (norm_rows.h), which is read once: o waits in registers for
// its mean square, h for its own, and y, where it is quantised with one scale for the
// row, for its largest value.
//
// Bound by memory: 16384 x 4096 bf16 with h, y in 8 bits and both kept copies 119 to 121 us, 5.1
// TB/s of its 611 MB, more than half of them written (fp16 121, fp32 217); with h and y in 8-bit
// integers alone 88, 5.3 TB/s; 8192 x 8192 128, 4096 x 16384 144, 2048 x 32768 137, packed rows
// of 4095 153.  A row in registers from its first read to its last output is what keeps it to
// one pass.  One row 5.1 us: a trip to memory, two sums over the workgroup and the launch.
#include "norm_internal.h"
#include "norm_rows.h"

namespace sgemm {
namespace {

// Zeros past the row's end, at the cost of a branch in the wavefronts that do not reach it.
__device__ __forceinline__ void zero_past(float (&v)[8], int c, int cols)
{
    if (__ballot(c + 8 > cols)) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = c + j < cols ? v[j] : 0.0f;
    }
}

// The largest |v| as bits, by the maximum that carries a NaN through, whose operands take an
// absolute value for nothing.
__device__ __forceinline__ uint32_t abs_maximum8(const float (&v)[8])
{
    float m = fabsf(v[0]);
#pragma unroll
    for (int j = 1; j < 8; ++j)
        m = __builtin_elementwise_maximum(m, fabsf(v[j]));
    return abs_bits(m);
}

// 8 values in e4m3 with the scale of their block of 128 columns, which 16 consecutive
// lanes hold (zero past the row's end).
__device__ __forceinline__ void put_block8(uint8_t *row, float *scale_row, int64_t lds, int c, int cols,
                                           const float (&v)[8])
{
    float inv, scale;
    block_scale<0>(max16(abs_maximum8(v)), inv, scale);
    if (c < cols) {
        const uint32_t lo = f8_pack4<0>(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
        const uint32_t hi = f8_pack4<0>(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
        row_store8b(row, c, cols, lo, hi);
        if ((threadIdx.x & 15) == 0)
            scale_row[(int64_t)(c / F8_BLOCK) * lds] = scale;
    }
}

// The workgroup's place among the rows: runs of 32 rows, whose scales of one block share a
// line, go to one XCD (workgroups go to the 8 in turn), as far as there are whole rounds.
template <int ROWS> __device__ __forceinline__ int64_t workgroup_rows()
{
    constexpr int RUN = ROWS >= 32 ? 1 : 32 / ROWS;
    const uint32_t b = blockIdx.x, round = b / (8 * RUN);
    if ((round + 1) * (8 * RUN) > gridDim.x)
        return b;
    return (int64_t)round * (8 * RUN) + b % 8 * RUN + b / 8 % RUN;
}

template <typename T, int NT, int L, int V>
__global__ __launch_bounds__(NT) void block_norm_kernel(BlockNormArgs g)
{
    __shared__ float slot[2][NT / 64];
    __shared__ uint32_t top[NT / 64];
    const int lane = threadIdx.x % L;                                    // of the row's
    const int64_t row = workgroup_rows<NT / L>() * (NT / L) + threadIdx.x / L;
    if (row >= g.rows)
        return;  // whole rows of lanes, and only where no row needs the workgroup
    typedef typename Elt<T>::Raw Raw;
    Raw x[V], o[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = 8 * (lane + L * i);
        x[i] = row_raw8<true>(static_cast<const T *>(g.X) + row * g.ldx, c, g.cols);
        if (g.O)
            o[i] = row_raw8<true>(static_cast<const T *>(g.O) + row * g.ldo, c, g.cols);
    }
    float h[V][8];
    if (g.O) {
        float rstd_post = 1.0f;
        if (g.WP) {
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    ss = fmaf((float)o[i][j], (float)o[i][j], ss);
            ss = row_sum<NT, L>(ss, slot[0]);
            rstd_post = 1.0f / sqrtf(ss / (float)g.cols + g.eps);
            if (g.rstd_post && lane == 0)
                g.rstd_post[row] = rstd_post;
        }
        const int64_t at = g.G ? (int64_t)((uint32_t)row / (uint32_t)g.gate_rows) * g.ldg : 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = 8 * (lane + L * i);
            float v[8], w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = (float)o[i][j];
            if (g.O8)
                put_block8(g.O8 + row * g.ldo8, g.SO + row, g.ldso, c, g.cols, v);
            if (g.WP) {
                load_w8<T>(g.WP, g.w_f32, c, g.cols, w);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] = v[j] * rstd_post * w[j];
            }
            if (g.G) {
                load_w8<T>(static_cast<const uint8_t *>(g.G) + at * (g.w_f32 ? 4 : (int)sizeof(T)), g.w_f32, c, g.cols, w);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] *= w[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                h[i][j] = fmaf(g.alpha, (float)x[i][j], v[j]);
            zero_past(h[i], c, g.cols);  // (v may be NaN there)
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                h[i][j] = g.alpha * (float)x[i][j];
    }
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = 8 * (lane + L * i);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            ss = fmaf(h[i][j], h[i][j], ss);
        if (g.H && c < g.cols)
            row_store8(static_cast<T *>(g.H) + row * g.ldh, c, g.cols, h[i]);
        if (g.H8)
            put_block8(g.H8 + row * g.ldh8, g.SH + row, g.ldsh, c, g.cols, h[i]);
    }
    if (!g.Y && !g.Q && !g.rstd)
        return;
    ss = row_sum<NT, L>(ss, slot[1]);
    const float rstd = 1.0f / sqrtf(ss / (float)g.cols + g.eps);
    if (g.rstd && lane == 0)
        g.rstd[row] = rstd;
    if (!g.Y && !g.Q)
        return;
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = 8 * (lane + L * i);
        float w[8];
        load_w8<T>(g.W, g.w_f32, c, g.cols, w);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            h[i][j] = h[i][j] * rstd * w[j];
        zero_past(h[i], c, g.cols);
        if (g.Y && c < g.cols)
            row_store8(static_cast<T *>(g.Y) + row * g.ldy, c, g.cols, h[i]);
        if (g.Q && g.q_i8)
            m = max(m, abs_maximum8(h[i]));
        else if (g.Q)
            put_block8(g.Q + row * g.ldq, g.S + row, g.lds, c, g.cols, h[i]);
    }
    if (!g.Q || !g.q_i8)
        return;
    float inv, scale;
    i8_scale(row_max<NT, L>(m, top), inv, scale);
    if (lane == 0)
        g.S[row] = scale;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = 8 * (lane + L * i);
        if (c >= g.cols)
            continue;
        int q[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            q[j] = i8_round(h[i][j] * inv);
        row_store8b(g.Q + row * g.ldq, c, g.cols, i8_pack4(q[0], q[1], q[2], q[3]), i8_pack4(q[4], q[5], q[6], q[7]));
    }
}

struct Launch {
    const BlockNormArgs &a;
    hipStream_t s;
    template <typename T, int NT, int L, int V> void run()
    {
        block_norm_kernel<T, NT, L, V><<<(unsigned)ceil_div(a.rows, NT / L), NT, 0, s>>>(a);
    }
};

}  // namespace

hipError_t launch_block_norm(const BlockNormArgs &a, int type, hipStream_t s)
{
    by_type(type, a.cols, Launch{a, s});
    return hipGetLastError();
}

}  // namespace sgemm
