// Backward pass of the norms around a block: who takes which rows, and the joining of
// the sums over rows.
#include "block_norm_bwd.h"

#include <algorithm>

namespace sgemm {
namespace {

// Sum over `n` arrays of g.cols floats from `from` on, `step` apart, of column c: 32
// strips of them per workgroup, joined through the LDS; complete in strip 0.
__device__ __forceinline__ float column_sum(const float *from, int64_t step, int n, int c, bool live, float (&part)[32][33])
{
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    float s = 0.0f;
    if (live)
        for (int i = y; i < n; i += 8 * 32) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = i + 32 * j < n ? from[(i + 32 * j) * step + c] : 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                s += v[j];
        }
    __syncthreads();
    part[y][x] = s;
    __syncthreads();
    s = 0.0f;
    if (y == 0)
#pragma unroll
        for (int i = 0; i < 32; ++i)
            s += part[i][x];
    return s;
}

template <typename T> __device__ __forceinline__ float weight(const void *W, int64_t at, int w_f32)
{
    return !W ? 1.0f : w_f32 ? static_cast<const float *>(W)[at] : (float)static_cast<const T *>(W)[at];
}

// 32 columns per workgroup.  blockIdx.y: 0 dw; 1 dw_post, and the gate's gradient where it
// has one row; from 2 on the rows of the gate that several walkers share, `starts` of them
// to be looked at: by the gate's row where it has at least as many rows as a walker takes,
// else by the walker in whose last row it is.
template <typename T>
__global__ __launch_bounds__(1024) void block_norm_sums_kernel(BlockNormBwdArgs g, bool several, int walkers, int starts)
{
    __shared__ float part[32][33];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31);
    const bool live = c < g.cols, writes = live && threadIdx.x < 32;
    if (blockIdx.y == 0) {
        if (g.DW) {
            const float s = column_sum(g.ws, g.cols, g.groups, c, live, part);
            if (writes)
                g.DW[c] = s;
        }
    } else if (blockIdx.y == 1) {
        if (g.DWP || (!several && g.DG)) {
            const float s = column_sum(g.ws + (int64_t)g.groups * g.cols, g.cols, g.groups, c, live, part);
            if (writes && g.DWP)
                g.DWP[c] = several ? s : s * weight<T>(g.G, c, g.w_f32);
            if (writes && !several && g.DG)
                g.DG[c] = s * weight<T>(g.WP, c, g.w_f32);
        }
    } else {
        const float *slots = g.ws + 2 * (int64_t)g.groups * g.cols;
        for (int i = blockIdx.y - 2; i < starts; i += gridDim.y - 2) {
            const bool by_gate = g.gate_rows >= g.chunk;
            const int64_t last = min<int64_t>(g.rows, (int64_t)(i + 1) * g.chunk) - 1;  // of walker i
            const int64_t gr = by_gate ? i : last / g.gate_rows;
            const int64_t first = gr * g.gate_rows, end = min<int64_t>(g.rows, first + g.gate_rows);
            const int from = (int)(first / g.chunk), to = (int)((end - 1) / g.chunk);     // its walkers
            if (from == to || (!by_gate && from != i))
                continue;
            // `first` is not the walker's first row: the slot of its last gate row
            float s = column_sum(slots + (2 * (int64_t)from + 2) * g.cols, 2 * (int64_t)g.cols, to - from, c, live, part);
            if (writes) {
                s += slots[(2 * (int64_t)from + (first > (int64_t)from * g.chunk)) * g.cols + c];
                g.DG[gr * g.lddg + c] = s * weight<T>(g.WP, c, g.w_f32);
            }
        }
    }
}

// 8 wavefronts per CU.
struct Walkers {
    int64_t rows;
    BlockNormSums *out;
    template <typename T, int NT, int L, int V> void run()
    {
        constexpr int64_t ROWS = NT / L, MOST = std::max(256 * 512 / NT, 256);
        const int64_t all = MOST * ROWS;
        out->chunk = std::max<int64_t>(1, ceil_div(rows, all));
        out->groups = ceil_div(ceil_div(rows, out->chunk), ROWS);
        out->walkers = ceil_div(rows, out->chunk);
    }
};

}  // namespace

BlockNormSums block_norm_sums(int64_t rows, int64_t cols, int64_t gate_rows)
{
    BlockNormSums n;
    if (rows <= 0 || cols <= 0)
        return n;
    bwd_by_cols<float>((int)cols, Walkers{rows, &n});
    n.several = gate_rows > 0 && gate_rows < rows;
    n.parts = 2 * n.groups + (n.several ? 2 * n.walkers : 0);
    return n;
}

hipError_t launch_block_norm_bwd(BlockNormBwdArgs a, int type, bool kept, hipStream_t s)
{
    const BlockNormSums n = block_norm_sums(a.rows, a.cols, a.G ? a.gate_rows : a.rows);
    a.groups = (int)n.groups;
    a.chunk = (int)n.chunk;
    if (n.groups > 0) {
        if (type == SGEMM_TYPE_F32)
            launch_block_norm_bwd_rows<float>(a, kept, n.several, s);
        else if (type == SGEMM_TYPE_FP16)
            launch_block_norm_bwd_rows<_Float16>(a, kept, n.several, s);
        else
            launch_block_norm_bwd_rows<__bf16>(a, kept, n.several, s);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    if (!a.DW && !a.DWP && !a.DG)
        return hipSuccess;
    int64_t starts = 0;
    if (n.several && a.DG)
        starts = a.gate_rows >= n.chunk ? ceil_div(a.rows, a.gate_rows) : n.chunk % a.gate_rows ? n.walkers : 0;
    const dim3 grid((unsigned)ceil_div(a.cols, 32), (unsigned)(2 + std::min<int64_t>(starts, 64)));
    if (type == SGEMM_TYPE_F32)
        block_norm_sums_kernel<float><<<grid, 1024, 0, s>>>(a, n.several, (int)n.walkers, (int)starts);
    else if (type == SGEMM_TYPE_FP16)
        block_norm_sums_kernel<_Float16><<<grid, 1024, 0, s>>>(a, n.several, (int)n.walkers, (int)starts);
    else
        block_norm_sums_kernel<__bf16><<<grid, 1024, 0, s>>>(a, n.several, (int)n.walkers, (int)starts);
    return hipGetLastError();
}

}  // namespace sgemm
