// Backward pass of the norms around a block: who takes which rows, and the joining of
// the sums over rows.
#include "block_norm_bwd.h"

#include <algorithm>

namespace sgemm {
namespace {

template <typename T> __device__ __forceinline__ float weight(const void *W, int64_t at, int w_f32)
{
    return !W ? 1.0f : w_f32 ? static_cast<const float *>(W)[at] : (float)static_cast<const T *>(W)[at];
}

// Sum over `n` arrays of g.cols floats from `from` on, `step` apart, of column c: STRIPS of
// them per workgroup of COLS columns, 16 loads of a strip at a time (their latency is this
// kernel's time), joined through the LDS; complete in strip 0.
template <int COLS, int STRIPS>
__device__ __forceinline__ float column_sum(const float *from, int64_t step, int n, int c, bool live,
                                            float (&part)[STRIPS][COLS + 1])
{
    const int x = threadIdx.x % COLS, y = threadIdx.x / COLS;
    float s = 0.0f;
    if (live)
        for (int i = y; i < n; i += 16 * STRIPS) {
            float v[16];
#pragma unroll
            for (int j = 0; j < 16; ++j)
                v[j] = i + STRIPS * j < n ? from[(i + STRIPS * j) * step + c] : 0.0f;
#pragma unroll
            for (int j = 0; j < 16; ++j)
                s += v[j];
        }
    __syncthreads();
    part[y][x] = s;
    __syncthreads();
    s = 0.0f;
    if (y == 0)
#pragma unroll
        for (int i = 0; i < STRIPS; ++i)
            s += part[i][x];
    return s;
}

// COLS columns per workgroup.  blockIdx.y: 0 dw; 1 dw_post; from 2 on the gates whose sums
// several workgroups or walkers left, `gates` of them to be looked at
// (block_norm_gates_to_join): with teams and where a gate has more rows than a walker takes
// all gates, else by the walker in whose last row one is.
template <typename T, int COLS, int STRIPS>
__global__ __launch_bounds__(COLS *STRIPS) void block_norm_sums_kernel(BlockNormBwdArgs g, int gates)
{
    __shared__ float part[STRIPS][COLS + 1];
    const int c = blockIdx.x * COLS + threadIdx.x % COLS;
    const bool live = c < g.cols, writes = live && threadIdx.x < COLS;
    const float *second = g.ws + (int64_t)g.groups * g.cols;
    if (blockIdx.y == 0) {
        if (g.DW) {
            const float s = column_sum<COLS, STRIPS>(g.ws, g.cols, g.groups, c, live, part);
            if (writes)
                g.DW[c] = s;
        }
    } else if (blockIdx.y == 1) {
        if (g.DWP) {
            // gate d m, or d m where there is one gate
            const bool one = g.team == g.groups;
            const float s = column_sum<COLS, STRIPS>(g.team && !one ? second + (int64_t)g.groups * g.cols : second, g.cols, g.groups, c, live,
                                       part);
            if (writes)
                g.DWP[c] = one ? s * weight<T>(g.G, c, g.w_f32) : s;
        }
    } else {
        for (int i = blockIdx.y - 2; i < gates; i += gridDim.y - 2) {
            if (g.team) {
                const float s = column_sum<COLS, STRIPS>(second + (int64_t)i * g.team * g.cols, g.cols, g.team, c, live, part);
                if (writes)
                    g.DG[i * g.lddg + c] = s * weight<T>(g.WP, c, g.w_f32);
                continue;
            }
            const float *slots = second + (int64_t)g.groups * g.cols;
            const bool by_gate = g.gate_rows > g.chunk;
            const int64_t last = min<int64_t>(g.rows, (int64_t)(i + 1) * g.chunk) - 1;  // of walker i
            const int64_t gr = by_gate ? i : last / g.gate_rows;
            const int64_t first = gr * g.gate_rows, end = min<int64_t>(g.rows, first + g.gate_rows);
            const int from = (int)(first / g.chunk), to = (int)((end - 1) / g.chunk);     // its walkers
            if (from == to || (!by_gate && from != i))
                continue;
            float s = column_sum<COLS, STRIPS>(slots + (2 * (int64_t)from + 2) * g.cols, 2 * (int64_t)g.cols, to - from, c, live, part);
            if (writes) {
                // `first` is not the walker's first row: the slot of its last gate row
                s += slots[(2 * (int64_t)from + (first > (int64_t)from * g.chunk)) * g.cols + c];
                g.DG[gr * g.lddg + c] = s * weight<T>(g.WP, c, g.w_f32);
            }
        }
    }
}

// 8 wavefronts per CU (8 / 16: 16384 x 4096 bf16 142 / 144 us, 16384 x 1000 43.5 / 49.4), 16 of
// rows that take them.  Past one workgroup to a CU each takes four rows at least: the second
// kernel adds fewer sums (one row / two / four / eight: 1000 x 1017 fp32 15.7 / 13.8 / 14.0 /
// 14.0 us, 2000 x 1017 19.0 / 18.7 / 17.2 / 19.2, 1000 x 2000 16.2 / 16.1 / 14.8 / 14.8).
// Up to a quarter as many gates as workgroups get a team each, of equal size.
struct Walkers {
    int64_t rows, gate_rows;
    BlockNormSums *out;
    template <typename T, int NT, int L, int V> void run()
    {
        constexpr int64_t ROWS = NT / L, MOST = std::max(256 * 512 / NT, 256);
        const int64_t gates = ceil_div(rows, gate_rows);
        if (gates <= MOST / 4) {
            const int64_t most = std::min(MOST, std::max<int64_t>(256, ceil_div(rows, 4 * ROWS)));
            out->team = std::min(std::max<int64_t>(most / gates, 1), ceil_div(gate_rows, ROWS));
            out->groups = gates * out->team;
            out->parts = (gates > 1 ? 3 : 2) * out->groups;
        } else {
            out->chunk = ceil_div(rows, MOST * ROWS);
            out->walkers = ceil_div(rows, out->chunk);
            out->groups = ceil_div(out->walkers, ROWS);
            out->parts = 2 * out->groups + 2 * out->walkers;
        }
    }
};

// Of up to 256 arrays 8 strips of 64 columns, else 32 of 32 columns: the former are a quarter
// of the wavefronts (8 / 32 strips, both kernels: 16384 x 4096 with 8 gates, 256 arrays, 142 /
// 150 us, 16384 x 1000, 1024 arrays, 44.7 / 43.5).
template <typename T> void launch_sums(const BlockNormBwdArgs &a, int gates, hipStream_t s)
{
    const unsigned y = (unsigned)(2 + std::min(gates, 64));
    if (a.groups <= 256)
        block_norm_sums_kernel<T, 64, 8><<<dim3((unsigned)ceil_div(a.cols, 64), y), 512, 0, s>>>(a, gates);
    else
        block_norm_sums_kernel<T, 32, 32><<<dim3((unsigned)ceil_div(a.cols, 32), y), 1024, 0, s>>>(a, gates);
}

}  // namespace

BlockNormSums block_norm_sums(int64_t rows, int64_t cols, int64_t gate_rows)
{
    BlockNormSums n;
    if (rows > 0 && cols > 0)
        bwd_by_cols<float>((int)cols, Walkers{rows, gate_rows > 0 && gate_rows < rows ? gate_rows : rows, &n});
    return n;
}

hipError_t launch_block_norm_bwd(BlockNormBwdArgs a, int type, bool kept, hipStream_t s)
{
    const BlockNormSums n = block_norm_sums(a.rows, a.cols, a.gate_rows);
    a.groups = (int)n.groups;
    a.team = (int)n.team;
    a.chunk = (int)n.chunk;
    if (n.groups > 0) {
        if (type == SGEMM_TYPE_F32)
            launch_block_norm_bwd_rows<float>(a, kept, s);
        else if (type == SGEMM_TYPE_FP16)
            launch_block_norm_bwd_rows<_Float16>(a, kept, s);
        else
            launch_block_norm_bwd_rows<__bf16>(a, kept, s);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    const int64_t gates = a.DG ? block_norm_gates_to_join(n, a.rows, a.gate_rows) : 0;
    if (!a.DW && !a.DWP && gates == 0)
        return hipSuccess;
    if (type == SGEMM_TYPE_F32)
        launch_sums<float>(a, (int)gates, s);
    else if (type == SGEMM_TYPE_FP16)
        launch_sums<_Float16>(a, (int)gates, s);
    else
        launch_sums<__bf16>(a, (int)gates, s);
    return hipGetLastError();
}

}  // namespace sgemm
