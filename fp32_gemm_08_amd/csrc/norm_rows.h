// Rows held in registers by 16 to 1024 work-items: what the norms and the quantisation
// by rows share.
#pragma once
#include "f8_types.h"

namespace sgemm {
namespace {

// Sum of `v` over the work-items of a row, in every one of them.  `slot` has
// NT/64 floats that no other sum uses at the same time.
template <int NT, int L>
__device__ __forceinline__ float row_sum(float v, float *slot)
{
    if constexpr (L <= 64)
        return lanes_sum<L>(v);
    static_assert(L <= 64 || L == NT, "a row of several wavefronts is the workgroup's only one");
    v = lanes_sum<64>(v);
    if ((threadIdx.x & 63) == 0)
        slot[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i)
        v += slot[i];
    return v;
}

// Largest `m` (as bits, see abs_bits) over the work-items of a row, in every one of them.
template <int NT, int L>
__device__ __forceinline__ uint32_t row_max(uint32_t m, uint32_t *slot)
{
    m = max16(m);
    if constexpr (L >= 32)
        m = max(m, (uint32_t)__shfl_xor((int)m, 16));
    if constexpr (L >= 64)
        m = max(m, (uint32_t)__shfl_xor((int)m, 32));
    if constexpr (L <= 64)
        return m;
    if ((threadIdx.x & 63) == 0)
        slot[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NT / 64; ++i)
        m = max(m, slot[i]);
    return m;
}

template <typename T>
__device__ __forceinline__ void load_w8(const void *W, int w_f32, int c, int cols, float (&v)[8])
{
    if (w_f32)
        row_load8<false>(static_cast<const float *>(W), c, cols, v);
    else
        row_load8<false>(static_cast<const T *>(W), c, cols, v);
}

// Calls f.run<T, NT, L, V> with what covers `cols`: work-items of a workgroup
// and of a row, and pieces per work-item.
template <typename T, typename F>
void by_cols(int cols, F f)
{
    if (cols <= 128)
        f.template run<T, 256, 16, 1>();
    else if (cols <= 256)
        f.template run<T, 256, 32, 1>();
    else if (cols <= 512)
        f.template run<T, 256, 64, 1>();
    else if (cols <= 1024)
        f.template run<T, 256, 64, 2>();
    else if (cols <= 2048)
        f.template run<T, 256, 256, 1>();
    else if (cols <= 4096)
        f.template run<T, 256, 256, 2>();
    else if (cols <= 8192)
        f.template run<T, 512, 512, 2>();
    else if (cols <= 16384)
        f.template run<T, 1024, 1024, 2>();
    else
        f.template run<T, 1024, 1024, 4>();
}

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
}  // namespace sgemm
