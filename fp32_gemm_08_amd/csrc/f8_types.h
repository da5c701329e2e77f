// Device helpers of the 8-bit block-scaled family: element types, 8-bit
// rounding and the block maximum.
#pragma once
#include <hip/hip_runtime.h>

#include "f8_internal.h"

namespace sgemm {

typedef float f8_f32x4 __attribute__((ext_vector_type(4)));
typedef int f8_i32x4 __attribute__((ext_vector_type(4)));
typedef int f8_i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t f8_u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t f8_u32x4 __attribute__((ext_vector_type(4)));

// Formats: 0 = e4m3, 1 = e5m2 (the matrix instruction's own numbering).
template <int FMT> __device__ __forceinline__ constexpr float f8_largest() { return FMT == 0 ? 448.0f : 57344.0f; }

// Four values rounded to 8 bits (to nearest, ties to even), value i in byte i.
// The values are within the format's range by construction (or NaN).
template <int FMT>
__device__ __forceinline__ uint32_t f8_pack4(float a, float b, float c, float d)
{
    if constexpr (FMT == 0) {
        const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true);
    } else {
        const int lo = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, 0, false);
        return (uint32_t)__builtin_amdgcn_cvt_pk_bf8_f32(c, d, lo, true);
    }
}

// Vectors at any address: the hardware's global loads and stores of up to 16
// bytes take every byte alignment, so rows that start anywhere are accessed whole.
typedef f8_f32x4 f8_f32x4_any __attribute__((aligned(1)));
typedef f8_u32x2 f8_u32x2_any __attribute__((aligned(1)));
typedef _Float16 f8_h8 __attribute__((ext_vector_type(8)));
typedef __bf16 f8_b8 __attribute__((ext_vector_type(8)));
typedef f8_h8 f8_h8_any __attribute__((aligned(1)));
typedef f8_b8 f8_b8_any __attribute__((aligned(1)));

// Row elements: loads and stores of 8 consecutive ones as FP32.
template <typename T> struct Elt;
template <> struct Elt<float> {
    struct Raw {
        f8_f32x4 a, b;
        __device__ __forceinline__ float operator[](int i) const { return i < 4 ? a[i] : b[i - 4]; }
    };
    static __device__ __forceinline__ Raw raw8(const float *p)
    {
        return {*reinterpret_cast<const f8_f32x4_any *>(p), *reinterpret_cast<const f8_f32x4_any *>(p + 4)};
    }
    static __device__ __forceinline__ void set(Raw &r, int i, float v) { i < 4 ? r.a[i] = v : r.b[i - 4] = v; }
    static __device__ __forceinline__ void load8(const float *p, float (&v)[8])
    {
        const f8_f32x4 a = *reinterpret_cast<const f8_f32x4_any *>(p), b = *reinterpret_cast<const f8_f32x4_any *>(p + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = a[i];
            v[4 + i] = b[i];
        }
    }
    static __device__ __forceinline__ void store8(float *p, const float (&v)[8])
    {
        *reinterpret_cast<f8_f32x4_any *>(p) = f8_f32x4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<f8_f32x4_any *>(p + 4) = f8_f32x4{v[4], v[5], v[6], v[7]};
    }
    static __device__ __forceinline__ float get(const float *p) { return *p; }
    static __device__ __forceinline__ void put(float *p, float v) { *p = v; }
};
template <typename T, typename V8, typename V8any> struct Elt16 {
    typedef V8 Raw;
    static __device__ __forceinline__ Raw raw8(const T *p) { return *reinterpret_cast<const V8any *>(p); }
    static __device__ __forceinline__ void set(Raw &r, int i, T v) { r[i] = v; }
    static __device__ __forceinline__ void load8(const T *p, float (&v)[8])
    {
        const V8 a = *reinterpret_cast<const V8any *>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = (float)a[i];
    }
    static __device__ __forceinline__ void store8(T *p, const float (&v)[8])
    {
        V8 a;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            a[i] = (T)v[i];
        *reinterpret_cast<V8any *>(p) = a;
    }
    static __device__ __forceinline__ float get(const T *p) { return (float)*p; }
    static __device__ __forceinline__ void put(T *p, float v) { *p = (T)v; }
};
template <> struct Elt<_Float16> : Elt16<_Float16, f8_h8, f8_h8_any> {};
template <> struct Elt<__bf16> : Elt16<__bf16, f8_b8, f8_b8_any> {};

// Elements c .. c+7 of a row of `cols`, zero past its end.
template <typename T>
__device__ __forceinline__ void row_load8(const T *row, int c, int cols, float (&v)[8])
{
    if (c + 8 <= cols) {
        Elt<T>::load8(row + c, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = c + i < cols ? Elt<T>::get(row + c + i) : 0.0f;
    }
}
// The same, unconverted (values requested ahead stay in as few registers as they have bytes).
template <typename T>
__device__ __forceinline__ typename Elt<T>::Raw row_raw8(const T *row, int c, int cols)
{
    if (c + 8 <= cols)
        return Elt<T>::raw8(row + c);
    typename Elt<T>::Raw r{};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c + i < cols)
            Elt<T>::set(r, i, row[c + i]);
    return r;
}
template <typename T>
__device__ __forceinline__ void row_store8(T *row, int c, int cols, const float (&v)[8])
{
    if (c + 8 <= cols) {
        Elt<T>::store8(row + c, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < cols)
                Elt<T>::put(row + c + i, v[i]);
    }
}
// The same for 8 bytes held in two words.
__device__ __forceinline__ void row_store8b(uint8_t *row, int c, int cols, uint32_t lo, uint32_t hi)
{
    if (c + 8 <= cols) {
        *reinterpret_cast<f8_u32x2_any *>(row + c) = f8_u32x2{lo, hi};
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < cols)
                row[c + i] = (uint8_t)((i < 4 ? lo >> (8 * i) : hi >> (8 * (i - 4))) & 0xff);
    }
}

// |x| as an unsigned number: ordered as |x| is, infinity above every finite
// value and NaN above infinity, so that an integer maximum carries a NaN
// through (the FP32 maximum instruction drops it).
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

__device__ __forceinline__ uint32_t abs_max8(const float (&v)[8])
{
    uint32_t m = abs_bits(v[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i)
        m = max(m, abs_bits(v[i]));
    return m;
}

// Maximum over each aligned group of 16 lanes, in every lane of the group: a
// butterfly of data-parallel primitives (swap pairs, swap pairs of two, mirror
// the half row, mirror the row).
__device__ __forceinline__ uint32_t max16(uint32_t m)
{
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xf, 0xf, false));   // quad_perm 1,0,3,2
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xf, 0xf, false));   // quad_perm 2,3,0,1
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x141, 0xf, 0xf, false));  // row_half_mirror
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x140, 0xf, 0xf, false));  // row_mirror
    return m;
}

// Sum over each aligned group of L lanes (16, 32 or 64), in every lane of the
// group: the same butterfly, and exchanges between the groups of 16.
template <int L>
__device__ __forceinline__ float lanes_sum(float v)
{
    static_assert(L == 16 || L == 32 || L == 64, "whole groups of 16 lanes");
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xf, 0xf, false));
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xf, 0xf, false));
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xf, 0xf, false));
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x140, 0xf, 0xf, false));
    if constexpr (L >= 32)
        v += __shfl_xor(v, 16);
    if constexpr (L == 64)
        v += __shfl_xor(v, 32);
    return v;
}

// A block's maximum (as bits) -> the factor that quantises it and its scale.
template <int FMT>
__device__ __forceinline__ void block_scale(uint32_t bits, float &inv, float &scale)
{
    const float a = __uint_as_float(max(bits, __float_as_uint(F8_FLOOR)));
    inv = f8_largest<FMT>() / a;
    scale = a / f8_largest<FMT>();
}

}  // namespace sgemm
