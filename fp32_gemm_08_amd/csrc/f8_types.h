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
typedef f8_i32x4 f8_i32x4_any __attribute__((aligned(1)));
typedef _Float16 f8_h8 __attribute__((ext_vector_type(8)));
typedef __bf16 f8_b8 __attribute__((ext_vector_type(8)));

// A streaming store, of outputs in 16 and 8 bits: the line is not kept in the L2,
// where no other XCD could read it anyway.  STREAM loads likewise, of 16-bit rows
// that are read once.  Measured against ordinary accesses, inputs from memory: norm
// of 2048 x 4096 (bf16, all outputs) 17.0 -> 13.9 us, of 16384 x 4096 112.8 -> 105.2,
// its backward pass 102.0 -> 92.5, quantisation of 4096 x 4096 (fp32, tiles) 24.3 ->
// 17.9, a product's bf16 C of 8192 x 8192 (K = 1024) 95.8 -> 88.3; rows that share
// lines lose a little (backward of 65536 x 300 84.0 -> 88.4).  Those of 32-bit
// elements are ordinary: a lane's 32 bytes are two accesses that meet in one line
// (backward of 16384 x 4096 in fp32 197 against 229 us).
template <typename V> __device__ __forceinline__ void f8_stream(V v, void *p)
{
    typedef V Vany __attribute__((aligned(1)));
    __builtin_nontemporal_store(v, reinterpret_cast<Vany *>(p));
}

// Row elements: loads and stores of 8 consecutive ones as FP32.
template <typename T> struct Elt;
template <> struct Elt<float> {
    struct Raw {
        f8_f32x4 a, b;
        __device__ __forceinline__ float operator[](int i) const { return i < 4 ? a[i] : b[i - 4]; }
    };
    template <bool STREAM> static __device__ __forceinline__ Raw raw8(const float *p)
    {
        return {*reinterpret_cast<const f8_f32x4_any *>(p), *reinterpret_cast<const f8_f32x4_any *>(p + 4)};
    }
    static __device__ __forceinline__ void set(Raw &r, int i, float v) { i < 4 ? r.a[i] = v : r.b[i - 4] = v; }
    // Elements s .. 7 moved to the front, zeros behind them (s = 1 .. 7).
    static __device__ __forceinline__ Raw drop(Raw r, int s)
    {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = r[i];
#pragma unroll
        for (int step = 4; step; step >>= 1)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = s & step ? (i + step < 8 ? v[i + step] : 0.0f) : v[i];
        return {{v[0], v[1], v[2], v[3]}, {v[4], v[5], v[6], v[7]}};
    }
    // Elements at .. at+N-1 (N = 1, 2, 4) to p, unaligned.
    template <int N> static __device__ __forceinline__ void put_part(float *p, const float *v)
    {
        typedef float VN __attribute__((ext_vector_type(N == 1 ? 2 : N)));
        typedef VN VNany __attribute__((aligned(1)));
        if constexpr (N == 1) {
            *p = v[0];
        } else {
            VN o;
#pragma unroll
            for (int i = 0; i < N; ++i)
                o[i] = v[i];
            *reinterpret_cast<VNany *>(p) = o;
        }
    }
    static __device__ __forceinline__ void store8(float *p, const float (&v)[8])
    {
        *reinterpret_cast<f8_f32x4_any *>(p) = f8_f32x4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<f8_f32x4_any *>(p + 4) = f8_f32x4{v[4], v[5], v[6], v[7]};
    }
};
template <typename T, typename V8> struct Elt16 {
    typedef V8 Raw;
    typedef V8 V8any __attribute__((aligned(1)));  // (as a template argument it would lose the attribute)
    template <bool STREAM> static __device__ __forceinline__ Raw raw8(const T *p)
    {
        if constexpr (STREAM)
            return __builtin_nontemporal_load(reinterpret_cast<const V8any *>(p));
        else
            return *reinterpret_cast<const V8any *>(p);
    }
    static __device__ __forceinline__ void set(Raw &r, int i, T v) { r[i] = v; }
    static __device__ __forceinline__ Raw drop(Raw r, int s)
    {
        f8_u32x4 d;
        __builtin_memcpy(&d, &r, 16);
        uint32_t v[4] = {d[0], d[1], d[2], d[3]};
#pragma unroll
        for (int step = 2; step; step >>= 1)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = s & 2 * step ? (i + step < 4 ? v[i + step] : 0u) : v[i];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            d[i] = s & 1 ? __builtin_amdgcn_alignbit(i < 3 ? v[i + 1] : 0u, v[i], 16) : v[i];
        __builtin_memcpy(&r, &d, 16);
        return r;
    }
    template <int N> static __device__ __forceinline__ void put_part(T *p, const float *v)
    {
        typedef T VN __attribute__((ext_vector_type(N == 1 ? 2 : N)));
        typedef VN VNany __attribute__((aligned(1)));
        if constexpr (N == 1) {
            *p = (T)v[0];
        } else {
            VN o;
#pragma unroll
            for (int i = 0; i < N; ++i)
                o[i] = (T)v[i];
            *reinterpret_cast<VNany *>(p) = o;
        }
    }
    static __device__ __forceinline__ void store8(T *p, const float (&v)[8])
    {
        V8 a;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            a[i] = (T)v[i];
        f8_stream(a, p);
    }
};
template <> struct Elt<_Float16> : Elt16<_Float16, f8_h8> {};
template <> struct Elt<__bf16> : Elt16<__bf16, f8_b8> {};

// Elements c .. c+7 of a row of `cols`, zero past its end, unconverted (values
// requested ahead stay in as few registers as they have bytes).  The row's last
// piece, where it is shorter, is read as the row's last 8 elements and shifted.
template <bool STREAM, typename T>
__device__ __forceinline__ typename Elt<T>::Raw row_raw8(const T *row, int c, int cols)
{
    if (c + 8 <= cols)
        return Elt<T>::template raw8<STREAM>(row + c);
    typename Elt<T>::Raw r{};
    if (c < cols) {
        if (cols >= 8) {
            r = Elt<T>::drop(Elt<T>::template raw8<false>(row + cols - 8), c + 8 - cols);
        } else {
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (c + i < cols)
                    Elt<T>::set(r, i, row[c + i]);
        }
    }
    return r;
}
template <bool STREAM, typename T>
__device__ __forceinline__ void row_load8(const T *row, int c, int cols, float (&v)[8])
{
    const typename Elt<T>::Raw r = row_raw8<STREAM>(row, c, cols);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = (float)r[i];
}
// A shorter last piece is written as 4, 2 and 1 elements, where its length has them.
template <typename T>
__device__ __forceinline__ void row_store8(T *row, int c, int cols, const float (&v)[8])
{
    if (c + 8 <= cols) {
        Elt<T>::store8(row + c, v);
        return;
    }
    const int n = cols - c;
    if (n <= 0)
        return;
    T *p = row + c;
    float u[4] = {v[0], v[1], v[2], v[3]};
    if (n & 4) {
        Elt<T>::template put_part<4>(p, v);
        p += 4;
        u[0] = v[4], u[1] = v[5], u[2] = v[6];
    }
    if (n & 2) {
        Elt<T>::template put_part<2>(p, u);
        p += 2;
        u[0] = u[2];
    }
    if (n & 1)
        Elt<T>::template put_part<1>(p, u);
}
// The same for 8 bytes held in two words.
__device__ __forceinline__ void row_store8b(uint8_t *row, int c, int cols, uint32_t lo, uint32_t hi)
{
    typedef uint32_t u32_any __attribute__((aligned(1)));
    typedef uint16_t u16_any __attribute__((aligned(1)));
    if (c + 8 <= cols) {
        f8_stream(f8_u32x2{lo, hi}, row + c);
        return;
    }
    const int n = cols - c;
    if (n <= 0)
        return;
    uint8_t *p = row + c;
    if (n & 4) {
        *reinterpret_cast<u32_any *>(p) = lo;
        p += 4;
        lo = hi;
    }
    if (n & 2) {
        *reinterpret_cast<u16_any *>(p) = (uint16_t)lo;
        p += 2;
        lo >>= 16;
    }
    if (n & 1)
        *p = (uint8_t)lo;
}

// Bytes c .. c+7 of a row of `cols`, zero past its end; a shorter last piece as in row_raw8.
template <bool STREAM>
__device__ __forceinline__ f8_u32x2 row_raw8b(const uint8_t *row, int c, int cols)
{
    typedef f8_u32x2 u32x2_any __attribute__((aligned(1)));
    if (c + 8 <= cols) {
        const u32x2_any *p = reinterpret_cast<const u32x2_any *>(row + c);
        if constexpr (STREAM)
            return __builtin_nontemporal_load(p);
        else
            return *p;
    }
    uint64_t v = 0;
    if (c < cols) {
        if (cols >= 8) {
            const f8_u32x2 d = *reinterpret_cast<const u32x2_any *>(row + cols - 8);
            v = (d[0] | (uint64_t)d[1] << 32) >> (8 * (c + 8 - cols));
        } else {
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (c + i < cols)
                    v |= (uint64_t)row[c + i] << (8 * i);
        }
    }
    return f8_u32x2{(uint32_t)v, (uint32_t)(v >> 32)};
}
// The same in two steps, so that a load that is requested ahead is not waited for: of rows of
// at least 8 elements the row's last 8 where the piece at c is shorter or past the end, and,
// when they are used, the elements that are past the piece's start by `past` = c + 8 - cols
// moved to the front.
template <bool STREAM, typename T>
__device__ __forceinline__ typename Elt<T>::Raw row_any8(const T *row, int c, int cols)
{
    return Elt<T>::template raw8<STREAM>(row + min(c, cols - 8));
}
template <typename T> __device__ __forceinline__ void row_fix8(typename Elt<T>::Raw &r, int past)
{
    if (past >= 8)
        r = typename Elt<T>::Raw{};
    else if (past > 0)
        r = Elt<T>::drop(r, past);
}
template <bool STREAM> __device__ __forceinline__ f8_u32x2 row_any8b(const uint8_t *row, int c, int cols)
{
    return row_raw8b<STREAM>(row + min(c, cols - 8), 0, 8);
}
__device__ __forceinline__ void row_fix8b(f8_u32x2 &q, int past)
{
    if (past > 0) {
        const uint64_t v = past >= 8 ? 0 : (q[0] | (uint64_t)q[1] << 32) >> (8 * past);
        q = f8_u32x2{(uint32_t)v, (uint32_t)(v >> 32)};
    }
}
// What 8 bytes of that format stand for, without their scale.
template <int FMT>
__device__ __forceinline__ void f8_unpack8(f8_u32x2 q, float (&v)[8])
{
    typedef float f2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        f2 lo, hi;
        if constexpr (FMT == 0) {
            lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[i], false);
            hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[i], true);
        } else {
            lo = __builtin_amdgcn_cvt_pk_f32_bf8((int)q[i], false);
            hi = __builtin_amdgcn_cvt_pk_f32_bf8((int)q[i], true);
        }
        v[4 * i] = lo[0], v[4 * i + 1] = lo[1], v[4 * i + 2] = hi[0], v[4 * i + 3] = hi[1];
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

// The same for 8-bit integers with one scale.
__device__ __forceinline__ void i8_scale(uint32_t bits, float &inv, float &scale)
{
    const float a = __uint_as_float(max(bits, __float_as_uint(F8_FLOOR)));
    inv = 127.0f / a;
    scale = a / 127.0f;
}

// To the nearest integer, ties to even; NaN (of a row that holds one, or an infinity): 0.
__device__ __forceinline__ int i8_round(float t) { return (int)rintf(t == t ? t : 0.0f); }

__device__ __forceinline__ uint32_t i8_pack4(int a, int b, int c, int d)
{
    return ((uint32_t)a & 0xff) | ((uint32_t)b & 0xff) << 8 | ((uint32_t)c & 0xff) << 16 | (uint32_t)d << 24;
}

}  // namespace sgemm
