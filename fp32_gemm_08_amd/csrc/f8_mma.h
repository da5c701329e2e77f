// Device helpers of the 8-bit products: the matrix instructions over one k-block
// and the loads of operand rows at any alignment.
#pragma once
#include "f8_types.h"

#include <type_traits>

namespace sgemm {

// A lane's 32 values of one row: as they are (EXACT = false), or as bf16.
template <int FMT, bool EXACT> struct Frag;
template <int FMT> struct Frag<FMT, false> {
    f8_i32x8 v;
    __device__ __forceinline__ void set(const f8_i32x8 &x) { v = x; }
};
template <int FMT> struct Frag<FMT, true> {
    f8_b8 v[4];
    static __device__ __forceinline__ void eight(int a, int b, f8_b8 &o)
    {
        typedef __bf16 b2 __attribute__((ext_vector_type(2)));
        b2 p[4];
        if constexpr (FMT == 0) {
            p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)a, 1.0f, false);
            p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)a, 1.0f, true);
            p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)b, 1.0f, false);
            p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)b, 1.0f, true);
        } else {
            p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((unsigned)a, 1.0f, false);
            p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((unsigned)a, 1.0f, true);
            p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((unsigned)b, 1.0f, false);
            p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((unsigned)b, 1.0f, true);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[2 * i] = p[i][0];
            o[2 * i + 1] = p[i][1];
        }
    }
    __device__ __forceinline__ void set(const f8_i32x8 &x)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            eight(x[2 * i], x[2 * i + 1], v[i]);
    }
};

// A lane's two chunks of a row as one operand.
__device__ __forceinline__ f8_i32x8 f8_join(f8_i32x4 lo, f8_i32x4 hi)
{
    return f8_i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}

// The 128 products of a 16 x 16 block's k-block.
template <int FA, int FB>
__device__ __forceinline__ f8_f32x4 f8_mma(const Frag<FB, false> &b, const Frag<FA, false> &a)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b.v, a.v, f8_f32x4{}, FB, FA, 0, 0, 0, 0);
}
template <int FA, int FB>
__device__ __forceinline__ f8_f32x4 f8_mma(const Frag<FB, true> &b, const Frag<FA, true> &a)
{
    f8_f32x4 t{};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b.v[i], a.v[i], t, 0, 0, 0);
    return t;
}

// A quarter of them, added to t.
template <int PART, int FA, int FB>
__device__ __forceinline__ f8_f32x4 f8_mma_part(const Frag<FB, true> &b, const Frag<FA, true> &a, f8_f32x4 t)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(b.v[PART], a.v[PART], t, 0, 0, 0);
}

// 16 bytes of a row at any byte address, of which the first `valid` count (the
// rest read as zero): whole aligned words, of which only those that hold a
// counted byte are read, shifted into place.
__device__ __forceinline__ f8_i32x4 load16_any(const uint8_t *p, int valid)
{
    f8_i32x4 v{};
    if (valid <= 0)
        return v;
    const int sh = (int)(reinterpret_cast<uintptr_t>(p) & 3);
    const uint32_t *q = reinterpret_cast<const uint32_t *>(p - sh);
    uint32_t d[5];
#pragma unroll
    for (int i = 0; i < 5; ++i)
        d[i] = 4 * i < sh + valid ? q[i] : 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t x = __builtin_amdgcn_alignbyte(d[i + 1], d[i], sh);
        const int keep = valid - 4 * i;  // bytes of this word that count
        v[i] = (int)(keep >= 4 ? x : keep <= 0 ? 0u : x & (0xffffffffu >> (8 * (4 - keep))));
    }
    return v;
}

// The first `valid` bytes of 16, the others zero.
__device__ __forceinline__ f8_i32x4 keep16(f8_i32x4 x, int valid)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int keep = valid - 4 * i;
        x[i] = keep >= 4 ? x[i] : keep <= 0 ? 0 : (int)((uint32_t)x[i] & (0xffffffffu >> (8 * (4 - keep))));
    }
    return x;
}

// Host side.  The variant of a kernel for a call's formats, B blocks, alignment and type
// of C: f is called with the template arguments as integral constants.
template <bool V> using Bool = std::integral_constant<bool, V>;
template <int V> using Int = std::integral_constant<int, V>;
template <class F> inline void on_bool(bool v, F f) { v ? f(Bool<true>{}) : f(Bool<false>{}); }
template <class F> inline void on_format(int v, F f) { v == SGEMM_F8_E4M3 ? f(Int<0>{}) : f(Int<1>{}); }

}  // namespace sgemm
