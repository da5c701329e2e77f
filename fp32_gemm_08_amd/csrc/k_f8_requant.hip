// Values kept in 8 bits with row blocks, laid out with blocks along the columns and
// transposed: x = fl(q * s),  a = max(max|x| over 128 rows of a column, 2^-90),
// q' = rne8(x * (L / a)),  s' = a / L.
//
// A wavefront has a tile of 128 rows and 64 columns for itself, lane l the rows 16 (l / 8)
// .. +15 and the columns 8 (l % 8) .. +7 of it: 16 loads of 8 bytes, 8 lanes to a row.  The
// tile stays in registers as bytes and is turned into numbers twice, for the maxima and for
// the output, 16 consecutive bytes of each of a lane's 8 columns.  A column's maximum is over
// the 8 lanes that share it: with each exchange a lane keeps half of its columns, so that it
// ends with the complete maximum of one and divides for one; the factors come back the same
// way.  No barrier, and the LDS's crossbar only for the order in which lanes write.
//
// Bound by memory: 16384 x 4096 23.5 to 25.6 us, 5.9 TB/s (as an input of k_f8_quant.hip, a 128
// x 128 tile through the LDS, 45.1).  Without the swap of lanes before the stores, whose
// neighbouring lanes then write to different lines, 37.4; with the loads past the L2 too, which
// a line's two halves meet in, 47.4 with a wavefront a workgroup.
#include "f8_types.h"

namespace sgemm {
namespace {

typedef uint32_t u2 __attribute__((ext_vector_type(2)));

// The lanes' halves by bit `bit` (32 or 16) of the lane: x of the lower half beside y's lower
// half (in place of x's upper), y of the upper half beside x's upper.
template <int BIT> __device__ __forceinline__ void trade(uint32_t &x, uint32_t &y)
{
    u2 r;
    if constexpr (BIT == 32)
        r = __builtin_amdgcn_permlane32_swap(x, y, false, false);
    else
        r = __builtin_amdgcn_permlane16_swap(x, y, false, false);
    x = r[0];
    y = r[1];
}
// The lane 8 further of its row of 16.
__device__ __forceinline__ uint32_t beside(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xf, 0xf, false);  // row_ror:8
}

// v of the lane 8 (l % 8) + l / 8.
__device__ __forceinline__ uint32_t swapped(uint32_t v, int l)
{
    return (uint32_t)__builtin_amdgcn_ds_bpermute(4 * (8 * (l % 8) + l / 8), (int)v);
}
// Two neighbouring values of 8 bytes, the first at the even place j.
template <int FX> __device__ __forceinline__ void two(f8_u32x2 q, int j, float &a, float &b)
{
    typedef float f2 __attribute__((ext_vector_type(2)));
    const int w = (int)q[j / 4];
    f2 v;
    if constexpr (FX == 0)
        v = j & 2 ? __builtin_amdgcn_cvt_pk_f32_fp8(w, true) : __builtin_amdgcn_cvt_pk_f32_fp8(w, false);
    else
        v = j & 2 ? __builtin_amdgcn_cvt_pk_f32_bf8(w, true) : __builtin_amdgcn_cvt_pk_f32_bf8(w, false);
    a = v[0];
    b = v[1];
}

template <int W, int FX, int FMT>
__global__ __launch_bounds__(64 * W) void f8_requantize_kernel(F8QuantArgs g)
{
    const int lane = threadIdx.x & 63, part = lane / 8;
    const int tr = blockIdx.x / g.tiles_c, tc = W * (blockIdx.x % g.tiles_c) + threadIdx.x / 64;
    if (tc * 64 >= g.cols)
        return;  // (the whole wavefront: the last workgroup of a row of tiles may have too many)
    const int r0 = tr * 128 + 16 * part, c = tc * 64 + 8 * (lane % 8);

    f8_u32x2 raw[16];
    float s[16];
    const float *sx = g.SX + (int64_t)(tc / 2) * g.ldsx;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int r = r0 + i;
        raw[i] = r < g.rows && c < g.cols
                     ? row_raw8b<false>(static_cast<const uint8_t *>(g.X) + (int64_t)r * g.ldx, c, g.cols)
                     : f8_u32x2{0, 0};
    }
    if (r0 + 16 <= g.rows) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f8_f32x4 v = *reinterpret_cast<const f8_f32x4_any *>(sx + r0 + 4 * i);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                s[4 * i + j] = v[j];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            s[i] = r0 + i < g.rows ? sx[r0 + i] : 0.0f;
    }

    uint32_t m[8] = {};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float v[8];
        f8_unpack8<FX>(raw[i], v);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            m[j] = max(m[j], abs_bits(v[j] * s[i]));
    }
    // lanes l and l ^ 32: columns 0-3 to the lower half, 4-7 to the upper
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        trade<32>(m[j], m[j + 4]);
        m[j] = max(m[j], m[j + 4]);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        trade<16>(m[j], m[j + 2]);
        m[j] = max(m[j], m[j + 2]);
    }
    const bool upper = lane & 8;
    const uint32_t away = upper ? m[0] : m[1];
    const uint32_t top = max(upper ? m[1] : m[0], beside(away));
    // this lane's column: of its 8, number 4 (bit 32) + 2 (bit 16) + (bit 8)
    float inv, scale;
    block_scale<FMT>(top, inv, scale);
    const int own = c + 4 * (lane >> 5 & 1) + 2 * (lane >> 4 & 1) + (lane >> 3 & 1);
    if (own < g.cols)
        g.ST[(int64_t)tr * g.ldst + own] = scale;
    uint32_t f[8];
    const uint32_t mine = __float_as_uint(inv), other = beside(mine);
    f[0] = upper ? other : mine;
    f[1] = upper ? mine : other;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        f[j + 2] = f[j];
        trade<16>(f[j], f[j + 2]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[j + 4] = f[j];
        trade<32>(f[j], f[j + 4]);
    }

    // the bytes are turned into numbers again: the compiler would keep all of those
#pragma unroll
    for (int i = 0; i < 16; ++i)
        asm volatile("" : "+v"(raw[i][0]), "+v"(raw[i][1]));
    // the 16 rows of a column, two columns at a time; lane l then takes what the lane with its
    // two places swapped has, so that 8 lanes beside each other write 128 bytes of one column
    const int out_c = tc * 64 + 8 * part, out_r = tr * 128 + 16 * (lane % 8);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const float f0 = __uint_as_float(f[j]), f1 = __uint_as_float(f[j + 1]);
        uint32_t q0[4], q1[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float a[4], b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                two<FX>(raw[4 * k + i], j, a[i], b[i]);
                a[i] = a[i] * s[4 * k + i] * f0;
                b[i] = b[i] * s[4 * k + i] * f1;
            }
            q0[k] = swapped(f8_pack4<FMT>(a[0], a[1], a[2], a[3]), lane);
            q1[k] = swapped(f8_pack4<FMT>(b[0], b[1], b[2], b[3]), lane);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            if (out_c + j + x >= g.cols || out_r >= g.rows)
                continue;
            const uint32_t *q = x ? q1 : q0;
            uint8_t *p = g.QT + (int64_t)(out_c + j + x) * g.ldqt + out_r;
            if (out_r + 16 <= g.rows) {
                f8_stream(f8_u32x4{q[0], q[1], q[2], q[3]}, p);
            } else {
                row_store8b(p, 0, min(g.rows - out_r, 8), q[0], q[1]);
                row_store8b(p, 8, g.rows - out_r, q[2], q[3]);
            }
        }
    }
}

template <int W>
void launch_tiles(F8QuantArgs a, int format_x, int format, hipStream_t s)
{
    const int64_t tr = ((int64_t)a.rows + 127) / 128, tc = ((int64_t)a.cols + 64 * W - 1) / (64 * W);
    a.tiles_c = (int)tc;
    const unsigned grid = (unsigned)(tr * tc);
    const bool e4 = format == SGEMM_F8_E4M3;
    if (format_x == SGEMM_F8_E4M3) {
        if (e4)
            f8_requantize_kernel<W, 0, 0><<<grid, 64 * W, 0, s>>>(a);
        else
            f8_requantize_kernel<W, 0, 1><<<grid, 64 * W, 0, s>>>(a);
    } else if (e4) {
        f8_requantize_kernel<W, 1, 0><<<grid, 64 * W, 0, s>>>(a);
    } else {
        f8_requantize_kernel<W, 1, 1><<<grid, 64 * W, 0, s>>>(a);
    }
}

}  // namespace

// Tiles beside each other share lines of the rows: 4 of them a workgroup where that fills the
// CUs, else 2 (2 / 4: 8192 x 16384 75.8 / 67.3 us, 16384 x 4097 packed 35.1 / 29.1, 1000 x 1017
// packed 7.1 / 7.6).
hipError_t launch_f8_requantize(const F8QuantArgs &a, int format_x, int format, hipStream_t s)
{
    if (((int64_t)a.rows + 127) / 128 * (((int64_t)a.cols + 255) / 256) >= 256)
        launch_tiles<4>(a, format_x, format, s);
    else
        launch_tiles<2>(a, format_x, format, s);
    return hipGetLastError();
}

}  // namespace sgemm
