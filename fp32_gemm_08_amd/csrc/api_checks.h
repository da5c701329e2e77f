// Argument checks that the entry points of the 8-bit and norm families share.
#pragma once
#include "f8_internal.h"

#include <cmath>
#include <limits>

namespace sgemm {
namespace {

constexpr int64_t kMaxDim = (int64_t{1} << 31) - 1025;
constexpr int64_t kAnyRoom = std::numeric_limits<int64_t>::max();
constexpr int64_t kMaxWorkItems = (int64_t{1} << 32) - 1;

int type_bytes(int t) { return t == SGEMM_TYPE_F32 ? 4 : 2; }
bool known_type(int t) { return t == SGEMM_TYPE_F32 || t == SGEMM_TYPE_FP16 || t == SGEMM_TYPE_BF16; }
bool known_format(int f) { return f == SGEMM_F8_E4M3 || f == SGEMM_F8_E5M2; }
bool known_block(int b) { return b == SGEMM_F8_ROW || b == SGEMM_F8_TILE; }
bool dim_ok(int64_t d) { return d >= 0 && d <= kMaxDim; }
bool on(const void *p, int bytes) { return p != nullptr && reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes == 0; }

// A rows x cols operand of `size`-byte elements: what its bytes span, and
// whether every row starts on a `to`-byte boundary.
struct Operand {
    const void *p;
    int64_t rows, cols, ld;
    int size;
    // A leading dimension that holds a row, and a span within int64.
    bool shape_ok() const
    {
        return ld >= (cols > 1 ? cols : 1) && (rows <= 1 || ld <= std::numeric_limits<int64_t>::max() / 8 / rows);
    }
    int64_t bytes() const { return rows == 0 || cols == 0 ? 0 : ((rows - 1) * ld + cols) * size; }
    bool present() const { return on(p, size); }
    bool rows_on(int to) const
    {
        return reinterpret_cast<uintptr_t>(p) % (uintptr_t)to == 0 && (rows <= 1 || ld * size % to == 0);
    }
    // The same elements at the same places (an update in place).
    bool same(const Operand &o) const
    {
        return p == o.p && size == o.size && (rows <= 1 || ld == o.ld);
    }
};

bool overlap(const Operand &a, const Operand &b)
{
    if (a.p == nullptr || b.p == nullptr || a.bytes() == 0 || b.bytes() == 0)
        return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + (uintptr_t)b.bytes() && y < x + (uintptr_t)a.bytes();
}

// Whether some output overlaps another operand: every output against every
// input (in place where `in_place` allows that pair) and every other output.
template <int NO, int NI>
bool aliased(const Operand (&out)[NO], const Operand (&in)[NI], int in_place_out, unsigned in_place_in)
{
    for (int i = 0; i < NO; ++i) {
        for (int j = i + 1; j < NO; ++j)
            if (overlap(out[i], out[j]))
                return true;
        for (int j = 0; j < NI; ++j)
            if (overlap(out[i], in[j]) && !(i == in_place_out && (in_place_in >> j & 1) && out[i].same(in[j])))
                return true;
    }
    return false;
}

// A scale array of a rows x cols operand.
Operand scales(const float *p, int block, int64_t rows, int64_t cols, int64_t ld)
{
    if (block == SGEMM_F8_ROW)
        return Operand{p, ceil_div(cols, F8_BLOCK), rows, ld, 4};
    return Operand{p, ceil_div(rows, F8_BLOCK), ceil_div(cols, F8_BLOCK), ld, 4};
}

int finish(hipError_t e) { return e == hipSuccess ? SGEMM_OK : SGEMM_ERR_LAUNCH; }

}  // namespace
}  // namespace sgemm
