"""Pins of the 8-bit family's FP64 oracle: formats by hand, rounding against a
brute-force nearest code, and the norm's gradient against differences."""
import math

import numpy as np
import pytest

from oracle import oracle_f8 as o8


def test_formats_by_hand():
    e4, e5 = o8.VALUES["e4m3"], o8.VALUES["e5m2"]
    assert e4[0x01] == 2.0 ** -9 and e4[0x08] == 2.0 ** -6 and e4[0x38] == 1.0 and e4[0x7e] == 448.0
    assert e4[0xb9] == -1.125 and math.isnan(e4[0x7f]) and math.isnan(e4[0xff])
    assert e5[0x01] == 2.0 ** -16 and e5[0x04] == 2.0 ** -14 and e5[0x3c] == 1.0 and e5[0x7b] == 57344.0
    assert math.isinf(e5[0x7c]) and math.isnan(e5[0x7d]) and e5[0xc0] == -2.0


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_encode_is_nearest_and_ties_go_to_even(fmt):
    vals = o8.VALUES[fmt]
    fin = np.flatnonzero(np.isfinite(vals))
    assert np.array_equal(o8.decode(o8.encode(vals[fin].astype(np.float32), fmt), fmt), vals[fin])
    rng = np.random.default_rng(1)
    pos = np.unique(np.abs(vals[fin]))
    mid = (pos[:-1] + pos[1:]) / 2                       # exact in FP32
    x = np.concatenate([mid, -mid, rng.uniform(-pos[-1], pos[-1], 2000),
                        rng.uniform(-4, 4, 500) * pos[1]]).astype(np.float32)
    got = o8.encode(x, fmt)
    for v, code in zip(x.astype(np.float64), got):
        d = np.abs(vals[fin] - v)
        best = fin[d == d.min()]
        assert code in best
        if len(set(np.abs(vals[best]))) > 1:
            assert code % 2 == 0
    assert o8.encode(np.array([np.nan], np.float32), fmt)[0] == 0x7f


@pytest.mark.parametrize("block", ["row", "tile"])
@pytest.mark.parametrize("fmt,step,sub", [("e4m3", 2.0 ** -4, 2.0 ** -10), ("e5m2", 2.0 ** -3, 2.0 ** -17)])
def test_quantized_values_are_half_a_step_from_x(block, fmt, step, sub):
    rng = np.random.default_rng(2)
    x = (rng.standard_normal((200, 300)) * np.exp(2 * rng.standard_normal((200, 1)))).astype(np.float32)
    q, s = o8.quantize(x, block, fmt)
    v = o8.values(q, s, block, fmt)
    per = o8.spread((s.T if block == "row" else s).astype(np.float64), block, *x.shape)
    # half a step of the format, and two FP32 roundings of the factor and the product, one of the scale
    assert np.all(np.abs(v - x) <= np.maximum(step * np.abs(x), sub * per) * (1 + 1e-6) + 4 * 2.0 ** -24 * np.abs(x))
    top = o8._block_max(np.abs(x), block)
    assert np.allclose(o8._block_max(np.abs(v).astype(np.float32), block), top, rtol=1e-6)


def test_zero_and_special_blocks():
    x = np.zeros((3, 256), np.float32)
    x[1, 5], x[2, 130] = np.nan, np.inf
    q, s = o8.quantize(x, "row", "e4m3")
    v = o8.values(q, s, "row", "e4m3")
    assert np.all(v[0] == 0) and np.all(np.isfinite(s[:, 0])) and np.all(s[:, 0] > 0)
    assert np.all(np.isnan(v[1, :128])) and np.all(v[1, 128:] == 0)
    assert np.all(np.isnan(v[2, 128:])) and np.all(v[2, :128] == 0)


@pytest.mark.parametrize("cols", [1, 2, 7, 33])
def test_norm_gradient_against_differences(cols):
    rng = np.random.default_rng(cols)
    x, r, dy, dh = (rng.standard_normal((3, cols)) for _ in range(4))
    w, eps = rng.standard_normal(cols), 1e-3

    def loss(x, w):
        h, _, y = o8.rmsnorm(x, r, w, eps)
        return (y * dy).sum() + (h * dh).sum()

    h, rstd, _ = o8.rmsnorm(x, r, w, eps)
    dx, dw = o8.rmsnorm_backward(dy, h, w, rstd, dh)
    d = 1e-6
    for i in range(3):
        for j in range(cols):
            e = np.zeros_like(x)
            e[i, j] = d
            assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * d) - dx[i, j]) < 1e-6 * max(1.0, abs(dx[i, j]))
    for j in range(cols):
        e = np.zeros(cols)
        e[j] = d
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * d) - dw[j]) < 1e-6 * max(1.0, abs(dw[j]))


def test_gemm_definition():
    rng = np.random.default_rng(3)
    x, y = rng.standard_normal((5, 300)).astype(np.float32), rng.standard_normal((200, 300)).astype(np.float32)
    (qa, sa), (qb, sb) = o8.quantize(x, "row", "e4m3"), o8.quantize(y, "tile", "e5m2")
    c = rng.standard_normal((5, 200)).astype(np.float32)
    d, s = o8.gemm_f8(o8.values(qa, sa, "row", "e4m3"), o8.values(qb, sb, "tile", "e5m2"), 1.5, -0.5, c)
    for i, j in ((0, 0), (4, 199), (2, 130)):
        t = [o8.VALUES["e4m3"][qa[i, k]] * float(sa[k // 128, i]) * o8.VALUES["e5m2"][qb[j, k]] * float(sb[j // 128, k // 128])
             for k in range(300)]
        assert abs(1.5 * math.fsum(t) - 0.5 * float(c[i, j]) - d[i, j]) < 1e-12 * (s[i, j] + 1)
        assert abs(math.fsum(map(abs, t)) - s[i, j]) < 1e-12 * s[i, j]
