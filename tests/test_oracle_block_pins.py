"""The FP64 oracle of the norms around a block and of 8-bit integers against values worked
out by hand, and its gradients against differences."""
import numpy as np

from oracle import oracle_block as ob


def test_norm_by_hand():
    # o = (3, 4): mean square 12.5; x = 2
    x, o = np.full((1, 2), 2.0), np.array([[3.0, 4.0]])
    h, y, rstd, rp, z = ob.block_norm(x, o, np.array([1.0, 2.0]), 0.0, np.array([1.0, 0.5]), np.array([[10.0, 0.0]]), 1, 3.0)
    r = 12.5 ** -0.5
    assert np.allclose(rp, r) and np.allclose(z, [[3 * r, 2 * r]]) and np.allclose(h, [[6 + 30 * r, 6.0]])
    s = (((6 + 30 * r) ** 2 + 36) / 2) ** -0.5
    assert np.allclose(rstd, s) and np.allclose(y, [[(6 + 30 * r) * s, 12 * s]])
    h, y, _, rp, z = ob.block_norm(x, None, None, 1e-6, alpha=-1.0)
    assert rp is None and z is None and y is None and np.all(h == -2)


def test_gates_take_consecutive_rows():
    g = np.arange(6.0).reshape(3, 2)
    assert np.array_equal(ob.gate_of_rows(g, 2, 5)[:, 0], [0, 0, 2, 2, 4])
    assert ob.gate_of_rows(None, 2, 5) == 1.0


def test_gradients_against_differences():
    rng = np.random.default_rng(0)
    rows, cols, gate_rows, alpha, d = 5, 6, 2, -0.7, 1e-5
    p = dict(x=rng.standard_normal((rows, cols)), o=rng.standard_normal((rows, cols)), w=rng.standard_normal(cols),
             wp=rng.standard_normal(cols), gate=rng.standard_normal((3, cols)))
    v, u = rng.standard_normal((rows, cols)), rng.standard_normal((rows, cols))
    for post in (True, False):
        def loss(p):
            h, y, *_ = ob.block_norm(p["x"], p["o"], p["w"], 1e-3, p["wp"] if post else None, p["gate"], gate_rows, alpha)
            return (y * v + h * u).sum()

        h, y, rstd, rp, _ = ob.block_norm(p["x"], p["o"], p["w"], 1e-3, p["wp"] if post else None, p["gate"], gate_rows, alpha)
        e = ob.block_norm_backward(v, u, h, p["o"], p["w"], rstd, p["wp"] if post else None, rp, p["gate"], gate_rows, alpha)
        for name, key in (("x", "dx"), ("o", "do"), ("w", "dw"), ("gate", "dgate")) + ((("wp", "dw_post"),) if post else ()):
            for i in np.ndindex(*p[name].shape):
                up, down = ({k: a.copy() for k, a in p.items()} for _ in range(2))
                up[name][i] += d
                down[name][i] -= d
                assert abs((loss(up) - loss(down)) / (2 * d) - e[key][i]) < 1e-7 * (1 + abs(e[key][i])), (name, i)


def test_integers_by_hand():
    q, s = ob.quantize_rows_i8(np.array([[127.0, 0.5, 1.5, -2.5, -126.5], [0, 0, 0, 0, 0], [2, 1, -1, 0.25, np.inf]], np.float32))
    assert q.tolist() == [[127, 0, 2, -2, -126], [0] * 5, [0] * 5]
    assert s[0] == 1 and s[1] == np.float32(2.0 ** -90) / np.float32(127) and np.isinf(s[2])
    a, b = np.array([[-128, 127]], np.int8), np.array([[-128, 127], [1, 0]], np.int8)
    d, t = ob.gemm_i8(a, np.array([2.0]), b, np.array([0.5, 3.0]), alpha=2.0, beta=1.0, c=np.array([[1.0, 1.0]]))
    assert t.tolist() == [[128 * 128 + 127 * 127, -128]] and d.tolist() == [[2 * (16384 + 16129) + 1, -2 * 768 + 1]]
