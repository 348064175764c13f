"""Pins of the block operators' oracle (CPU): closed forms, the e4m3 grid, gradients against differences."""
import numpy as np
import pytest

from oracle import block


def test_norm_closed_forms():
    # a row of equal magnitudes normalises to its signs; a zero row stays zero
    y, r = block.rms_norm(np.array([[3.0, -3.0, 3.0, 3.0], [0, 0, 0, 0]]), np.array([1.0, 2.0, 0.5, 1.0]), 1e-12)
    assert np.allclose(y[0], [1, -2, 0.5, 1], rtol=1e-12) and np.all(y[1] == 0)
    # 3, 4: mean square 12.5
    y, _ = block.rms_norm(np.array([[3.0, 4.0]]), np.ones(2), 0.0)
    assert np.allclose(y[0], np.array([3.0, 4.0]) / np.sqrt(12.5), rtol=1e-15)


def test_e4m3_grid():
    # every finite value of the format: subnormals k * 2^-9, normals (8 + m) * 2^(e - 3), 448 the largest
    grid = sorted({k * 2.0 ** -9 for k in range(8)} |
                  {(8 + m) * 2.0 ** (e - 3) for e in range(-6, 9) for m in range(8) if not (e == 8 and m == 7)})
    assert grid[-1] == 448 and len(grid) == 127
    g = np.array(grid)
    assert np.array_equal(block.e4m3(g), g) and np.array_equal(block.e4m3(-g), -g)
    mid = (g[:-1] + g[1:]) / 2
    even = np.array([lo if i % 2 == 0 else hi for i, (lo, hi) in enumerate(zip(g[:-1], g[1:]))])
    assert np.array_equal(block.e4m3(mid), even)                     # ties to the even code
    eps = 1e-9 * np.maximum(mid, 1e-3)
    assert np.array_equal(block.e4m3(mid - eps), g[:-1]) and np.array_equal(block.e4m3(mid + eps), g[1:])
    assert np.array_equal(block.e4m3([1e4, -460.0]), [448, -448])
    rng = np.random.default_rng(0)
    v = rng.uniform(-448, 448, 1000) * 2.0 ** rng.integers(-12, 1, 1000)
    near = g[np.argmin(np.abs(np.abs(v)[:, None] - g), axis=1)]
    assert np.allclose(np.abs(np.abs(v) - near), np.abs(block.e4m3(v) - v), rtol=0, atol=1e-15)
    assert np.all(np.abs(block.e4m3(v) - v) <= block.e4m3_half_step(v))


def test_activations():
    assert block.activation(np.zeros(1), "silu")[0] == 0 and block.activation(np.zeros(1), "silu")[1] == 0.5
    assert np.allclose(block.activation(np.ones(1), "silu")[0], 1 / (1 + np.exp(-1)))
    assert block.activation(np.zeros(1), "gelu")[1] == 0.5
    assert np.allclose(block.activation(np.ones(1), "gelu")[0], 0.8411919906082768, rtol=1e-12)


def _difference(f, x, e=1e-6):
    out = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[i] = e
        out[i] = (f(x + d) - f(x - d)) / (2 * e)
    return out


def test_norm_gradients_against_differences():
    rng = np.random.default_rng(1)
    h, dy, dres = (rng.standard_normal((3, 8)) for _ in range(3))
    w = rng.standard_normal(8)
    dx, dw = block.rms_norm_backward(dy, h, w, dres, 1e-3)
    J = lambda hh, ww: np.sum(dy * block.rms_norm(hh, ww, 1e-3)[0]) + np.sum(dres * hh)  # noqa: E731
    assert np.allclose(dx, _difference(lambda v: J(v, w), h), rtol=1e-6, atol=1e-8)
    assert np.allclose(dw, _difference(lambda v: J(h, v), w), rtol=1e-6, atol=1e-8)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_ffn_gradients_against_differences(act):
    rng = np.random.default_rng(2)
    x, wg, wu, do = (rng.standard_normal(s) for s in ((3, 4), (5, 4), (5, 4), (3, 5)))
    g = block.gated_ffn_backward(x, wg, wu, do, act)
    J = lambda a, b, c: np.sum(do * block.gated_ffn(a, b, c, act))  # noqa: E731
    assert np.allclose(g["dx"], _difference(lambda v: J(v, wg, wu), x), rtol=1e-6, atol=1e-8)
    assert np.allclose(g["dw_gate"], _difference(lambda v: J(x, v, wu), wg), rtol=1e-6, atol=1e-8)
    assert np.allclose(g["dw_up"], _difference(lambda v: J(x, wg, v), wu), rtol=1e-6, atol=1e-8)
