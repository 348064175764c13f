"""Oracle: the operators of the block around the attention layer (test infrastructure only).

The root-mean-square norm with the residual's addition, its e4m3 output with
a scale per row, the gated feed-forward product, and the gradients of both,
in float64 from their formulas:

    h = x + residual,  y = h / sqrt(mean(h^2) + eps) * w
    scale = max(max|y|, 2^-100) / 448,  q = e4m3(y / scale)
    out = act(x Wg^T) * (x Wu^T)

Pinned by tests/test_oracle_block.py: hand-derived values, the e4m3 grid
listed value by value, and gradients against central differences.
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0
SCALE_FLOOR = 2.0 ** -100


def rms_norm(h, w, eps):
    """h [N, d], w [d] -> (y [N, d], r [N, 1]) with r = 1 / sqrt(mean(h^2) + eps)."""
    h = np.asarray(h, dtype=np.float64)
    r = 1.0 / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    return h * r * np.asarray(w, dtype=np.float64), r


def rms_norm_backward(dy, h, w, dres, eps):
    """Gradients of sum(dy * y) + sum(dres * h): (dx [N, d], dw [d])."""
    _, r = rms_norm(h, w, eps)
    dn = dy * w
    dx = r * (dn - h * r * r * np.mean(dn * h, axis=1, keepdims=True))
    if dres is not None:
        dx = dx + dres
    return dx, np.sum(dy * h * r, axis=0)


def row_scale(y):
    """The e4m3 scale of each row, [N]."""
    return np.maximum(np.max(np.abs(y), axis=1), SCALE_FLOOR) / E4M3_MAX


def e4m3_half_step(v):
    """Half the distance between neighbouring e4m3 values at v (3 mantissa bits, least exponent -6)."""
    a = np.maximum(np.abs(np.asarray(v, dtype=np.float64)), 2.0 ** -6)
    return 2.0 ** (np.floor(np.log2(a)) - 4)


def e4m3(v):
    """Nearest e4m3 value, ties to even, saturating at 448."""
    step = 2 * e4m3_half_step(v)
    return np.clip(np.round(np.asarray(v, dtype=np.float64) / step) * step, -E4M3_MAX, E4M3_MAX)


def activation(g, act):
    """(act(g), act'(g))."""
    g = np.asarray(g, dtype=np.float64)
    if act == "silu":
        s = 0.5 * (1.0 + np.tanh(0.5 * g))
        return g * s, s * (1.0 + g * (1.0 - s))
    c = np.sqrt(2.0 / np.pi)
    t = np.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * g * g)


def gated_ffn(x, wg, wu, act):
    """x [N, d], wg, wu [F, d] -> [N, F]."""
    return activation(x @ wg.T, act)[0] * (x @ wu.T)


def gated_ffn_backward(x, wg, wu, dout, act):
    """dict(dx, dw_gate, dw_up) of sum(dout * out), with dg and du."""
    g, u = x @ wg.T, x @ wu.T
    a, da = activation(g, act)
    dg, du = dout * u * da, dout * a
    return dict(dx=dg @ wg + du @ wu, dw_gate=dg.T @ x, dw_up=du.T @ x, dg=dg, du=du)
