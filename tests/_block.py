"""Checks of the block operators' results against the fp64 oracle, shared by their GPU tests.

Tolerances count roundings, and are derived from the kernels' arithmetic.

Norm.  The fp32 chain per value is a sum of up to 40 squares per thread, a
tree of at most 5 + 16 adds, and about ten further operations: under 2^7
roundings of 2^-24 at most, so 2^-17 (CHAIN) relative to the sum of the terms'
magnitudes.  A stored value is off by half a step of its type more: 2^-24
(fp32, inside CHAIN), 2^-8 (bf16), the e4m3 grid's half step.

Gated feed-forward.  The tensor core adds K = 16 (bf16) or 32 (e4m3) products
a step into an fp32 accumulator and truncates: one unit, 2^-23, of the partial
sum a step, so a projection is off by E(g) = (d / 16) 2^-23 sum_k |x_k w_k| at
most (as for the Q/K/V projection).  exp and the quotient of the activation
are off by (16 + 8 |z|) 2^-23 relative, z the sigmoid's argument.  The result
is rounded to bf16: 2^-8.  In the backward dg and du carry those errors and one
bf16 rounding each, which the products that follow carry over term by term,
adding their own accumulation and rounding.
"""
import numpy as np

from oracle import block

CHAIN = 2.0 ** -17
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
BF = 2.0 ** -8
ULP = 2.0 ** -23


def to_np(t):
    return t.double().cpu().numpy()


def check_norm_y(y, scale, want, out):
    if out == "e4m3":
        s = block.row_scale(want)
        assert np.all(np.abs(scale - s) <= CHAIN * s)
        v = want / s[:, None]
        assert np.all(np.abs(y - v) <= block.e4m3_half_step(v) + CHAIN * np.abs(v))
        assert np.all(np.max(np.abs(y), axis=1) == 448.0)
    else:
        assert np.all(np.abs(y - want) <= (HALF[out] + CHAIN) * np.abs(want))


def check_norm_backward(dx, dw, dy, h, w, dres, eps, h_dt):
    """dx and dw (or None) against the formula's, all arguments float64 arrays."""
    rdx, rdw = block.rms_norm_backward(dy, h, w, dres, eps)
    _, r = block.rms_norm(h, w, eps)
    terms = r * (np.abs(dy * w) + np.abs(h) * r * r * np.mean(np.abs(dy * w * h), axis=1, keepdims=True))
    if dres is not None:
        terms = terms + np.abs(dres)
    assert np.all(np.abs(dx - rdx) <= HALF[h_dt] * np.abs(rdx) + CHAIN * terms)
    if dw is not None:   # at most N sequential adds and the rows' own chains
        assert np.all(np.abs(dw - rdw) <= (CHAIN + len(h) * 2.0 ** -24) * np.sum(np.abs(dy * h * r), axis=0))


def _parts(x, wg, wu, act):
    """g, u, their accumulation errors, act, act' and the activation's own relative error."""
    d = x.shape[1]
    g, u = x @ wg.T, x @ wu.T
    eg, eu = ((d / 16 + 4) * ULP * (np.abs(x) @ np.abs(w).T) for w in (wg, wu))
    a, da = block.activation(g, act)
    z = np.abs(g) if act == "silu" else 1.6 * (np.abs(g) + 0.045 * np.abs(g) ** 3)
    return g, u, eg, eu, a, da, (16 + 8 * z) * ULP


def check_ffn(out, x, wg, wu, act):
    g, u, eg, eu, a, da, ez = _parts(x, wg, wu, act)
    want = a * u
    # |act'| over the error's reach: at most |act'(g)| + 1.2 E(g)
    slack = (np.abs(da) + 1.2 * eg) * eg * (np.abs(u) + eu) + np.abs(a) * eu + ez * np.abs(want)
    err = np.abs(out - want)
    tol = BF * np.abs(want) + 1.01 * slack + 2.0 ** -126
    assert np.all(err <= tol), "worst error / tolerance %.3f" % np.max(err / tol)


def check_ffn_backward(got, x, wg, wu, do, act, keys=("dx", "dw_gate", "dw_up")):
    N, F = do.shape
    g, u, eg, eu, a, da, ez = _parts(x, wg, wu, act)
    ref = block.gated_ffn_backward(x, wg, wu, do, act)
    # errors of the stored dg and du
    dda = 1.2 * eg + ez * (1 + np.abs(a) + np.abs(da) + (0 if act == "silu" else 2 * np.abs(a) * (1 + 0.14 * g * g)))
    edg = np.abs(do) * (np.abs(da) * eu + (np.abs(u) + eu) * dda)
    edg = edg + BF * (np.abs(ref["dg"]) + edg)
    edu = np.abs(do) * ((np.abs(da) + 1.2 * eg) * eg + ez * np.abs(a))
    edu = edu + BF * (np.abs(ref["du"]) + edu)
    ag, au = np.abs(ref["dg"]) + edg, np.abs(ref["du"]) + edu
    tol = {
        "dx": edg @ np.abs(wg) + edu @ np.abs(wu) + (2 * F / 16 + 12) * ULP * (ag @ np.abs(wg) + au @ np.abs(wu)),
        "dw_gate": edg.T @ np.abs(x) + (N / 16 + 6) * ULP * (ag.T @ np.abs(x)),
        "dw_up": edu.T @ np.abs(x) + (N / 16 + 6) * ULP * (au.T @ np.abs(x)),
    }
    for k in keys:
        out = to_np(got[k])
        err = np.abs(out - ref[k])
        t = BF * np.abs(ref[k]) + 1.01 * tol[k] + 2.0 ** -126
        assert np.all(err <= t), "%s: worst error / tolerance %.3f" % (k, np.max(err / t))
        if ref[k].size >= 4096:   # independent roundings: rms 2^-8 / sqrt 3 each, two of them
            assert np.linalg.norm(out - ref[k]) <= 1.3 * BF * np.sqrt(2 / 3) * np.linalg.norm(ref[k]), k
