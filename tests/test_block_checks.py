"""Argument checks of the block operators, in the binding and in the C ABI (CPU only: nothing is launched)."""
import ctypes

import pytest
import torch

import sparse_attention_long_moga_b200 as moga
from sparse_attention_long_moga_b200 import _lib
from sparse_attention_long_moga_b200.build import build

BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
N, D, F = 6, 32, 48


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.load()


def _t(*shape, dt=BF):
    return torch.zeros(shape, dtype=dt)


def test_norm_binding():
    x, w = _t(N, D), _t(D, dt=F32)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):   # well-formed: stops at the residence check
        moga.moga_rms_norm(x, w, residual=_t(N, D, dt=F32), out_dtype=E4)
    for bad, msg in ((dict(x=_t(N, D, dt=torch.float16)), "x must be float32 or bfloat16"),
                     (dict(x=_t(N, 2, D)), "x must have 2 dims"),
                     (dict(x=_t(D, N).T), "x must be contiguous"),
                     (dict(weight=_t(D + 8)), "weight must have shape"),
                     (dict(weight=_t(D, dt=torch.float64)), "weight must be"),
                     (dict(residual=_t(N + 1, D)), "residual must have shape"),
                     (dict(residual=_t(N, D, dt=torch.float16)), "residual must be"),
                     (dict(out_dtype=torch.float16), "out_dtype must be"),
                     (dict(h=_t(N, D)), "there is no residual"),
                     (dict(residual=_t(N, D), h=_t(N, D, dt=F32)), "h must be")):
        with pytest.raises(ValueError, match=msg):
            moga.moga_rms_norm(**dict(dict(x=x, weight=w), **bad))


def test_norm_backward_binding():
    h, dy, w = _t(N, D, dt=F32), _t(N, D), _t(D, dt=F32)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        moga.moga_rms_norm_backward(dy, h, w, dres=_t(N, D, dt=F32), branch_dtype=BF)
    for bad, msg in ((dict(dy=_t(N, D + 8)), "dy must have shape"), (dict(weight=_t(D - 8)), "weight must have shape"),
                     (dict(dres=_t(N, D)), "dres must be"), (dict(dx=_t(N, D)), "dx must be"),
                     (dict(branch_dtype=F32), "branch_dtype must be"), (dict(h=_t(N, D).t()), "h must be contiguous")):
        with pytest.raises(ValueError, match=msg):
            moga.moga_rms_norm_backward(**dict(dict(dy=dy, h=h, weight=w), **bad))


def test_ffn_binding():
    x, wg, wu = _t(N, D), _t(F, D), _t(F, D)
    s = dict(x_scale=_t(N, dt=F32), w_gate_scale=_t(F, dt=F32), w_up_scale=_t(F, dt=F32))
    q = dict(x=x.to(E4), w_gate=wg.to(E4), w_up=wu.to(E4))
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        moga.moga_gated_ffn(x, wg, wu, act="gelu")
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        moga.moga_gated_ffn(**q, **s)
    good = dict(x=x, w_gate=wg, w_up=wu)
    for bad, msg in ((dict(x=x.float()), "x must be bfloat16 or float8"), (dict(w_gate=wg.float()), "w_gate must be"),
                     (dict(w_gate=_t(F, D + 8)), "w_gate must be"), (dict(w_up=_t(F + 8, D)), "w_up must have shape"),
                     (dict(act="relu"), "act must be"), (dict(x_scale=s["x_scale"]), "x_scale goes with float8"),
                     (dict(x=x[None]), "x must have 2 dims"), (dict(w_up=_t(D, F).t()), "w_up must be contiguous")):
        with pytest.raises(ValueError, match=msg):
            moga.moga_gated_ffn(**dict(good, **bad))
    for name, n in (("x_scale", N), ("w_gate_scale", F), ("w_up_scale", F)):
        with pytest.raises(ValueError, match="need %s" % name):
            moga.moga_gated_ffn(**q, **dict(s, **{name: None}))
        with pytest.raises(ValueError, match="%s must have shape" % name):
            moga.moga_gated_ffn(**q, **dict(s, **{name: _t(n + 1, dt=F32)}))
        with pytest.raises(ValueError, match="%s must be" % name):
            moga.moga_gated_ffn(**q, **dict(s, **{name: _t(n)}))
    with pytest.raises(ValueError, match="dout must have shape"):
        moga.moga_gated_ffn_backward(x, wg, wu, _t(N, F + 8))
    with pytest.raises(ValueError, match="x must be"):
        moga.moga_gated_ffn_backward(q["x"], q["w_gate"], q["w_up"], _t(N, F))


P = ctypes.c_void_p(4096)     # never dereferenced: validation fails first
ODD = ctypes.c_void_p(4104)
W = 1 << 40


def _norm(lib, **kw):
    a = dict(x=P, x_dt=1, res=P, res_dt=1, w=P, w_dt=0, N=10, d=64, eps=1e-6, h=P, y=P, y_dt=1, scale=None)
    a.update(kw)
    return lib.moga_rms_norm(*a.values(), None)


@pytest.mark.parametrize("bad,status", [
    (dict(x=None), 1), (dict(w=None), 1), (dict(y=None), 1), (dict(res=None), 1), (dict(h=None), 1), (dict(N=0), 1),
    (dict(N=1 << 30), 1), (dict(d=12), 1), (dict(d=0), 1), (dict(d=16392), 2), (dict(eps=0.0), 1),
    (dict(eps=float("nan")), 1), (dict(eps=-1.0), 1), (dict(eps=float("inf")), 1), (dict(x_dt=2), 1),
    (dict(x_dt=0), 2), (dict(y_dt=2), 1), (dict(scale=P), 1), (dict(y_dt=3), 1), (dict(y_dt=0), 2), (dict(w_dt=2), 1),
    (dict(x=ODD), 1), (dict(y=ODD), 1), (dict(h=ODD), 1), (dict(w=ODD), 1)])
def test_norm_abi(lib, bad, status):
    assert _norm(lib, **bad) == status and b"moga_rms_norm" in lib.moga_last_error()


def _norm_bwd(lib, **kw):
    a = dict(dy=P, dy_dt=1, h=P, h_dt=1, w=P, w_dt=0, dres=P, N=10, d=64, eps=1e-6, dx=P, dxb=None, dw=P, ws=P, n=W)
    a.update(kw)
    return lib.moga_rms_norm_bwd(*a.values(), None)


@pytest.mark.parametrize("bad,status", [
    (dict(dy=None), 1), (dict(h=None), 1), (dict(dx=None), 1), (dict(w=None), 1), (dict(dy_dt=0), 2), (dict(dxb=P), 1),
    (dict(ws=None), 1), (dict(n=64), 3), (dict(N=-1), 1), (dict(d=4), 1), (dict(d=1 << 15), 2), (dict(dres=ODD), 1),
    (dict(dw=ODD), 1), (dict(dy_dt=2), 1), (dict(eps=0.0), 1)])
def test_norm_bwd_abi(lib, bad, status):
    assert _norm_bwd(lib, **bad) == status and b"moga_rms_norm_bwd" in lib.moga_last_error()


def _ffn(lib, **kw):
    a = dict(x=P, wg=P, wu=P, dt=1, xs=None, gs=None, us=None, N=10, d=64, F=32, act=0, out=P)
    a.update(kw)
    return lib.moga_gated_ffn(*a.values(), None)


E = dict(dt=2, xs=P, gs=P, us=P)


@pytest.mark.parametrize("bad,status", [
    (dict(x=None), 1), (dict(wu=None), 1), (dict(out=None), 1), (dict(dt=0), 1), (dict(dt=3), 1), (dict(xs=P), 1),
    (dict(dt=2), 1), (dict(E, us=None), 1), (dict(N=0), 1), (dict(N=1 << 30), 1), (dict(d=4), 1), (dict(E, d=24), 1),
    (dict(F=12), 1), (dict(F=0), 1), (dict(F=(1 << 20) + 8), 1), (dict(N=(1 << 30) - 1, F=1 << 20), 1), (dict(act=2), 1),
    (dict(act=-1), 1), (dict(x=ODD), 1), (dict(out=ODD), 1), (dict(E, gs=ctypes.c_void_p(4100)), 1),
    (dict(E, xs=ctypes.c_void_p(4098)), 1)])
def test_ffn_abi(lib, bad, status):
    assert _ffn(lib, **bad) == status and b"moga_gated_ffn" in lib.moga_last_error()


def _ffn_bwd(lib, **kw):
    a = dict(x=P, wg=P, wu=P, N=10, d=64, F=32, act=0, dout=P, dx=P, dwg=P, dwu=P, ws=P, n=W)
    a.update(kw)
    return lib.moga_gated_ffn_bwd(*a.values(), None)


@pytest.mark.parametrize("bad,status", [
    (dict(x=None), 1), (dict(dout=None), 1), (dict(ws=None), 1), (dict(dwg=None), 1), (dict(dwu=None), 1),
    (dict(dx=None, dwg=None, dwu=None), 1), (dict(N=0), 1), (dict(d=4), 1), (dict(F=4), 1), (dict(act=7), 1),
    (dict(n=100), 3), (dict(dx=ODD), 1), (dict(ws=ODD), 1)])
def test_ffn_bwd_abi(lib, bad, status):
    assert _ffn_bwd(lib, **bad) == status and b"moga_gated_ffn_bwd" in lib.moga_last_error()


def test_workspace_sizes(lib):
    norm, ffn = lib.moga_rms_norm_bwd_ws_bytes, lib.moga_gated_ffn_bwd_ws_bytes
    # rejected sizes
    for a in ((0, 64), (10, 12), (10, 16392), (1 << 30, 64)):
        assert norm(*a) == 0
    for a in ((0, 64, 64), (10, 12, 64), (10, 64, 12), (10, (1 << 20) + 8, 64), ((1 << 30) - 1, 8, 1 << 20),
              ((1 << 30) - 1, 1 << 20, 8)):
        assert ffn(*a) == 0
    # one partial row per CTA: no more CTAs than groups of rows
    assert norm(1, 1536) == 1536 * 4 and norm(8, 256) == 256 * 4 and norm(9, 256) == 2 * 256 * 4
    # dg and du alone where the tiles fill the GPU; partial sums as well where K is split
    assert ffn(32760, 1536, 4096) == 4 * 32760 * 4096
    assert ffn(100, 64, 64) == 4 * 100 * 64 and ffn(5000, 64, 64) > 4 * 5000 * 64
