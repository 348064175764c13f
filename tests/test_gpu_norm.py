"""GPU parity of the RMS norm with the residual's addition and of its backward against the fp64 oracle
(tolerances: _block.py)."""
import numpy as np
import pytest

from _block import CHAIN, check_norm_backward, check_norm_y
from _block import to_np as _np
from oracle import block

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _t(torch):
    return {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


def _rand(torch, dev, shape, dt, seed, scale=1.0):
    g = torch.Generator(device=dev).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=dev) * scale).to(_t(torch)[dt])


# one width per thread layout and its borders, the widest, and the least; N of one row, of one CTA's rows and a
# rest, and above the SM count (where the layout for few rows ends)
SHAPES = [(1, 8), (5, 64), (149, 136), (3, 768), (300, 776), (1, 1536), (301, 1544), (3, 2560), (150, 2568), (1, 5120),
          (151, 5128), (2, 10240), (149, 10248), (1, 16384), (150, 16384),
          # many short rows, several at a time
          (9500, 8), (9473, 64), (9999, 128), (9481, 136), (9490, 256), (9475, 264), (9500, 512)]
TYPES = [("bf16", None, "bf16"), ("bf16", None, "e4m3"), ("f32", None, "f32"), ("f32", None, "bf16"),
         ("f32", None, "e4m3"), ("bf16", "bf16", "bf16"), ("bf16", "bf16", "e4m3"), ("bf16", "f32", "bf16"),
         ("bf16", "f32", "f32"), ("bf16", "f32", "e4m3"), ("f32", "f32", "f32"), ("f32", "f32", "bf16"),
         ("f32", "f32", "e4m3")]


@pytest.mark.parametrize("x_dt,r_dt,out", TYPES)
def test_forward_matches_oracle(x_dt, r_dt, out, cuda_device):
    import torch
    import sparse_attention_long_moga_b200 as moga
    for i, (N, d) in enumerate(SHAPES):
        x = _rand(torch, cuda_device, (N, d), x_dt, 10 + i)
        res = _rand(torch, cuda_device, (N, d), r_dt, 40 + i, 3.0) if r_dt else None
        w = _rand(torch, cuda_device, (d,), "bf16" if i % 2 else "f32", 70 + i)
        y, h, scale = moga.moga_rms_norm(x, w, residual=res, eps=EPS, out_dtype=_t(torch)[out])
        moga.device_status()
        assert y.dtype == _t(torch)[out] and (scale is None) == (out != "e4m3")
        if res is None:
            assert h is x
        else:
            assert torch.equal(h, (x.float() + res.float()).to(res.dtype))   # the stored sum, bit for bit
        want = block.rms_norm(_np(h), _np(w), EPS)[0]
        check_norm_y(_np(y.float()), None if scale is None else _np(scale), want, out)


@pytest.mark.parametrize("h_dt", ["bf16", "f32"])
@pytest.mark.parametrize("N,d", [(30001, 8), (15003, 40), (15001, 64), (29999, 64), (14999, 104), (15002, 128),
                                 (7501, 200), (7499, 256), (701, 7176), (700, 8192)])
def test_backward_of_many_rounds(N, d, h_dt, cuda_device):
    """Several rounds: of several rows a warp, the last without some of them, and of one row an SM."""
    import torch
    import sparse_attention_long_moga_b200 as moga
    h = _rand(torch, cuda_device, (N, d), h_dt, 10, 3.0)
    dy = _rand(torch, cuda_device, (N, d), "bf16", 11)
    dres = _rand(torch, cuda_device, (N, d), h_dt, 12)
    w = _rand(torch, cuda_device, (d,), "f32", 13)
    dx, dw, _ = moga.moga_rms_norm_backward(dy, h, w, dres=dres, eps=EPS)
    moga.device_status()
    check_norm_backward(_np(dx), _np(dw), _np(dy), _np(h), _np(w), _np(dres), EPS, h_dt)


@pytest.mark.parametrize("dy_dt,h_dt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("with_dres", [False, True])
def test_backward_matches_oracle(dy_dt, h_dt, with_dres, cuda_device):
    import torch
    import sparse_attention_long_moga_b200 as moga
    for i, (N, d) in enumerate(SHAPES + [(2500, 1536), (700, 5120), (5000, 136), (3001, 520)]):
        h = _rand(torch, cuda_device, (N, d), h_dt, 10 + i, 3.0)
        dy = _rand(torch, cuda_device, (N, d), dy_dt, 40 + i)
        dres = _rand(torch, cuda_device, (N, d), h_dt, 70 + i) if with_dres else None
        w = _rand(torch, cuda_device, (d,), "bf16" if i % 2 else "f32", 100 + i)
        branch = torch.bfloat16 if h_dt == "f32" else None
        dx, dw, dxb = moga.moga_rms_norm_backward(dy, h, w, dres=dres, eps=EPS, branch_dtype=branch)
        moga.device_status()
        assert dw.dtype == torch.float32
        check_norm_backward(_np(dx), _np(dw), _np(dy), _np(h), _np(w), None if dres is None else _np(dres), EPS, h_dt)
        if branch is None:
            assert dxb is None
        else:
            assert torch.equal(dxb, dx.to(torch.bfloat16))
        # the same again bit for bit; without dw; into dres's own buffer
        dx2, dw2, _ = moga.moga_rms_norm_backward(dy, h, w, dres=dres, eps=EPS)
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
        buf = None if dres is None else dres.clone()
        dx3, dw3, _ = moga.moga_rms_norm_backward(dy, h, w, dres=buf, eps=EPS, need_dw=False, dx=buf)
        assert dw3 is None and torch.equal(dx, dx3) and (buf is None or dx3 is buf)


def test_residual_updated_in_place(cuda_device):
    import torch
    import sparse_attention_long_moga_b200 as moga
    x = _rand(torch, cuda_device, (333, 1536), "bf16", 1)
    w = _rand(torch, cuda_device, (1536,), "f32", 2)
    for dt in ("bf16", "f32"):
        res = _rand(torch, cuda_device, (333, 1536), dt, 3, 3.0)
        y, h, _ = moga.moga_rms_norm(x, w, residual=res)
        stream = res.clone()
        y2, h2, _ = moga.moga_rms_norm(x, w, residual=stream, h=stream)
        assert h2 is stream and torch.equal(h, stream) and torch.equal(y, y2)


def test_extreme_rows(cuda_device):
    """Zero rows, the smallest and largest magnitudes, and rows with NaN or infinity."""
    import torch
    import sparse_attention_long_moga_b200 as moga
    d = 1536
    f8 = torch.float8_e4m3fn
    x = _rand(torch, cuda_device, (9, d), "f32", 5)
    x[1] = 0
    x[2] *= 1e-38                   # squares vanish; y is x / sqrt(eps)
    x[3] *= 1e15
    x[4, 7] = float("nan")
    x[5, 9] = float("inf")
    x[6] *= 1e-44                   # below the scale's floor even after 1 / sqrt(eps)
    w = _rand(torch, cuda_device, (d,), "f32", 6)
    y, _, _ = moga.moga_rms_norm(x, w, out_dtype=torch.float32)
    q, _, s = moga.moga_rms_norm(x, w, out_dtype=f8)
    with np.errstate(invalid="ignore"):   # the rows with NaN and infinity
        want = block.rms_norm(_np(x), _np(w), 1e-6)[0]
    ok = [0, 1, 3, 7, 8]
    assert np.all(np.abs(_np(y)[ok] - want[ok]) <= CHAIN * np.abs(want[ok]))
    assert torch.isnan(y[4]).all() and torch.isnan(y[5, 9])
    assert torch.isnan(s[4]) and torch.isnan(s[5])
    for r in (1, 6):                # all zero, scale at its floor
        assert float(s[r]) == np.float32(2.0 ** -100) / np.float32(448) and not q[r].float().any()
    check_norm_y(_np(q.float())[[0, 3, 7, 8]], _np(s)[[0, 3, 7, 8]], want[[0, 3, 7, 8]], "e4m3")
    # row 2: values of 1e-38 (some subnormal) times 1e3; every value within the grid's half step
    v = _np(q.float())[2] * float(s[2])
    assert np.all(np.abs(v - want[2]) <= block.e4m3_half_step(want[2] / float(s[2])) * float(s[2]) * 1.01 + 1e-41)
    # neighbours of bad rows are untouched by them
    y0, _, _ = moga.moga_rms_norm(x[[0, 1, 7, 8]].contiguous(), w, out_dtype=torch.float32)
    assert torch.equal(y0, y[[0, 1, 7, 8]])


def test_offsets_past_32_bits(cuda_device):
    """More than 2^31 elements: the last rows equal a small call's."""
    import torch
    import sparse_attention_long_moga_b200 as moga
    N, d = 140_000, 16384
    x = torch.empty((N, d), dtype=torch.bfloat16, device=cuda_device)
    x.view(torch.int16).random_(0x3c00, 0x4200)     # positive bf16 values of 2^-7 to 2^5
    w = _rand(torch, cuda_device, (d,), "f32", 8)
    y, h, _ = moga.moga_rms_norm(x, w, residual=x)
    tail = x[-3:].clone()
    y2, h2, _ = moga.moga_rms_norm(tail, w, residual=tail)
    assert torch.equal(y[-3:], y2) and torch.equal(h[-3:], h2)
    dx, _, _ = moga.moga_rms_norm_backward(y, h, w, need_dw=False)
    dx2, _, _ = moga.moga_rms_norm_backward(y2, h2, w, need_dw=False)
    assert torch.equal(dx[-3:], dx2)
    moga.device_status()
