"""GPU: the norm's backward on rows of extreme magnitude and its launches' residence (oracle and tolerances:
_block.py)."""
import ctypes

import numpy as np
import pytest

from _block import check_norm_backward
from _block import to_np as _np

pytestmark = pytest.mark.gpu

# one width per form of the backward: a quarter, half and a whole warp a row, three vectors a lane, a row a CTA of one,
# two (plain and with the next row under way) and four vectors a thread
WIDTHS = [64, 128, 256, 264, 768, 776, 1536, 5120, 8192, 10240]
PAIRS = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]


def _rows(torch, dev, N, d, dy_dt, h_dt, seed):
    """h and a dy that leans on it (so that the projection term counts), w."""
    t = {"bf16": torch.bfloat16, "f32": torch.float32}
    g = torch.Generator(device=dev).manual_seed(seed)
    h = torch.randn((N, d), generator=g, device=dev)
    dy = (h + 0.5 * torch.randn((N, d), generator=g, device=dev)) * 1e-2
    return h, dy.to(t[dy_dt]), torch.randn(d, generator=g, device=dev) * 0.2 + 1, t[h_dt]


@pytest.mark.parametrize("dy_dt,h_dt", PAIRS)
def test_backward_of_large_and_tiny_rows(dy_dt, h_dt, cuda_device):
    """Root mean squares from 1e-20 to 1e17: the sum of squares stays in the fp32 range."""
    import torch
    import sparse_attention_long_moga_b200 as moga
    for i, d in enumerate(WIDTHS):
        h, dy, w, t = _rows(torch, cuda_device, 9, d, dy_dt, h_dt, i)
        for r, m in enumerate((1e-20, 1e-4, 1e8, 1e13, 1e14, 1e15, 1e16, 1e17)):
            h[r] *= m
        h = h.to(t)
        dx, dw, _ = moga.moga_rms_norm_backward(dy, h, w)
        moga.device_status()
        check_norm_backward(_np(dx), _np(dw), _np(dy), _np(h), _np(w), None, 1e-6, h_dt)
        # each row by itself as well: dw's bound above is that of the largest terms
        for r in range(9):
            dx1, dw1, _ = moga.moga_rms_norm_backward(dy[r:r + 1], h[r:r + 1], w)
            check_norm_backward(_np(dx1), _np(dw1), _np(dy[r:r + 1]), _np(h[r:r + 1]), _np(w), None, 1e-6, h_dt)


@pytest.mark.parametrize("dy_dt,h_dt", PAIRS)
def test_backward_with_a_small_eps(dy_dt, h_dt, cuda_device):
    """1 / sqrt(eps)^3 leaves the fp32 range; a zero row's gradient is dy w / sqrt(eps)."""
    import torch
    import sparse_attention_long_moga_b200 as moga
    for i, d in enumerate(WIDTHS):
        h, dy, w, t = _rows(torch, cuda_device, 4, d, dy_dt, h_dt, 20 + i)
        h[1] = 0
        h[2] *= 1e-3
        h = h.to(t)
        eps = float(np.float32(1e-30))
        dx, dw, _ = moga.moga_rms_norm_backward(dy, h, w, eps=eps)
        moga.device_status()
        check_norm_backward(_np(dx), _np(dw), _np(dy), _np(h), _np(w), None, eps, h_dt)


@pytest.mark.parametrize("dy_dt,h_dt", PAIRS)
def test_backward_of_exceptional_rows(dy_dt, h_dt, cuda_device):
    """NaN and infinity reach their own row (and dw), nothing else; past the range of the sum of squares y is
    constant, so only dres is left."""
    import torch
    import sparse_attention_long_moga_b200 as moga
    for i, d in enumerate(WIDTHS):
        h, dy, w, t = _rows(torch, cuda_device, 10, d, dy_dt, h_dt, 40 + i)
        h[2, 5] = float("nan")
        h[4, 3] = float("inf")
        h[7] *= 1e25
        h = h.to(t)
        dy[8, 1] = float("nan")
        dres = (torch.ones_like(h) * 0.25).to(t)
        dx, dw, _ = moga.moga_rms_norm_backward(dy, h, w, dres=dres)
        moga.device_status()
        for r in (2, 4, 8):
            assert torch.isnan(dx[r]).all()
        assert torch.isnan(dw).all()
        assert torch.equal(dx[7], dres[7])
        good = [0, 1, 3, 5, 6, 9]
        dx1, dw1, _ = moga.moga_rms_norm_backward(dy[good].contiguous(), h[good].contiguous(), w,
                                                  dres=dres[good].contiguous())
        assert torch.equal(dx[good], dx1) and torch.isfinite(dw1).all()


def test_backward_launches_are_resident(cuda_device):
    """All CTAs of a backward launch fit the SMs at once, at every width and type."""
    import torch  # noqa: F401  (the context)
    import sparse_attention_long_moga_b200 as moga
    fn = moga._lib.lib().moga_test_norm_bwd_ctas
    fn.restype = ctypes.c_int64
    fn.argtypes = [ctypes.c_int32] * 3 + [ctypes.POINTER(ctypes.c_int32)]
    n = ctypes.c_int32(0)
    bad = []
    for h_dt, dy_dt in ((1, 1), (0, 1), (0, 0)):
        for d in range(8, 16385, 8):
            want = fn(d, h_dt, dy_dt, ctypes.byref(n))
            if not 1 <= want <= n.value:
                bad.append((d, h_dt, dy_dt, want, n.value))
    assert not bad, (len(bad), bad[:5])
