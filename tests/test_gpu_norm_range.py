"""GPU: the norm's backward on rows of extreme magnitude and its launches' residence, the e4m3 output next to its
rounding borders (oracle and tolerances: _block.py)."""
import ctypes

import numpy as np
import pytest

from _block import check_norm_backward
from _block import to_np as _np
from oracle import block

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


# ------------------------------------------------------- e4m3: values next to a rounding border

SUBNORMAL_TIES = (2 * np.arange(8) + 1) * 2.0 ** -10
NORMAL_TIES = np.concatenate([(2 * (8 + np.arange(8)) + 1) * 2.0 ** (e - 3) / 2 for e in range(-6, 9)])
NORMAL_TIES = NORMAL_TIES[NORMAL_TIES < 448]


def _nearest(hw, top):
    """(lower, upper) e4m3 values that hw 448 / top may round to, equal but at an exact tie.  hw and top are products
    of two fp32 values, so |hw| 448 and tie top are exact in float64 and their order decides."""
    a = np.abs(hw)
    v = a * 448.0 / top
    step = 2 * block.e4m3_half_step(v)
    lo = np.floor(v / step) * step
    left, right = a * 448.0, (lo + step / 2) * top
    return np.where(left > right, lo + step, lo), np.where(left < right, lo, lo + step)


def _check_nearest(moga, torch, dev, h, w, copies=1):
    ht = torch.from_numpy(np.tile(h, (copies, 1))).to(dev)
    q, _, _ = moga.moga_rms_norm(ht, torch.from_numpy(w).to(dev), out_dtype=torch.float8_e4m3fn)
    moga.device_status()
    hw = h.astype(np.float64) * w.astype(np.float64)
    lo, hi = _nearest(hw, np.max(np.abs(hw), axis=1, keepdims=True))
    got = np.abs(_np(q.float()))[:len(h)]
    assert torch.equal(q.view(torch.uint8).view(copies, len(h), -1)[-1], q.view(torch.uint8)[:len(h)])
    bad = (got < lo) | (got > hi)
    assert not bad.any(), "%d of %d" % (bad.sum(), bad.size)


def _near(ties, top, w, ulps):
    """fp32 h with h w within some ulps of tie top / 448."""
    c = (ties * top / 448 / w).astype(np.float32)
    return (c.view(np.int32) + ulps).view(np.float32)


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("d,copies", [(120, 1), (120, 200), (248, 200), (1024, 1), (1024, 6), (2048, 3), (5120, 2)])
@pytest.mark.parametrize("ties", [SUBNORMAL_TIES, NORMAL_TIES], ids=["subnormal", "normal"])
def test_e4m3_nearest_value(ties, d, copies, weighted, cuda_device):
    """Values within two fp32 steps of a tie, whose fp32 product often lies on its other side."""
    import torch
    import sparse_attention_long_moga_b200 as moga
    rng = np.random.default_rng(d + copies)
    h = np.empty((64, d), dtype=np.float32)
    w = rng.uniform(0.5, 2, d).astype(np.float32) if weighted else np.ones(d, dtype=np.float32)
    for r in range(64):
        h[r, 0] = rng.uniform(4, 8)        # the largest product: no tie reaches it
        w[0] = 2 if weighted else 1
        top = float(h[r, 0]) * float(w[0])
        t = rng.choice(ties, d - 1)
        h[r, 1:] = _near(t, top, w[1:].astype(np.float64), rng.integers(-2, 3, d - 1).astype(np.int32))
        h[r, 1:] *= rng.choice([-1, 1], d - 1).astype(np.float32)
        h[r, rng.integers(1, d, d // 16)] = 0
    _check_nearest(moga, torch, cuda_device, h, w, copies)


def _equal_products(rng):
    """(h1, w1, h2, w2): products that round to one fp32 value, the second exact one the larger by half a step."""
    while True:
        h1, w1 = (rng.uniform(1.5, 2, 4000).astype(np.float32) for _ in range(2))
        w2 = rng.uniform(1.5, 2, 4000).astype(np.float32)
        t = h1 * w1
        h2 = t / w2
        e1, e2 = (h.astype(np.float64) * w - t.astype(np.float64) for h, w in ((h1, w1), (h2, w2)))
        ulp = np.spacing(t)
        ok = np.nonzero((h2 * w2 == t) & (e1 < -0.3 * ulp) & (e2 > 0.3 * ulp))[0]
        if len(ok):
            i = ok[0]
            return h1[i], w1[i], h2[i], w2[i]


@pytest.mark.parametrize("order", [0, 1])
def test_e4m3_of_equal_largest_products(order, cuda_device):
    """Two products of one thread that round to the same fp32 value: the exactly larger one is the row's maximum."""
    import torch
    import sparse_attention_long_moga_b200 as moga
    rng = np.random.default_rng(order)
    d = 2048
    for _ in range(24):
        h1, w1, h2, w2 = _equal_products(rng)
        h, w = np.empty((1, d), dtype=np.float32), np.ones(d, dtype=np.float32)
        a, b = (2, 6) if order == 0 else (6, 2)
        top = float(h2) * float(w2)
        h[0] = _near(rng.choice(NORMAL_TIES, d), top, 1.0, rng.integers(-1, 2, d).astype(np.int32))
        h[0, a], w[a], h[0, b], w[b] = h1, w1, h2, w2
        _check_nearest(moga, torch, cuda_device, h, w)


def test_e4m3_products_past_the_range(cuda_device):
    """Where h w passes the fp32 range the row's scale says so (infinite or NaN); its neighbours are untouched."""
    import torch
    import sparse_attention_long_moga_b200 as moga
    for N, d in ((5, 1536), (9500, 64)):
        h = torch.randn((N, d), generator=torch.Generator(device=cuda_device).manual_seed(d), device=cuda_device)
        h[1] *= 1e17          # the sum of squares stays in the range, the products do not
        h[3] = 3e38           # neither does
        w = torch.full((d,), 2.0, device=cuda_device)
        w[5] = 1e23
        good = [r for r in range(N) if r not in (1, 3)]
        q, _, s = moga.moga_rms_norm(h, w, out_dtype=torch.float8_e4m3fn)
        q1, _, s1 = moga.moga_rms_norm(h[good].contiguous(), w, out_dtype=torch.float8_e4m3fn)
        moga.device_status()
        assert not torch.isfinite(s[[1, 3]]).any()
        assert torch.equal(s[good], s1) and torch.equal(q.view(torch.uint8)[good], q1.view(torch.uint8))
