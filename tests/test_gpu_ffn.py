"""GPU parity of the gated feed-forward (bf16 and e4m3) and of its backward against the fp64 oracle (tolerances:
_block.py)."""
import pytest

from _block import check_ffn, check_ffn_backward
from _block import to_np as _np

pytestmark = pytest.mark.gpu

SHAPES = [(1, 16, 8), (100, 16, 8), (2000, 16, 8), (1, 64, 128), (1, 1536, 264), (2, 80, 136), (7, 528, 96), (8, 128, 16), (9, 256, 520),
          (16, 1536, 512), (17, 144, 360), (31, 2048, 128), (32, 96, 1032), (33, 512, 256), (64, 1536, 384),
          (65, 208, 72), (127, 128, 128), (129, 512, 264), (256, 1536, 512), (257, 1552, 1032), (600, 1536, 4096),
          (2100, 64, 2056)]


def _inputs(torch, dev, N, d, F, seed, e4m3=False):
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn((N, d), generator=g, device=dev)
    wg, wu = (torch.randn((F, d), generator=g, device=dev) * (2 / d ** 0.5) for _ in range(2))
    do = torch.randn((N, F), generator=g, device=dev).to(torch.bfloat16)
    if not e4m3:
        return [t.to(torch.bfloat16) for t in (x, wg, wu)], do
    out = []
    for t in (x, wg, wu):
        s = t.abs().amax(1, keepdim=True) / 448
        out.append(((t / s).to(torch.float8_e4m3fn), s.reshape(-1).contiguous()))
    return out, do


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("N,d,F", SHAPES)
def test_forward_bf16(N, d, F, act, cuda_device):
    import torch
    import sparse_attention_long_moga_b200 as moga
    (x, wg, wu), _ = _inputs(torch, cuda_device, N, d, F, N + d + F)
    out = moga.moga_gated_ffn(x, wg, wu, act=act)
    moga.device_status()
    assert out.dtype == torch.bfloat16 and out.shape == (N, F)
    check_ffn(_np(out), _np(x), _np(wg), _np(wu), act)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("N,d,F", SHAPES)
def test_forward_e4m3(N, d, F, act, cuda_device):
    import torch
    import sparse_attention_long_moga_b200 as moga
    ((x, xs), (wg, gs), (wu, us)), _ = _inputs(torch, cuda_device, N, d, F, N + d + F, e4m3=True)
    out = moga.moga_gated_ffn(x, wg, wu, act=act, x_scale=xs, w_gate_scale=gs, w_up_scale=us)
    moga.device_status()
    check_ffn(_np(out), _np(x.float()) * _np(xs)[:, None], _np(wg.float()) * _np(gs)[:, None],
               _np(wu.float()) * _np(us)[:, None], act)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("N,d,F", SHAPES)
def test_backward(N, d, F, act, cuda_device):
    import torch
    import sparse_attention_long_moga_b200 as moga
    (x, wg, wu), do = _inputs(torch, cuda_device, N, d, F, N + d + F)
    got = moga.moga_gated_ffn_backward(x, wg, wu, do, act=act)
    moga.device_status()
    check_ffn_backward(got, _np(x), _np(wg), _np(wu), _np(do), act)
    again = moga.moga_gated_ffn_backward(x, wg, wu, do, act=act)
    only_x = moga.moga_gated_ffn_backward(x, wg, wu, do, act=act, need_dw=False)
    only_w = moga.moga_gated_ffn_backward(x, wg, wu, do, act=act, need_dx=False)
    for k in ("dx", "dw_gate", "dw_up"):
        assert torch.equal(got[k], again[k])
    assert only_x["dw_gate"] is None and only_x["dw_up"] is None and torch.equal(only_x["dx"], got["dx"])
    assert only_w["dx"] is None and torch.equal(only_w["dw_up"], got["dw_up"])
    moga.device_status()


# 512-row gradient tiles: ragged on every side; units that end on a half; K of dx split as well
@pytest.mark.parametrize("N,d,F,act", [(1100, 1536, 4104, "silu"), (2600, 1288, 3080, "gelu"), (3415, 280, 13232, "silu")])
def test_backward_of_many_tiles(N, d, F, act, cuda_device):
    import torch
    import sparse_attention_long_moga_b200 as moga
    (x, wg, wu), do = _inputs(torch, cuda_device, N, d, F, N + d + F)
    got = moga.moga_gated_ffn_backward(x, wg, wu, do, act=act)
    moga.device_status()
    check_ffn_backward(got, _np(x), _np(wg), _np(wu), _np(do), act)
    for kw in (dict(need_dx=False), dict(need_dw=False)):
        alone = moga.moga_gated_ffn_backward(x, wg, wu, do, act=act, **kw)
        assert all(torch.equal(got[k], v) for k, v in alone.items() if v is not None)


def test_narrowest_bf16(cuda_device):
    """d = 8: one 16-byte row of x, less than a box on every side."""
    import torch
    import sparse_attention_long_moga_b200 as moga
    for N in (3, 70, 600):
        (x, wg, wu), do = _inputs(torch, cuda_device, N, 8, 8, N)
        check_ffn(_np(moga.moga_gated_ffn(x, wg, wu)), _np(x), _np(wg), _np(wu), "silu")
        check_ffn_backward(moga.moga_gated_ffn_backward(x, wg, wu, do), _np(x), _np(wg), _np(wu), _np(do), "silu")
    moga.device_status()


def test_large_gates_and_zeros(cuda_device):
    """Gates far out on both sides of the activation, zero tokens and zero weights: finite, and as the formula."""
    import torch
    import sparse_attention_long_moga_b200 as moga
    for N in (5, 200):
        for act in ("silu", "gelu"):
            (x, wg, wu), do = _inputs(torch, cuda_device, N, 128, 256, 3)
            wg *= 64                    # gates of some hundreds
            x[1] = 0
            wu[5] = 0
            out = moga.moga_gated_ffn(x, wg, wu, act=act)
            assert torch.isfinite(out.float()).all() and not out[1].any() and not out[:, 5].any()
            check_ffn(_np(out), _np(x), _np(wg), _np(wu), act)
            got = moga.moga_gated_ffn_backward(x, wg, wu, do, act=act)
            assert all(torch.isfinite(t.float()).all() for t in got.values())


def test_bad_token_stays_in_its_row(cuda_device):
    """NaN in one token reaches that token's outputs only."""
    import torch
    import sparse_attention_long_moga_b200 as moga
    for N in (9, 300):
        (x, wg, wu), _ = _inputs(torch, cuda_device, N, 136, 264, 4)
        good = moga.moga_gated_ffn(x, wg, wu)
        x[3, 5] = float("nan")
        out = moga.moga_gated_ffn(x, wg, wu)
        assert torch.isnan(out[3].float()).all()
        keep = [i for i in range(N) if i != 3]
        assert torch.equal(out[keep], good[keep])


def test_offsets_past_32_bits(cuda_device):
    """More than 2^31 outputs: the last rows equal a small call's; their gradients, whose K may be split differently
    there, are the oracle's."""
    import torch
    import sparse_attention_long_moga_b200 as moga
    N, d, F = 270_000, 64, 8192
    (x, wg, wu), _ = _inputs(torch, cuda_device, 512, d, F, 5)
    big = x.repeat((N + 511) // 512, 1)[:N].contiguous()
    out = moga.moga_gated_ffn(big, wg, wu)
    small = moga.moga_gated_ffn(x, wg, wu)
    n = N % 512
    assert torch.equal(out[-n:], small[:n]) and torch.equal(out[:512], small)
    got = moga.moga_gated_ffn_backward(big, wg, wu, out, need_dw=False)
    moga.device_status()
    for rows in (slice(N - n, N), slice(0, n)):
        check_ffn_backward(dict(dx=got["dx"][rows]), _np(x[:n]), _np(wg), _np(wu), _np(small[:n]), "silu", keys=("dx",))
