"""The block operators as a user's program runs them: together around the attention layer, captured and replayed, on
other streams, two at once, in buffers with neighbours.  Results are checked against the fp64 oracle stage by stage
(tolerances: _block.py), or bit for bit against the plain call."""
import numpy as np
import pytest

from _block import check_ffn, check_ffn_backward, check_norm_backward, check_norm_y
from _block import to_np as _np
from _data import Case
from oracle import block
from synth import workloads as W

pytestmark = pytest.mark.gpu

EPS = 1e-6
WL = W.Workload("block_2shot", T=4, h=8, w=16, d=128, H=2, hd=64, M=3, shots=(2, 2), tg_max=0, win_h=4, win_w=8)


def _rand(torch, dev, shape, seed, scale=1.0, dt=None):
    g = torch.Generator(device=dev).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=dev) * scale).to(dt or torch.bfloat16)


def _rows_e4m3(torch, t):
    s = t.float().abs().amax(1, keepdim=True) / 448
    return (t.float() / s).to(torch.float8_e4m3fn), s.reshape(-1).contiguous()


@pytest.mark.parametrize("stream_dt", ["bf16", "f32"])
@pytest.mark.parametrize("e4m3", [False, True])
def test_block_around_the_attention_layer(stream_dt, e4m3, cuda_device):
    """norm -> projection and router -> attention -> norm with the residual -> gated feed-forward -> down projection ->
    norm with the residual, and the backward of its second half."""
    import torch
    import sparse_attention_long_moga_b200 as moga
    wl, F, dt = WL, 264 if not e4m3 else 272, {"bf16": torch.bfloat16, "f32": torch.float32}[stream_dt]
    case = Case(wl, with_qkv=False)
    d = wl.d
    stream = _rand(torch, cuda_device, (wl.N, d), 1, dt=dt)
    w1, w2, w3 = (1 + _rand(torch, cuda_device, (d,), 2 + i, 0.2, torch.float32) for i in range(3))
    w_qkv = _rand(torch, cuda_device, (3 * wl.H * wl.hd, d), 5, d ** -0.5)
    w_r = _rand(torch, cuda_device, (d, wl.M), 6, d ** -0.5)
    wg, wu = (_rand(torch, cuda_device, (F, d), 7 + i, d ** -0.5) for i in range(2))
    w_down = _rand(torch, cuda_device, (d, F), 9, F ** -0.5)

    y1, h0, _ = moga.moga_rms_norm(stream, w1, eps=EPS)
    assert h0 is stream
    check_norm_y(_np(y1), None, block.rms_norm(_np(stream), _np(w1), EPS)[0], "bf16")
    q, k, v, g, gate, _ = moga.moga_qkv_route(y1, w_qkv, w_r, None, wl.H, wl.hd)
    perm, cu, _, _ = moga.moga_permute(g, wl.M)
    attn = moga.stga_attn_mean(q, k, v, case.geom, moga.moga_group_attn(q, k, v, perm, cu, gate, wl.M))
    branch = attn.reshape(wl.N, d)
    out_dt = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    y2, h1, s2 = moga.moga_rms_norm(branch, w2, residual=stream, eps=EPS, out_dtype=out_dt)
    assert torch.equal(h1, (branch.float() + stream.float()).to(dt))
    check_norm_y(_np(y2.float()), None if s2 is None else _np(s2), block.rms_norm(_np(h1), _np(w2), EPS)[0],
                 "e4m3" if e4m3 else "bf16")
    if e4m3:
        (qg, gs), (qu, us) = _rows_e4m3(torch, wg), _rows_e4m3(torch, wu)
        a = moga.moga_gated_ffn(y2, qg, qu, x_scale=s2, w_gate_scale=gs, w_up_scale=us)
        check_ffn(_np(a), _np(y2.float()) * _np(s2)[:, None], _np(qg.float()) * _np(gs)[:, None],
                  _np(qu.float()) * _np(us)[:, None], "silu")
    else:
        a = moga.moga_gated_ffn(y2, wg, wu)
        check_ffn(_np(a), _np(y2), _np(wg), _np(wu), "silu")
    b = a @ w_down.T
    y3, h2, _ = moga.moga_rms_norm(b, w3, residual=h1, eps=EPS)
    assert torch.equal(h2, (b.float() + h1.float()).to(dt))
    check_norm_y(_np(y3), None, block.rms_norm(_np(h2), _np(w3), EPS)[0], "bf16")
    moga.device_status()
    if e4m3:
        return
    # backward of the second half, from a gradient of y3: each stage takes the one before's output
    dy3 = _rand(torch, cuda_device, (wl.N, d), 10)
    dh2, dw3, db = moga.moga_rms_norm_backward(dy3, h2, w3, eps=EPS,
                                               branch_dtype=torch.bfloat16 if stream_dt == "f32" else None)
    check_norm_backward(_np(dh2), _np(dw3), _np(dy3), _np(h2), _np(w3), None, EPS, stream_dt)
    da = (dh2 if db is None else db) @ w_down
    got = moga.moga_gated_ffn_backward(y2, wg, wu, da)
    check_ffn_backward(got, _np(y2), _np(wg), _np(wu), _np(da), "silu")
    dh1, dw2, dbr = moga.moga_rms_norm_backward(got["dx"], h1, w2, dres=dh2, eps=EPS,
                                                branch_dtype=torch.bfloat16 if stream_dt == "f32" else None)
    check_norm_backward(_np(dh1), _np(dw2), _np(got["dx"]), _np(h1), _np(w2), _np(dh2), EPS, stream_dt)
    assert (dbr is None) == (stream_dt == "bf16") and (dh1 if dbr is None else dbr).shape == branch.shape
    moga.device_status()


def _calls(torch, dev, seed, N=300, d=136, F=264):
    """(name, inputs, call) of each operator, forward and backward, both few and many tokens."""
    import sparse_attention_long_moga_b200 as moga
    out = []
    for n in (9, N):
        x, res, dy = (_rand(torch, dev, (n, d), seed + i) for i in range(3))
        w = _rand(torch, dev, (d,), seed + 3, dt=torch.float32)
        wg, wu = (_rand(torch, dev, (F, d), seed + 4 + i, d ** -0.5) for i in range(2))
        do = _rand(torch, dev, (n, F), seed + 6)
        out += [("norm", (x, res, w), lambda x, res, w: moga.moga_rms_norm(x, w, residual=res)[:2]),
                ("norm e4m3", (x, w), lambda x, w: moga.moga_rms_norm(x, w, out_dtype=torch.float8_e4m3fn)[::2]),
                ("norm bwd", (dy, x, w, res), lambda dy, x, w, r: moga.moga_rms_norm_backward(dy, x, w, dres=r)[:2]),
                ("ffn", (x, wg, wu), lambda x, wg, wu: (moga.moga_gated_ffn(x, wg, wu),)),
                ("ffn bwd", (x, wg, wu, do),
                 lambda x, wg, wu, do: tuple(moga.moga_gated_ffn_backward(x, wg, wu, do, act="gelu").values()))]
    return out


def _same(torch, a, b):
    return all(torch.equal(s.view(torch.uint8) if s.dtype == torch.float8_e4m3fn else s,
                           t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t) for s, t in zip(a, b))


def test_captured_and_replayed(cuda_device):
    """Two graphs of every call, replayed in turn on inputs that change, give the plain calls' bits."""
    import torch
    import sparse_attention_long_moga_b200 as moga
    first, second = _calls(torch, cuda_device, 1), _calls(torch, cuda_device, 50)
    fresh = [[_calls(torch, cuda_device, s)[i][1] for i in range(len(first))] for s in (100, 200)]
    side = torch.cuda.Stream()
    graphs = []
    for calls in (first, second):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _, a, f in calls:
                f(*a)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = [f(*a) for _, a, f in calls]
        graphs.append((g, outs))
    for rnd in range(2):
        for calls, (g, _), inputs in zip((first, second), graphs, fresh if rnd == 0 else fresh[::-1]):
            for (_, a, _), b in zip(calls, inputs):
                for s, t in zip(a, b):
                    s.copy_(t)
        for g, _ in graphs:
            g.replay()
        for calls, (_, outs) in zip((first, second), graphs):
            for (name, a, f), o in zip(calls, outs):
                assert _same(torch, o, f(*a)), name
    moga.device_status()


def test_two_streams_at_once(cuda_device):
    """Every call on two streams at the same time, inputs made on those streams."""
    import torch
    import sparse_attention_long_moga_b200 as moga
    want = [[f(*a) for _, a, f in _calls(torch, cuda_device, s)] for s in (1, 2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    made = []
    for st, s in zip(streams, (1, 2)):
        with torch.cuda.stream(st):
            made.append(_calls(torch, cuda_device, s))
    got = [[], []]
    for i in range(len(made[0])):
        for which, st in enumerate(streams):
            with torch.cuda.stream(st):
                _, a, f = made[which][i]
                got[which].append([f(*a) for _ in range(3)])
    torch.cuda.synchronize()
    for which in range(2):
        for (name, _, _), rs, w in zip(made[which], got[which], want[which]):
            assert all(_same(torch, r, w) for r in rs), name
    moga.device_status()


@pytest.mark.parametrize("N,d,F", [(1, 72, 40), (9, 136, 72), (65, 136, 72), (300, 200, 328), (520, 264, 136)])
def test_neighbours_stay_untouched(N, d, F, cuda_device):
    """Outputs and workspaces inside larger buffers: nothing outside of them is written (C ABI)."""
    import torch
    import sparse_attention_long_moga_b200 as moga
    L, P = moga.lib(), moga._ptr
    bufs = []

    def inside(shape, dt):
        n = int(np.prod(shape)) * dt.itemsize
        raw = torch.full((4096 + -(-n // 256) * 256 + 4096,), 0xA5, dtype=torch.uint8, device=cuda_device)
        bufs.append((raw, n))
        return raw[4096:4096 + n].view(dt).reshape(shape)

    bf, f32, f8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
    x, res, dy = (_rand(torch, cuda_device, (N, d), i) for i in range(3))
    w = _rand(torch, cuda_device, (d,), 3, dt=f32)
    wg, wu = (_rand(torch, cuda_device, (F, d), 4 + i, d ** -0.5) for i in range(2))
    do = _rand(torch, cuda_device, (N, F), 6)
    st = moga._stream()
    h, y, q, s = inside((N, d), bf), inside((N, d), bf), inside((N, d), f8), inside((N,), f32)
    assert L.moga_rms_norm(P(x), 1, P(res), 1, P(w), 0, N, d, EPS, P(h), P(y), 1, None, st) == 0
    assert L.moga_rms_norm(P(x), 1, None, 0, P(w), 0, N, d, EPS, None, P(q), 2, P(s), st) == 0
    dx, dw = inside((N, d), bf), inside((d,), f32)
    n = L.moga_rms_norm_bwd_ws_bytes(N, d)
    ws = inside((n,), torch.uint8)
    assert L.moga_rms_norm_bwd(P(dy), 1, P(x), 1, P(w), 0, P(res), N, d, EPS, P(dx), None, P(dw), P(ws), n, st) == 0
    out = inside((N, F), bf)
    assert L.moga_gated_ffn(P(x), P(wg), P(wu), 1, None, None, None, N, d, F, 0, P(out), st) == 0
    gx, gg, gu = inside((N, d), bf), inside((F, d), bf), inside((F, d), bf)
    n = L.moga_gated_ffn_bwd_ws_bytes(N, d, F)
    ws2 = inside((n,), torch.uint8)
    assert L.moga_gated_ffn_bwd(P(x), P(wg), P(wu), N, d, F, 0, P(do), P(gx), P(gg), P(gu), P(ws2), n, st) == 0
    moga.device_status()
    for raw, n in bufs:
        assert (raw[:4096] == 0xA5).all() and (raw[4096 + n:] == 0xA5).all()
    # and what lies inside is the binding's result
    assert _same(torch, (y, h), moga.moga_rms_norm(x, w, residual=res)[:2])
    assert _same(torch, (q, s), moga.moga_rms_norm(x, w, out_dtype=f8)[::2])
    assert _same(torch, (dx, dw), moga.moga_rms_norm_backward(dy, x, w, dres=res)[:2])
    assert _same(torch, (out,), (moga.moga_gated_ffn(x, wg, wu),))
    assert _same(torch, (gx, gg, gu), tuple(moga.moga_gated_ffn_backward(x, wg, wu, do).values()))


def test_gpu_refusals(cuda_device):
    """Refused on the host, with the state untouched: the next call works."""
    import torch
    import sparse_attention_long_moga_b200 as moga
    x, w = _rand(torch, cuda_device, (4, 64), 1), _rand(torch, cuda_device, (64,), 2)
    wg = _rand(torch, cuda_device, (32, 64), 3)
    with pytest.raises(moga.MogaError, match="fp32 output needs an fp32 stream"):
        moga.moga_rms_norm(x, w, out_dtype=torch.float32)
    with pytest.raises(moga.MogaError, match="fp32 x needs an fp32 residual"):
        moga.moga_rms_norm(x.float(), w, residual=x)
    with pytest.raises(moga.MogaError, match="eps must be positive"):
        moga.moga_rms_norm(x, w, eps=0.0)
    with pytest.raises(moga.MogaError, match="N=0"):
        moga.moga_rms_norm(x[:0], w)
    with pytest.raises(moga.MogaError, match="fp32 dy needs an fp32 h"):
        moga.moga_rms_norm_backward(x.float(), x, w)
    with pytest.raises(moga.MogaError, match="dx_branch"):
        moga.moga_rms_norm_backward(x, x, w, branch_dtype=torch.bfloat16)
    with pytest.raises(moga.MogaError, match="multiple of 8"):
        moga.moga_gated_ffn(x, wg[:12], wg[:12])
    with pytest.raises(moga.MogaError, match="no gradient"):
        moga.moga_gated_ffn_backward(x, wg, wg, _rand(torch, cuda_device, (4, 32), 4), need_dx=False, need_dw=False)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        moga.moga_gated_ffn(x, wg.cpu(), wg)
    with pytest.raises(ValueError, match="must be contiguous"):
        moga.moga_rms_norm(x[:, ::2], w[:32])
    with pytest.raises(moga.MogaError, match="16-byte aligned"):
        base = torch.zeros(4 * 64 + 4, dtype=torch.bfloat16, device=cuda_device)
        moga.moga_rms_norm(base[4:].view(4, 64), w)
    y, _, _ = moga.moga_rms_norm(x, w)
    check_norm_y(_np(y), None, block.rms_norm(_np(x), _np(w), EPS)[0], "bf16")
    moga.device_status()


def test_norm_gradient_against_differences(cuda_device):
    """dx along a direction v against the forward's central difference.  y is fp32 with 2^-22 relative error at most, so
    J = sum(dy * y) in float64 is off by 2^-22 sum|dy y| (about 2e-6 x 1e4 = 0.02, and independent errors far less); the
    step e = 2^-6 leaves a truncation of e^2 / 6 |J'''| with J''' of the size of J' / |h|^2 ~ J'.  Against J' ~ 50 both
    are below 2e-2 / 2e + 4e-5 J': the independent errors (0.02 / sqrt(12800) / 2e = 6e-3) are allowed five times."""
    import torch
    import sparse_attention_long_moga_b200 as moga
    N, d, e = 100, 128, 2.0 ** -6
    h, dy, v, dres = (_rand(torch, cuda_device, (N, d), i, dt=torch.float32) for i in range(4))
    w = 1 + _rand(torch, cuda_device, (d,), 5, 0.2, torch.float32)

    def J(t):
        y, _, _ = moga.moga_rms_norm(t, w, eps=EPS, out_dtype=torch.float32)
        return float((dy.double() * y.double()).sum() + (dres.double() * t.double()).sum())
    dx, _, _ = moga.moga_rms_norm_backward(dy, h, w, dres=dres, eps=EPS)
    got = float((dx.double() * v.double()).sum())
    diff = (J(h + e * v) - J(h - e * v)) / (2 * e)
    assert abs(got - diff) <= 3e-2 + 2e-3 * abs(diff)
