"""The block operators beside the attention layer, as measured work: RMS norm with the residual's addition (bf16, fp32
or e4m3 output with a scale a row), its backward, the gated feed-forward product (bf16 and e4m3) and its backward.

`own` False: the plain form in elementary torch operations, 32-bit arithmetic, one rounding at the end.
`own` True: the calls a user makes of sparse_attention_long_moga_b200.
"""
import math

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
SCALE_FLOOR = 2.0 ** -100      # least row maximum that the e4m3 scale is taken from
F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
TYPES = {"f32": F32, "bf16": BF16, "e4m3": E4M3}
SIZE = {"f32": 4, "bf16": 2, "e4m3": 1}

# largest costs a drawn case may have (below those of the listed cases)
MOST_NORM_BYTES = 1.2e9
MOST_FFN_FLOPS = {"ffn": 2.0e12, "ffn_bwd": 2.0e12}


def listed():
    return [
        # one token of a 5120-wide stream, on its way into an e4m3 feed-forward: latency
        dict(name="norm_1tok_e4m3", op="norm", N=1, d=5120, x="bf16", res="bf16", out="e4m3"),
        # the 32,760 tokens of a 5 s video, 1536 wide: the norm in front of the Q/K/V projection
        dict(name="norm_32k", op="norm", N=32760, d=1536, x="bf16", res="bf16", out="bf16"),
        # a 5120-wide fp32 residual stream, bf16 branch, e4m3 output
        dict(name="norm_32k_d5120_e4m3", op="norm", N=32760, d=5120, x="bf16", res="f32", out="e4m3"),
        # a small fp32 training step of odd sizes
        dict(name="normbwd_ragged", op="norm_bwd", N=1001, d=136, dy="f32", h="f32", dres=True, branch=False),
        # training on the 63,960 tokens of a 10 s video, fp32 residual stream, gradient for the bf16 branch too
        dict(name="normbwd_64k", op="norm_bwd", N=63960, d=1536, dy="bf16", h="f32", dres=True, branch=True),
        # one token through a 5120-wide block: the weights' read is the time
        dict(name="ffn_1tok", op="ffn", N=1, d=5120, F=13824, x="bf16", act="silu"),
        # a handful of tokens, e4m3
        dict(name="ffn_17tok_e4m3", op="ffn", N=17, d=1536, F=4096, x="e4m3", act="silu"),
        # odd sizes, tails on every axis
        dict(name="ffn_ragged", op="ffn", N=1001, d=136, F=360, x="bf16", act="gelu"),
        # the 5 s video's tokens
        dict(name="ffn_32k", op="ffn", N=32760, d=1536, F=4096, x="bf16", act="silu"),
        # half of them, 5120 wide, both operands in e4m3
        dict(name="ffn_16k_d5120_e4m3", op="ffn", N=16380, d=5120, F=13824, x="e4m3", act="gelu"),
        # backward at odd sizes
        dict(name="ffnbwd_ragged", op="ffn_bwd", N=777, d=264, F=712, act="gelu"),
        # backward on the 5 s video's tokens
        dict(name="ffnbwd_32k", op="ffn_bwd", N=32760, d=1536, F=4096, act="silu"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "ffn", "ffn", "ffn_bwd"])
    N = _log_int(rng, 1 if op in ("norm", "ffn") else 64, 65536)
    d = 8 * _log_int(rng, 8, 1024 if op.startswith("norm") else 640)
    if op == "norm":
        x, res = rng.choice([("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("bf16", "none"), ("f32", "none")])
        h = x if res == "none" else res
        out = rng.choice(["bf16", "e4m3"] + (["f32"] if h == "f32" else []))
        c = dict(op=op, N=N, d=d, x=x, res=res, out=out)
    elif op == "norm_bwd":
        dy, h = rng.choice([("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
        c = dict(op=op, N=N, d=d, dy=dy, h=h, dres=rng.random() < 0.7, branch=h == "f32" and rng.random() < 0.5)
    else:
        F = 8 * _log_int(rng, 16, 1728)
        c = dict(op=op, N=N, d=d, F=F, act=rng.choice(["silu", "gelu"]))
        if op == "ffn":
            c["x"] = rng.choice(["bf16", "bf16", "e4m3"])
            if c["x"] == "e4m3":
                c["d"] = max(64, d // 16 * 16)
    over = work(c)["bytes"] / MOST_NORM_BYTES if op.startswith("norm") else work(c)["flops"] / MOST_FFN_FLOPS[op]
    if over > 1:
        c["N"] = max(1, int(c["N"] / over))
    return c


def work(case):
    N, d = case["N"], case["d"]
    if case["op"] == "norm":
        e = SIZE[case["x"]] + SIZE[case["out"]]
        if case["res"] != "none":
            e += 2 * SIZE[case["res"]]
        return {"bytes": N * d * e + 4 * d + (4 * N if case["out"] == "e4m3" else 0), "flops": 6 * N * d}
    if case["op"] == "norm_bwd":
        e = SIZE[case["dy"]] + SIZE[case["h"]] * (2 + (1 if case["dres"] else 0)) + (2 if case["branch"] else 0)
        return {"bytes": N * d * e + 8 * d, "flops": 10 * N * d}
    F = case["F"]
    if case["op"] == "ffn":
        e = SIZE[case["x"]]
        scales = 4 * (N + 2 * F) if case["x"] == "e4m3" else 0
        return {"bytes": e * (N * d + 2 * F * d) + 2 * N * F + scales, "flops": 4 * N * d * F}
    return {"bytes": 2 * (2 * N * d + 4 * F * d + N * F), "flops": 12 * N * d * F}


def _normal(gen, shape, dtype, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=F32).mul_(std).to(dtype)


def _quantise_rows(t):
    """e4m3 rows with their scales, as weights are laid out once for serving."""
    s = t.abs().amax(1, keepdim=True).clamp_min(SCALE_FLOOR) / E4M3_MAX
    return (t / s).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3), s.reshape(-1).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    N, d = case["N"], case["d"]
    s = dict(case=case)
    if case["op"] == "norm":
        # a branch's output beside a stream that has grown over the layers; one row in 64 is small
        s["x"] = _normal(gen, (N, d), TYPES[case["x"]])
        s["res"] = None if case["res"] == "none" else _normal(gen, (N, d), TYPES[case["res"]], 3.0)
        small = torch.rand((N, 1), generator=gen, device="cuda") < 1 / 64
        s["x"] = torch.where(small, s["x"] * 1e-3, s["x"]).contiguous()
        s["w"] = 1 + _normal(gen, (d,), F32, 0.2)
    elif case["op"] == "norm_bwd":
        s["h"] = _normal(gen, (N, d), TYPES[case["h"]], 3.0)
        s["dy"] = _normal(gen, (N, d), TYPES[case["dy"]], 1e-2)
        s["dres"] = _normal(gen, (N, d), TYPES[case["h"]], 1e-2) if case["dres"] else None
        s["w"] = 1 + _normal(gen, (d,), F32, 0.2)
    else:
        F = case["F"]
        wg, wu = (_normal(gen, (F, d), F32, 1 / math.sqrt(d)) for _ in range(2))
        x = _normal(gen, (N, d), F32)
        if case["op"] == "ffn" and case["x"] == "e4m3":
            s["x"], s["xs"] = _quantise_rows(x)
            s["wg"], s["gs"] = _quantise_rows(wg)
            s["wu"], s["us"] = _quantise_rows(wu)
        else:
            s["x"], s["wg"], s["wu"] = x.to(BF16), wg.to(BF16), wu.to(BF16)
        if case["op"] == "ffn_bwd":
            s["dh"] = _normal(gen, (N, F), BF16, 1e-2)
    return s


# ------------------------------------------------------------------ plain forms

C_GELU = math.sqrt(2 / math.pi)


def _act(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    return 0.5 * g * (1 + torch.tanh(C_GELU * (g + 0.044715 * g * g * g)))


def _act_grad(g, act):
    if act == "silu":
        s = 1 / (1 + torch.exp(-g))
        return s * (1 + g * (1 - s))
    t = torch.tanh(C_GELU * (g + 0.044715 * g * g * g))
    return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * C_GELU * (1 + 3 * 0.044715 * g * g)


def _plain_norm(s):
    c = s["case"]
    x, w = s["x"], s["w"]
    h = x if s["res"] is None else (x.float() + s["res"].float()).to(s["res"].dtype)
    f = h.float()
    y = f * torch.rsqrt((f * f).mean(1, keepdim=True) + EPS) * w
    out = {} if s["res"] is None else {"h": h}
    if c["out"] == "e4m3":
        scale = y.abs().amax(1, keepdim=True).clamp_min(SCALE_FLOOR) / E4M3_MAX
        out["y"] = (y / scale).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3)
        out["scale"] = scale.reshape(-1)
    else:
        out["y"] = y.to(TYPES[c["out"]])
    return out


def _plain_norm_bwd(s):
    h, dy = s["h"].float(), s["dy"].float()
    r = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    dyw = dy * s["w"]
    dx = r * (dyw - h * (r * r * (dyw * h).mean(1, keepdim=True)))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    out = {"dx": dx.to(s["h"].dtype), "dw": (dy * h * r).sum(0)}
    if s["case"]["branch"]:
        out["dx_branch"] = dx.to(BF16)
    return out


def _plain_ffn(s):
    x, wg, wu = s["x"].float(), s["wg"].float(), s["wu"].float()
    g, u = x @ wg.T, x @ wu.T
    if s["case"]["x"] == "e4m3":
        g = g * s["xs"][:, None] * s["gs"]
        u = u * s["xs"][:, None] * s["us"]
    return {"out": (_act(g, s["case"]["act"]) * u).to(BF16)}


def _plain_ffn_bwd(s):
    x, wg, wu, dh, act = s["x"].float(), s["wg"].float(), s["wu"].float(), s["dh"].float(), s["case"]["act"]
    g, u = x @ wg.T, x @ wu.T
    dg, du = dh * u * _act_grad(g, act), dh * _act(g, act)
    return {"dx": (dg @ wg + du @ wu).to(BF16), "dw_gate": (dg.T @ x).to(BF16), "dw_up": (du.T @ x).to(BF16)}


# ------------------------------------------------------------------ the framework's calls

def _own_run(s):
    import sparse_attention_long_moga_b200 as moga
    c = s["case"]
    if c["op"] == "norm":
        y, h, scale = moga.moga_rms_norm(s["x"], s["w"], residual=s["res"], eps=EPS, out_dtype=TYPES[c["out"]])
        out = {} if s["res"] is None else {"h": h}
        out["y"] = y
        if scale is not None:
            out["scale"] = scale
        return out
    if c["op"] == "norm_bwd":
        dx, dw, dxb = moga.moga_rms_norm_backward(s["dy"], s["h"], s["w"], dres=s["dres"], eps=EPS,
                                                  branch_dtype=BF16 if c["branch"] else None)
        out = {"dx": dx, "dw": dw}
        if dxb is not None:
            out["dx_branch"] = dxb
        return out
    if c["op"] == "ffn":
        if c["x"] == "e4m3":
            return {"out": moga.moga_gated_ffn(s["x"], s["wg"], s["wu"], act=c["act"], x_scale=s["xs"],
                                               w_gate_scale=s["gs"], w_up_scale=s["us"])}
        return {"out": moga.moga_gated_ffn(s["x"], s["wg"], s["wu"], act=c["act"])}
    return moga.moga_gated_ffn_backward(s["x"], s["wg"], s["wu"], s["dh"], act=c["act"])


def run(state):
    if own:
        return _own_run(state)
    op = state["case"]["op"]
    if op == "norm":
        return _plain_norm(state)
    if op == "norm_bwd":
        return _plain_norm_bwd(state)
    return _plain_ffn(state) if op == "ffn" else _plain_ffn_bwd(state)


# ------------------------------------------------------------------ the definition in 64 bits

def _e4m3_of(v):
    """Nearest e4m3 value (3 mantissa bits, least exponent -6, ties to even) of doubles within +-448."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp_min(-6) - 3)
    return torch.round(v / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    D = torch.float64
    if case["op"] == "norm":
        h = s["x"].to(D)
        out = {}
        if s["res"] is not None:
            # the stored sum is a rounding to the stream's type: one add of two values of 24 bits at most
            h = (h + s["res"].to(D)).to(s["res"].dtype).to(D)
            out["h"] = h
        y = h / torch.sqrt(h.pow(2).sum(1, keepdim=True) / case["d"] + EPS) * s["w"].to(D)
        if case["out"] == "e4m3":
            scale = y.abs().max(1, keepdim=True).values.clamp(min=SCALE_FLOOR) / E4M3_MAX
            out["y"], out["scale"] = _e4m3_of(y / scale), scale.reshape(-1)
        else:
            out["y"] = y
        return out
    if case["op"] == "norm_bwd":
        h, dy, w = s["h"].to(D), s["dy"].to(D), s["w"].to(D)
        rms = torch.sqrt(h.pow(2).sum(1, keepdim=True) / case["d"] + EPS)
        n = h / rms
        dn = dy * w
        dx = (dn - n * (dn * n).sum(1, keepdim=True) / case["d"]) / rms
        if s["dres"] is not None:
            dx = dx + s["dres"].to(D)
        out = {"dx": dx, "dw": (dy * n).sum(0)}
        if case["branch"]:
            out["dx_branch"] = dx
        return out
    x, wg, wu = s["x"].to(D), s["wg"].to(D), s["wu"].to(D)
    if case["op"] == "ffn" and case["x"] == "e4m3":
        x, wg, wu = x * s["xs"].to(D)[:, None], wg * s["gs"].to(D)[:, None], wu * s["us"].to(D)[:, None]
    g, u = torch.mm(x, wg.t()), torch.mm(x, wu.t())
    if case["act"] == "silu":
        sg = torch.sigmoid(g)
        a, da = g * sg, sg + g * sg * (1 - sg)
    else:
        # 0.5 (1 + tanh z) = sigmoid(2 z)
        z2 = 2 * C_GELU * (g + 0.044715 * g ** 3)
        sg = torch.sigmoid(z2)
        a, da = g * sg, sg + g * sg * (1 - sg) * 2 * C_GELU * (1 + 0.134145 * g ** 2)
    if case["op"] == "ffn":
        return {"out": a * u}
    dh = s["dh"].to(D)
    dg, du = dh * u * da, dh * a
    return {"dx": torch.mm(dg, wg) + torch.mm(du, wu), "dw_gate": torch.mm(dg.t(), x), "dw_up": torch.mm(du.t(), x)}
