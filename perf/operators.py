"""Cases of the operators around the attention of a RAPT block, and their plain forms.

Three operators, each with the direction that a case names:

  residual_norm  the join of a block's output with the residual stream and the norm of the next block:
                 n = w_post y / rms(y),  r = x + scale act(gate) n,  h = w_pre r / rms(r)
  glu            the gated feed-forward: h = act(x w_gate^T) (x w_up^T)
  linear         the gradients of a projection y = x w^T

Sizes: d_model 2048 and 16384 tokens (batch 4 of 4096) with the q | k | v projection 2048 -> 6144 are
the layer workload of bench.py, 256 sequences its decode workload; 5504 is the usual 8/3 d_model hidden
size rounded up to 128; the others are odd or ragged sizes of the same ranges.
"""

import math

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ("none", "silu", "gelu", "relu", "sigmoid")


def _norm(name, direction, T, D, dtype, act):
    return {"name": name, "op": "residual_norm", "dir": direction, "T": T, "D": D, "dtype": dtype, "act": act}


def _glu(name, direction, M, K, F, act):
    return {"name": name, "op": "glu", "dir": direction, "M": M, "K": K, "F": F, "act": act}


def _linear(name, M, N, K):
    return {"name": name, "op": "linear", "dir": "bwd", "M": M, "N": N, "K": K}


def listed():
    return [
        # one token of one sequence while decoding: latency alone
        _norm("norm_fwd_token", "fwd", 1, 2048, "bf16", "sigmoid"),
        # prefill or training of the layer workload
        _norm("norm_fwd_prefill", "fwd", 16384, 2048, "bf16", "sigmoid"),
        # rows that start at any address: an odd width
        _norm("norm_fwd_odd_f32", "fwd", 3001, 1537, "f32", "silu"),
        _norm("norm_bwd_prefill", "bwd", 16384, 2048, "bf16", "sigmoid"),
        # wide rows in 32 bits, an odd number of them
        _norm("norm_bwd_wide_f32", "bwd", 4099, 5120, "f32", "sigmoid"),
        # decoding: one token reads every weight once
        _glu("glu_fwd_token", "fwd", 1, 2048, 5504, "silu"),
        # decoding: the 256 sequences of the decode workload
        _glu("glu_fwd_decode", "fwd", 256, 2048, 5504, "silu"),
        _glu("glu_fwd_prefill", "fwd", 16384, 2048, 5504, "silu"),
        # a training step of the layer workload
        _glu("glu_bwd_train", "bwd", 16384, 2048, 5504, "silu"),
        # no size a multiple of any tile
        _glu("glu_bwd_ragged", "bwd", 1531, 1032, 2744, "gelu"),
        # training of the q | k | v projection
        _linear("linear_bwd_qkv", 16384, 6144, 2048),
        # few weights, a long sum over tokens
        _linear("linear_bwd_long", 65521, 512, 520),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("residual_norm", "glu", "linear"))
    if op == "residual_norm":
        direction = rng.choice(("fwd", "bwd"))
        D = _between(rng, 64, 8192)
        if rng.random() < 0.6:
            D = -(-D // 8) * 8
        T = min(_between(rng, 1, 65536), (1 << 25) // D)
        return {"op": op, "dir": direction, "T": T, "D": D, "dtype": rng.choice(("bf16", "f32")),
                "act": rng.choice(ACTS)}
    K = 8 * _between(rng, 8, 512)
    M = _between(rng, 1, 32768)
    if op == "glu":
        F = 8 * _between(rng, 16, 1024)
        M = max(1, min(M, 16384 * 2048 * 5504 // (F * K)))
        return {"op": op, "dir": rng.choice(("fwd", "bwd")), "M": M, "K": K, "F": F, "act": rng.choice(ACTS)}
    N = 16 * _between(rng, 8, 512)
    M = max(1, min(M, 16384 * 6144 * 2048 // (N * K)))
    return {"op": op, "dir": "bwd", "M": M, "N": N, "K": K}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)

    def gain(n, lo, hi):
        return torch.rand((n,), generator=gen, device="cuda", dtype=torch.float32) * (hi - lo) + lo

    s = {"op": case["op"], "dir": case["dir"], "act": case.get("act")}
    if case["op"] == "residual_norm":
        T, D, dt = case["T"], case["D"], DTYPES[case["dtype"]]
        s.update(x=normal(T, D, scale=2.0, dtype=dt), y=normal(T, D, dtype=dt), gate=normal(T, D, dtype=dt),
                 w_post=gain(D, 0.8, 1.2), scale=gain(D, 0.1, 1.0), w_pre=gain(D, 0.8, 1.2))
        if case["dir"] == "bwd":
            s.update(dr=normal(T, D, dtype=dt), dh=normal(T, D, dtype=dt))
    elif case["op"] == "glu":
        M, K, F = case["M"], case["K"], case["F"]
        s.update(x=normal(M, K), w_gate=normal(F, K, scale=K ** -0.5), w_up=normal(F, K, scale=K ** -0.5))
        if case["dir"] == "bwd":
            s.update(dh=normal(M, F))
    else:
        M, N, K = case["M"], case["N"], case["K"]
        s.update(dy=normal(M, N), x=normal(M, K), w=normal(N, K, scale=K ** -0.5))
    return s


# ---------------------------------------------------------------- the plain forms


def _act(name, z):
    """act(z) and its derivative."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        on = (z > 0).to(z.dtype)
        return z * on, on
    if name == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(z * 0.5 ** 0.5))
        return z * cdf, cdf + z * torch.exp(-0.5 * z * z) * (2.0 * math.pi) ** -0.5
    sig = 1.0 / (1.0 + torch.exp(-z))
    if name == "sigmoid":
        return sig, sig * (1.0 - sig)
    return z * sig, sig * (1.0 + z * (1.0 - sig))


def _plain_norm_fwd(s):
    dt = s["x"].dtype
    y, x = s["y"].float(), s["x"].float()
    n = s["w_post"] * (y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS))
    r = x + s["scale"] * _act(s["act"], s["gate"].float())[0] * n
    h = s["w_pre"] * (r * torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS))
    return {"r": r.to(dt), "h": h.to(dt)}


def _plain_norm_bwd(s):
    dt = s["x"].dtype
    y, x, dr, dh = s["y"].float(), s["x"].float(), s["dr"].float(), s["dh"].float()
    a, da = _act(s["act"], s["gate"].float())
    ry = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS)
    yh = y * ry
    n = s["w_post"] * yh
    r = x + s["scale"] * a * n
    rr = torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS)
    rh = r * rr
    t = s["w_pre"] * dh
    g = dr + rr * (t - rh * (t * rh).mean(-1, keepdim=True))
    dn = s["scale"] * a * g
    u = s["w_post"] * dn
    return {"dx": g.to(dt), "dy": (ry * (u - yh * (u * yh).mean(-1, keepdim=True))).to(dt),
            "dgate": (s["scale"] * n * da * g).to(dt), "dw_post": (dn * yh).sum(0),
            "dscale": (a * n * g).sum(0), "dw_pre": (dh * rh).sum(0)}


def _plain_glu_fwd(s):
    x = s["x"].float()
    g, u = x @ s["w_gate"].float().t(), x @ s["w_up"].float().t()
    return {"h": (_act(s["act"], g)[0] * u).to(s["x"].dtype)}


def _plain_glu_bwd(s):
    dt = s["x"].dtype
    x, wg, wu, dh = s["x"].float(), s["w_gate"].float(), s["w_up"].float(), s["dh"].float()
    a, da = _act(s["act"], x @ wg.t())
    dg, du = dh * (x @ wu.t()) * da, dh * a
    return {"dx": (dg @ wg + du @ wu).to(dt), "dw_gate": (dg.t() @ x).to(dt), "dw_up": (du.t() @ x).to(dt)}


def _plain_linear_bwd(s):
    dt = s["x"].dtype
    dy = s["dy"].float()
    return {"dx": (dy @ s["w"].float()).to(dt), "dw": (dy.t() @ s["x"].float()).to(dt)}


_PLAIN = {("residual_norm", "fwd"): _plain_norm_fwd, ("residual_norm", "bwd"): _plain_norm_bwd,
          ("glu", "fwd"): _plain_glu_fwd, ("glu", "bwd"): _plain_glu_bwd, ("linear", "bwd"): _plain_linear_bwd}


# ---------------------------------------------------------------- the framework's calls


def _own(s):
    from relu_linear_attention_gb300 import binding as R

    if s["op"] == "residual_norm":
        if s["dir"] == "fwd":
            r, h = R.rapt_residual_norm_fwd(s["x"], s["y"], gate=s["gate"], w_post=s["w_post"], scale=s["scale"],
                                            w_pre=s["w_pre"], act=s["act"], eps=EPS)
            return {"r": r, "h": h}
        dx, dy, dgate, dw_post, dscale, dw_pre = R.rapt_residual_norm_bwd(
            s["dr"], s["dh"], s["x"], s["y"], gate=s["gate"], w_post=s["w_post"], scale=s["scale"],
            w_pre=s["w_pre"], act=s["act"], eps=EPS)
        return {"dx": dx, "dy": dy, "dgate": dgate, "dw_post": dw_post, "dscale": dscale, "dw_pre": dw_pre}
    if s["op"] == "glu":
        if s["dir"] == "fwd":
            return {"h": R.rapt_glu_fwd(s["x"], s["w_gate"], s["w_up"], act=s["act"])}
        dx, dw_gate, dw_up = R.rapt_glu_bwd(s["dh"], s["x"], s["w_gate"], s["w_up"], act=s["act"])
        return {"dx": dx, "dw_gate": dw_gate, "dw_up": dw_up}
    dx, dw = R.rapt_linear_bwd(s["dy"], s["x"], s["w"])
    return {"dx": dx, "dw": dw}


def run(s):
    if own:
        return _own(s)
    return _PLAIN[s["op"], s["dir"]](s)


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    if case["op"] == "residual_norm":
        T, D, e = case["T"], case["D"], 2 if case["dtype"] == "bf16" else 4
        if case["dir"] == "fwd":
            return {"bytes": 5 * T * D * e + 3 * D * 4, "flops": 20 * T * D}
        return {"bytes": 8 * T * D * e + 6 * D * 4, "flops": 50 * T * D}
    if case["op"] == "glu":
        M, K, F = case["M"], case["K"], case["F"]
        if case["dir"] == "fwd":
            return {"bytes": 2 * (M * K + 2 * F * K + M * F), "flops": 4 * M * F * K}
        return {"bytes": 2 * (2 * M * K + 4 * F * K + M * F), "flops": 12 * M * F * K}
    M, N, K = case["M"], case["N"], case["K"]
    return {"bytes": 2 * (M * N + 2 * M * K + 2 * N * K), "flops": 4 * M * N * K}


# ---------------------------------------------------------------- the definitions in 64 bits


def _exact_act(name, z):
    if name == "none":
        return z
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return torch.nn.functional.gelu(z)
    return torch.relu(z) if name == "relu" else torch.sigmoid(z)


def _rms(v):
    return v / torch.sqrt(torch.mean(v ** 2, dim=-1, keepdim=True) + EPS)


def exact(case, seed):
    """The forward from its definition in 64 bits; the gradients by differentiating that forward."""
    s = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in prepare(case, seed).items()}
    if case["op"] == "residual_norm":
        names = ("x", "y", "gate", "w_post", "scale", "w_pre")
        if case["dir"] == "bwd":
            for k in names:
                s[k].requires_grad_(True)
        r = s["x"] + _rms(s["y"]) * s["w_post"] * _exact_act(case["act"], s["gate"]) * s["scale"]
        h = _rms(r) * s["w_pre"]
        if case["dir"] == "fwd":
            return {"r": r, "h": h}
        got = torch.autograd.grad([r, h], [s[k] for k in names], [s["dr"], s["dh"]], allow_unused=True,
                                  materialize_grads=True)
        return dict(zip(["d" + k for k in names], got))
    if case["op"] == "glu":
        names = ("x", "w_gate", "w_up")
        if case["dir"] == "bwd":
            for k in names:
                s[k].requires_grad_(True)
        h = _exact_act(case["act"], torch.matmul(s["x"], s["w_gate"].T)) * torch.matmul(s["x"], s["w_up"].T)
        if case["dir"] == "fwd":
            return {"h": h}
        return dict(zip(["d" + k for k in names], torch.autograd.grad(h, [s[k] for k in names], s["dh"])))
    x, w = s["x"].requires_grad_(True), s["w"].requires_grad_(True)
    dx, dw = torch.autograd.grad(torch.matmul(x, w.T), [x, w], s["dy"])
    return {"dx": dx, "dw": dw}
