"""Cases of the selective state space block's operators, and their plain forms.

Three operators, each with the direction that a case names:

  conv        the short causal convolution of each channel over a sequence's tokens, with its activation:
              y_t = act(b + sum_k w_k x_{t-W+1+k}); for prompts (dense, packed) and for single tokens
  scan        the selective scan of a head's state S [N, P]:
              S_t = exp(dt_t A) S_{t-1} + dt_t B_t x_t^T,  y_t = (S_t^T C_t + D x_t) silu(z_t),
              dt = softplus(dt_raw + dt_bias); for prompts (dense, packed) and for single tokens
  layer_norm  y = w (x - mean) / std + b, and its gradients

Sizes: d_model 2048, 16384 tokens (batch 4 of 4096), 65536 packed tokens in documents of 128 to 8192 with
heads of 64 and 256 sequences decoding are the workloads of bench.py; the block's inner width is twice
d_model (64 heads of 64, or 32 of 128) with a state of 128 rows, shared by all heads or by groups of them;
the others are odd or ragged sizes of the same ranges. The scan's and the convolution's inputs are column
slices of the rows z | x | B | C | dt that a projection gives, as a block meets them.
"""

import math
import random

import torch

own = False

EPS = 1e-5
Q = 128  # tokens a chunk of the plain scan
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _conv(name, form, dtype, D, **kw):
    return {"name": name, "op": "conv", "form": form, "dtype": dtype, "D": D, "W": 4, "act": "silu", "first": False,
            "slice": False, **kw}


def _scan(name, form, dtype, H, P, G, N, **kw):
    return {"name": name, "op": "scan", "form": form, "dtype": dtype, "H": H, "P": P, "G": G, "N": N, "z": True,
            "skip": True, "first": False, **kw}


def _norm(name, form, dtype, T, D):
    return {"name": name, "op": "layer_norm", "form": form, "dtype": dtype, "T": T, "D": D}


def listed():
    return [
        # a prompt batch: the x | B | C columns of a projection's rows
        _conv("conv_prefill", "dense", "bf16", 4352, B=4, L=4096, slice=True),
        # packed documents in 32 bits, an odd number of channels
        _conv("conv_packed_odd_f32", "packed", "f32", 1537, T=30011, lo=1, hi=700, docs=5),
        # a prompt batch of the layer workload at twice its width, state carried out for decoding
        _scan("scan_prefill", "dense", "bf16", 64, 64, 1, 128, B=4, L=4096),
        # the packed workload: ragged documents, heads of 64 in groups
        _scan("scan_packed", "packed", "bf16", 32, 64, 4, 64, T=65536, lo=128, hi=8192, docs=1),
        # one long sequence, continued from a carried state: few heads, parallel along the tokens
        _scan("scan_long", "dense", "bf16", 16, 128, 1, 128, B=1, L=32768, first=True, z=False),
        # 32 bits throughout: small heads, odd length, three groups
        _scan("scan_odd_f32", "dense", "f32", 24, 32, 3, 16, B=3, L=1531),
        # decoding the 256 sequences of the decode workload: the state streams through once
        _scan("scan_step", "step", "bf16", 64, 64, 1, 128, B=256),
        # one sequence decoding: latency
        _scan("scan_step_one", "step", "bf16", 64, 64, 1, 128, B=1),
        _conv("conv_step", "step", "bf16", 4352, B=256),
        # the layer workload's norm
        _norm("norm_fwd", "fwd", "bf16", 16384, 2048),
        _norm("norm_bwd", "bwd", "bf16", 16384, 2048),
        # rows that start at any address, in 32 bits, an odd number of them
        _norm("norm_bwd_odd_f32", "bwd", "f32", 4099, 5121),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("conv", "scan", "scan", "layer_norm"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op == "layer_norm":
        D = _between(rng, 64, 16384)
        if rng.random() < 0.6:
            D = -(-D // 8) * 8
        return {"op": op, "form": rng.choice(("fwd", "bwd")), "dtype": dtype, "D": D,
                "T": min(_between(rng, 1, 65536), (1 << 25) // D)}
    form = rng.choice(("dense", "packed", "step"))
    if op == "conv":
        D = _between(rng, 64, 8192)
        sliced = form != "step" and rng.random() < 0.5
        if sliced or rng.random() < 0.5:
            D = -(-D // 8) * 8
        case = {"op": op, "form": form, "dtype": dtype, "D": D, "W": rng.choice((2, 3, 4, 4)),
                "act": rng.choice(("silu", "silu", "none")), "first": form == "dense" and rng.random() < 0.5,
                "slice": sliced}
        most = (1 << 26) // D
    else:
        P, N = rng.choice((16, 32, 64, 64, 128)), rng.choice((16, 32, 64, 128, 128))
        G = rng.choice((1, 1, 2, 4))
        H = G * _between(rng, 1, 96 // G)
        case = {"op": op, "form": form, "dtype": dtype, "H": H, "P": P, "G": G, "N": N, "z": rng.random() < 0.6,
                "skip": rng.random() < 0.8, "first": form == "dense" and rng.random() < 0.5}
        most = min((1 << 33) // (H * P * N), (1 << 21) // H, (90 << 20 if dtype == "bf16" else 45 << 20) // (H * P))
    if form == "step":
        return {**case, "B": max(1, min(_between(rng, 1, 512), (120 << 20) // (H * P * N) if op == "scan" else 512))}
    tokens = max(1, min(_between(rng, 1, 65536), most))
    if form == "dense":
        B = _between(rng, 1, min(32, tokens))
        return {**case, "B": B, "L": tokens // B}
    # documents long enough that their final states stay below the largest case's memory
    least = 8 if op == "conv" else max(32, H * P * N * tokens >> 26)
    hi = _between(rng, min(least, tokens), min(8192, tokens))
    return {**case, "T": tokens, "lo": rng.choice((0, 1, (hi + 1) // 2)), "hi": hi, "docs": rng.randrange(1000)}


def _lengths(case):
    """Document lengths of a packed case, drawn from [lo, hi] until they fill it (the last cut short)."""
    rng, left, lens = random.Random(case["docs"]), case["T"], []
    while left > 0:
        n = min(left, rng.randint(case["lo"], case["hi"]))
        lens.append(n)
        left -= n
    return lens


# ---------------------------------------------------------------- inputs


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)

    def uniform(n, lo, hi):
        return torch.rand((n,), generator=gen, device="cuda", dtype=torch.float32) * (hi - lo) + lo

    s = dict(case)
    if case["op"] == "layer_norm":
        T, D = case["T"], case["D"]
        s.update(x=(normal(T, D, scale=2.0, dtype=torch.float32) + 0.5).to(dt), w=uniform(D, 0.5, 1.5),
                 b=normal(D, scale=0.1, dtype=torch.float32))
        if case["form"] == "bwd":
            s.update(dy=normal(T, D))
        return s
    if case["form"] == "packed":
        lens = _lengths(case)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        s.update(cu=torch.tensor(cu, dtype=torch.int32, device="cuda"), longest=max(lens), n_docs=len(lens))
        rows = (case["T"],)
    else:
        rows = (case["B"], case["L"]) if case["form"] == "dense" else (case["B"],)
    if case["op"] == "conv":
        D, W = case["D"], case["W"]
        if case["slice"]:  # the middle columns of a projection's rows
            x = normal(*rows, 2 * D)[..., D // 16 * 8:D // 16 * 8 + D]
        else:
            x = normal(*rows, D)
        s.update(x=x, w=normal(D, W, scale=W ** -0.5, dtype=torch.float32), b=normal(D, scale=0.1, dtype=torch.float32))
        if case["first"] or case["form"] == "step":
            s.update(state=normal(case["B"], W - 1, D))
        return s
    H, P, G, N = case["H"], case["P"], case["G"], case["N"]
    width = -(-(2 * H * P + H) // 16) * 16  # z | dt of the projection's rows, x | B | C from the convolution
    proj, xbc = normal(*rows, width), normal(*rows, H * P + 2 * G * N)
    step = torch.exp(uniform(H, math.log(1e-3), math.log(0.1)))  # step sizes at dt_raw = 0
    s.update(x=xbc[..., :H * P].unflatten(-1, (H, P)), B_=xbc[..., H * P:H * P + G * N].unflatten(-1, (G, N)),
             C=xbc[..., H * P + G * N:].unflatten(-1, (G, N)), dt=proj[..., 2 * H * P:2 * H * P + H],
             A=-uniform(H, 1.0, 16.0), dt_bias=torch.log(torch.expm1(step)))
    s["z"] = proj[..., :H * P].unflatten(-1, (H, P)) if case["z"] else None
    s["skip"] = uniform(H, 0.5, 1.5) if case["skip"] else None
    if case["first"] or case["form"] == "step":
        s.update(S=normal(case["B"], H, N, P, dtype=torch.float32))
    return s


# ---------------------------------------------------------------- the plain forms


def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _plain_conv(s):
    x, W = s["x"], s["W"]
    D, dt = x.shape[-1], x.dtype
    if s["form"] == "step":
        window = torch.cat((s["state"], x[:, None]), 1)  # [B, W, D]
        y = (window.float() * s["w"].t()).sum(1) + s["b"]
        s["state"].copy_(window[:, 1:].clone())
        return {"out": (_silu(y) if s["act"] == "silu" else y).to(dt), "state": s["state"]}
    if s["form"] == "dense":
        head = s["state"] if s["first"] else x.new_zeros(x.shape[0], W - 1, D)
        long = torch.cat((head, x), 1)
        y = (long.float().unfold(1, W, 1) * s["w"]).sum(-1) + s["b"]
        last = long[:, long.shape[1] - (W - 1):]
    else:
        cu, T = s["cu"].long(), x.shape[0]
        t = torch.arange(T, device=x.device)
        start = cu[torch.searchsorted(cu, t, right=True) - 1]
        taps = torch.arange(W, device=x.device) - (W - 1)
        live = (t[:, None] + taps) >= start[:, None]  # [T, W]
        long = torch.cat((x.new_zeros(W - 1, D), x)).float()
        y = (torch.where(live[:, None], long.unfold(0, W, 1), 0.0) * s["w"]).sum(-1) + s["b"]
        at = cu[1:, None] + taps[:-1]  # the last W - 1 tokens of each document
        last = torch.where((at >= cu[:-1, None])[..., None], x[at.clamp(min=0)], x.new_zeros(()))
    return {"out": (_silu(y) if s["act"] == "silu" else y).to(dt), "state": last.clone()}


def _step_size(s):
    v = s["dt"].float() + s["dt_bias"]
    return torch.clamp(v, min=0.0) + torch.log1p(torch.exp(-v.abs()))


def _finish(s, y):
    if s["skip"] is not None:
        y = y + s["skip"][:, None] * s["x"].float()
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    return y.to(s["x"].dtype)


def _plain_step(s):
    R = s["H"] // s["G"]
    dt = _step_size(s)
    b, c = (s[k].float().repeat_interleave(R, 1) for k in ("B_", "C"))
    new = torch.exp(dt * s["A"])[..., None, None] * s["S"] + (dt[..., None] * b)[..., None] * s["x"].float()[:, :, None]
    y = (c[..., None, :] @ new)[..., 0, :]
    s["S"].copy_(new)
    return {"out": _finish(s, y), "S": s["S"]}


def _plain_scan(s):
    """Chunks of Q tokens: products of the chunk's scores C B^T under their decays, and of C with the state
    before the chunk, which is the sum of the earlier chunks' increments under theirs."""
    packed = s["form"] == "packed"
    x, dt, b, c = (v[None] if packed else v for v in (s["x"], _step_size(s), s["B_"], s["C"]))
    B, L, H, P = x.shape
    G, N = b.shape[2:]
    R, nc = H // G, -(-L // Q)
    dev = x.device

    def chunks(v):  # [B, L, ...] -> [B, nc, Q, ...], zeros behind the end
        v = torch.cat((v, v.new_zeros((B, nc * Q - L) + v.shape[2:])), 1) if nc * Q > L else v
        return v.reshape((B, nc, Q) + v.shape[2:])

    x, dt, b, c = chunks(x.float()), chunks(dt), chunks(b.float()), chunks(c.float())
    doc = torch.zeros(nc * Q, dtype=torch.long, device=dev)
    if packed:
        cu = s["cu"].long()
        doc = torch.searchsorted(cu, torch.arange(nc * Q, device=dev).clamp(max=L - 1), right=True) - 1
    doc = doc.view(nc, Q)
    # cumulative log decays, in 64 bits: differences of long sums
    cum = (dt.double() * s["A"].double()).cumsum(2).permute(0, 1, 3, 2)  # [B, nc, H, Q]
    seen = (doc[:, :, None] == doc[:, None, :]) & torch.ones(Q, Q, dtype=torch.bool, device=dev).tril()
    decay = torch.exp((cum[..., :, None] - cum[..., None, :]).float().masked_fill(~seen[:, None], -math.inf))
    cb = torch.einsum("bkign,bkjgn->bkgij", c, b)
    dx = (x * dt[..., None]).view(B, nc, Q, G, R, P)
    m = cb[:, :, :, None] * decay.view(B, nc, G, R, Q, Q)
    y = torch.einsum("bkgrij,bkjgrp->bkigrp", m, dx)
    # increments of the chunks, as seen by their last token
    w = torch.exp((cum[..., -1:] - cum).float()).masked_fill((doc != doc[:, -1:])[:, None], 0.0)
    w = w.permute(0, 1, 3, 2).view(B, nc, Q, G, R)
    inc = torch.einsum("bkjgn,bkjgrp->bkgrnp", b, dx * w[..., None])
    first = s["S"].view(B, 1, G, R, N, P) if s["first"] else inc.new_zeros(B, 1, G, R, N, P)
    states = torch.cat((first, inc), 1)
    total = torch.cat((cum.new_zeros(B, 1, H), cum[..., -1]), 1).cumsum(1).permute(0, 2, 1)  # [B, H, nc + 1]
    tail = torch.cat((doc[:1, 0], doc[:, -1]))  # the document that a chunk's end is in
    keep = (tail[:, None] == tail[None]) & torch.ones(nc + 1, nc + 1, dtype=torch.bool, device=dev).tril()
    carry = torch.exp((total[..., :, None] - total[..., None, :]).float().masked_fill(~keep, -math.inf))
    states = torch.einsum("bgrkl,blgrnp->bkgrnp", carry.view(B, G, R, nc + 1, nc + 1), states)
    before, after = states[:, :-1], states[:, -1].reshape(B, H, N, P)
    reach = torch.exp(cum.float()).masked_fill((doc != tail[:-1, None])[:, None], 0.0)  # from the chunk's start
    inter = torch.einsum("bkign,bkgrnp->bkigrp", c, before)
    y = y + inter * reach.permute(0, 1, 3, 2).reshape(B, nc, Q, G, R, 1)
    y = y.reshape(B, nc * Q, H, P)[:, :L]
    if packed:
        end = (cu[1:] - 1).clamp(min=0)
        k, q = end // Q, end % Q
        number = torch.arange(len(end), device=dev)
        mine = (doc[k] == number[:, None]) & (torch.arange(Q, device=dev) <= q[:, None])  # [docs, Q]
        at = cum[0, k]  # [docs, H, Q]
        last = at.gather(2, q.view(-1, 1, 1).expand(-1, H, 1))
        w = torch.exp((last - at).float().masked_fill(~mine[:, None], -math.inf)).permute(0, 2, 1)
        part = torch.einsum("djgn,djgrp->dgrnp", b[0, k], dx[0, k] * w.reshape(-1, Q, G, R, 1))
        on = torch.exp(last.float()).masked_fill((tail[k] != number).view(-1, 1, 1), 0.0)
        after = (part + before[0, k] * on.view(-1, G, R, 1, 1)).reshape(-1, H, N, P)
        after = after.masked_fill((cu[1:] == cu[:-1]).view(-1, 1, 1, 1), 0.0)
        y = y[0]
    return {"out": _finish(s, y), "S": after}


def _plain_norm(s):
    x, dt = s["x"].float(), s["x"].dtype
    xc = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((xc * xc).mean(-1, keepdim=True) + EPS)
    xh = xc * r
    if s["form"] == "fwd":
        return {"y": (xh * s["w"] + s["b"]).to(dt)}
    dy = s["dy"].float()
    g = dy * s["w"]
    dx = r * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    return {"dx": dx.to(dt), "dw": (dy * xh).sum(0), "db": dy.sum(0)}


# ---------------------------------------------------------------- the framework's calls


def _own(s):
    from relu_linear_attention_gb300 import binding as R

    if s["op"] == "layer_norm":
        if s["form"] == "fwd":
            return {"y": R.rapt_layer_norm_fwd(s["x"], s["w"], s["b"], eps=EPS)}
        dx, dw, db = R.rapt_layer_norm_bwd(s["dy"], s["x"], s["w"], eps=EPS)
        return {"dx": dx, "dw": dw, "db": db}
    if s["op"] == "conv":
        if s["form"] == "step":
            out = R.rapt_conv_decode_step(s["x"], s["state"], s["w"], s["b"], act=s["act"])
            return {"out": out, "state": s["state"]}
        if s["form"] == "dense":
            out, state = R.rapt_conv_prefill_fwd(s["x"], s["w"], s["b"], act=s["act"], state=s.get("state"),
                                                 final_state=True)
        else:
            out, state = R.rapt_conv_varlen_fwd(s["x"], s["cu"], s["w"], s["b"], act=s["act"], final_state=True)
        return {"out": out, "state": state}
    args = (s["x"], s["dt"], s["A"], s["B_"], s["C"])
    kw = {"D": s["skip"], "z": s["z"], "dt_bias": s["dt_bias"]}
    if s["form"] == "step":
        return {"out": R.rapt_ssm_decode_step(*args, s["S"], **kw), "S": s["S"]}
    if s["form"] == "dense":
        out, S = R.rapt_ssm_prefill_fwd(*args, S0=s.get("S"), final_state=True, **kw)
    else:
        out, S = R.rapt_ssm_varlen_fwd(*args, s["cu"], max_seqlen=s["longest"], final_state=True, **kw)
    return {"out": out, "S": S}


def run(s):
    if own:
        return _own(s)
    if s["op"] == "layer_norm":
        return _plain_norm(s)
    if s["op"] == "conv":
        return _plain_conv(s)
    return _plain_step(s) if s["form"] == "step" else _plain_scan(s)


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "layer_norm":
        T, D = case["T"], case["D"]
        if case["form"] == "fwd":
            return {"bytes": 2 * T * D * e + 8 * D, "flops": 8 * T * D}
        return {"bytes": 3 * T * D * e + 12 * D, "flops": 14 * T * D}
    if case["form"] == "packed":
        rows, seqs = case["T"], len(_lengths(case))
    else:
        rows, seqs = case["B"] * case.get("L", 1), case["B"]
    carried = 2 if case["first"] or case["form"] == "step" else 1  # the state is read where it is carried in
    if case["op"] == "conv":
        D, W = case["D"], case["W"]
        return {"bytes": 2 * rows * D * e + carried * seqs * (W - 1) * D * e + 4 * D * (W + 1),
                "flops": (2 * W + 5) * rows * D}
    H, P, G, N = case["H"], case["P"], case["G"], case["N"]
    rowbytes = ((3 if case["z"] else 2) * H * P + 2 * G * N + H) * e
    return {"bytes": rows * rowbytes + carried * seqs * H * N * P * 4, "flops": 4 * rows * H * N * P}


# ---------------------------------------------------------------- the definitions in 64 bits


def _exact_conv(s):
    x, W = s["x"], s["W"]
    w, b = s["w"][:, None], s["b"]
    act = torch.nn.functional.silu if s["act"] == "silu" else (lambda v: v)

    def one(doc, head):  # [n, D] behind its W - 1 earlier inputs
        long = torch.cat((head, doc))
        y = torch.nn.functional.conv1d(long.t()[None], w, b, groups=w.shape[0])[0].t() if doc.shape[0] else doc
        return act(y), long[long.shape[0] - (W - 1):]

    zero = x.new_zeros(W - 1, x.shape[-1])
    if s["form"] == "packed":
        cu = s["cu"].tolist()
        got = [one(x[i:j], zero) for i, j in zip(cu, cu[1:])]
        return {"out": torch.cat([g[0] for g in got]), "state": torch.stack([g[1] for g in got])}
    rows = x[:, None] if s["form"] == "step" else x
    got = [one(rows[i], s["state"][i] if "state" in s else zero) for i in range(rows.shape[0])]
    out = torch.stack([g[0] for g in got])
    return {"out": out[:, 0] if s["form"] == "step" else out, "state": torch.stack([g[1] for g in got])}


def _exact_scan(s):
    """The recurrence, token by token, all sequences at once."""
    R = s["H"] // s["G"]
    x, raw, bb, cc, z = s["x"], s["dt"], s["B_"], s["C"], s["z"]
    if s["form"] == "packed":
        n_rows, start, stop = x.shape[0], s["cu"].long()[:-1], s["cu"].long()[1:]
    else:
        B = x.shape[0]
        x, raw, bb, cc, z = (v if v is None else v[:, None] if s["form"] == "step" else v for v in (x, raw, bb, cc, z))
        L = x.shape[1]
        x, raw, bb, cc, z = (v if v is None else v.flatten(0, 1) for v in (x, raw, bb, cc, z))
        n_rows, start = B * L, torch.arange(B, device=x.device) * L
        stop = start + L
    dt = torch.nn.functional.softplus(raw + s["dt_bias"], threshold=60.0)
    if "S" in s:
        S = s["S"].clone()
    else:
        S = torch.zeros(len(start), s["H"], s["N"], s["P"], dtype=torch.float64, device=x.device)
    y = torch.zeros(n_rows + 1, s["H"], s["P"], dtype=torch.float64, device=x.device)
    for t in range(int((stop - start).max())):
        at = start + t
        live = at < stop
        at = at.clamp(max=n_rows - 1)
        step = dt[at] * live[:, None]
        S *= torch.exp(step * s["A"])[..., None, None]
        B_t, C_t = (v[at].repeat_interleave(R, 1) for v in (bb, cc))
        S += (step[..., None] * B_t)[..., None] * x[at][:, :, None]
        y[torch.where(live, at, n_rows)] = torch.einsum("bhn,bhnp->bhp", C_t, S)
    y = y[:n_rows]
    if s["skip"] is not None:
        y = y + s["skip"][:, None] * x
    if z is not None:
        y = y * torch.nn.functional.silu(z)
    return {"out": y.reshape(s["x"].shape), "S": S}


def _exact_norm(s):
    names = ("x", "w", "b")
    if s["form"] == "bwd":
        for k in names:
            s[k].requires_grad_(True)
    mean = torch.mean(s["x"], -1, keepdim=True)
    std = torch.sqrt(torch.mean((s["x"] - mean) ** 2, -1, keepdim=True) + EPS)
    y = s["w"] * ((s["x"] - mean) / std) + s["b"]
    if s["form"] == "fwd":
        return {"y": y}
    return dict(zip(("dx", "dw", "db"), torch.autograd.grad(y, [s[k] for k in names], s["dy"])))


def exact(case, seed):
    s = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v
         for k, v in prepare(case, seed).items()}
    return {"conv": _exact_conv, "scan": _exact_scan, "layer_norm": _exact_norm}[case["op"]](s)
