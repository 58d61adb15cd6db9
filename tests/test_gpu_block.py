"""A block as a user assembles it from the library's calls: norm, projections, RLA-2 attention, output
projection, join, gated feed-forward, down projection, join; forward and backward, against the same
block in 64 bits differentiated by autograd.

The reference rounds nothing between the steps. Each bf16 tensor on the way to a result adds a relative
error of at most half a step (2^-8), and the steps between them have gains near one (norms, weights of
scale 1 / sqrt(fan-in)), so a result behind n tensors is held to n 2^-8 in the 2-norm, with n counted
along the longest way: 12 forward (h1, q, features, scores, state, a, y, r1, h2, u, f, the result) and
26 backward (the forward's, the gradients of each, and the rounded operands of the products)."""

import numpy as np
import pytest
import torch

from relu_linear_attention_gb300 import binding as R

pytestmark = pytest.mark.gpu

B, L, H, D, F = 2, 150, 2, 64, 264
DM = 192
EPS_NORM, EPS_DEN, BASE = 1e-6, 1e-4, 1e4


def _rms(x):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS_NORM)


def _features(x, gain):
    """ReLU(RoPE(RMSNorm(x))) of [B, L, H, d]: adjacent pairs turn by position base^(-2j/d)."""
    y = _rms(x) * gain
    ang = torch.arange(x.shape[1], dtype=torch.float64)[:, None] * BASE ** (
        -2.0 * torch.arange(D // 2, dtype=torch.float64) / D)
    c, s = torch.cos(ang)[None, :, None], torch.sin(ang)[None, :, None]
    a, b = y[..., 0::2], y[..., 1::2]
    return torch.relu(torch.stack((a * c - b * s, a * s + b * c), -1).flatten(-2))


def _join(x, y, gate, w_post, scale):
    return x + scale * torch.sigmoid(gate) * (w_post * _rms(y))


def _reference(p):
    h1 = p["w1"] * _rms(p["x"])
    qkv = (h1 @ p["w_qkv"].T).view(B, L, 3, H, D)
    q, k, v = _features(qkv[:, :, 0], p["gq"]), _features(qkv[:, :, 1], p["gk"]), qkv[:, :, 2]
    s = torch.einsum("bthd,bshd->bhts", q, k).tril()
    a = torch.einsum("bhts,bshd->bthd", s, v) / (s.sum(-1).permute(0, 2, 1)[..., None] + EPS_DEN)
    y = a.reshape(B, L, H * D) @ p["w_o"].T
    r1 = _join(p["x"], y, p["z1"], p["wp1"], p["s1"])
    h2 = p["w2"] * _rms(r1)
    g, u = h2 @ p["w_gate"].T, h2 @ p["w_up"].T
    f = (torch.nn.functional.silu(g) * u) @ p["w_down"].T
    r2 = _join(r1, f, p["z2"], p["wp2"], p["s2"])
    return r2, p["w3"] * _rms(r2)


def _parameters():
    g = torch.Generator().manual_seed(7)
    n = lambda *s, scale=1.0: (torch.randn(s, generator=g) * scale).to(torch.bfloat16)
    u = lambda *s: torch.rand(s, generator=g) * 0.8 + 0.6
    return dict(x=n(B, L, DM), z1=n(B, L, DM), z2=n(B, L, DM), w_qkv=n(3 * H * D, DM, scale=DM ** -0.5),
                w_o=n(DM, H * D, scale=(H * D) ** -0.5), w_gate=n(F, DM, scale=DM ** -0.5),
                w_up=n(F, DM, scale=DM ** -0.5), w_down=n(DM, F, scale=F ** -0.5), w1=u(DM), w2=u(DM), w3=u(DM),
                wp1=u(DM), wp2=u(DM), s1=u(DM), s2=u(DM), gq=u(H, D), gk=u(H, D)), n(B, L, DM), n(B, L, DM)


def _forward(p, keep):
    x = p["x"]
    _, h1 = R.rapt_residual_norm_fwd(x, w_pre=p["w1"])
    t = h1.view(-1, DM)
    q, k, v = (R.rapt_linear_fwd(t, w.contiguous()).view(B, L, H, D) for w in p["w_qkv"].chunk(3))
    a, _, _ = R.rapt_prefill_fwd(q, k, v, p["gq"], p["gk"])
    y = R.rapt_linear_fwd(a.view(-1, H * D), p["w_o"]).view(B, L, DM)
    r1, h2 = R.rapt_residual_norm_fwd(x, y, gate=p["z1"], w_post=p["wp1"], scale=p["s1"], w_pre=p["w2"])
    u = R.rapt_glu_fwd(h2, p["w_gate"], p["w_up"])
    f = R.rapt_linear_fwd(u.view(-1, F), p["w_down"]).view(B, L, DM)
    r2, h3 = R.rapt_residual_norm_fwd(r1, f, gate=p["z2"], w_post=p["wp2"], scale=p["s2"], w_pre=p["w3"])
    keep.update(h1=h1, q=q, k=k, v=v, a=a, y=y, r1=r1, h2=h2, u=u, f=f)
    return r2, h3


def _backward(p, c, dr2, dh3):
    g = {}
    dr1, df, g["z2"], g["wp2"], g["s2"], g["w3"] = R.rapt_residual_norm_bwd(
        dr2, dh3, c["r1"], c["f"], gate=p["z2"], w_post=p["wp2"], scale=p["s2"], w_pre=p["w3"])
    du, g["w_down"] = R.rapt_linear_bwd(df, c["u"], p["w_down"])
    dh2, g["w_gate"], g["w_up"] = R.rapt_glu_bwd(du, c["h2"], p["w_gate"], p["w_up"])
    dx, dy, g["z1"], g["wp1"], g["s1"], g["w2"] = R.rapt_residual_norm_bwd(
        dr1, dh2, p["x"], c["y"], gate=p["z1"], w_post=p["wp1"], scale=p["s1"], w_pre=p["w2"])
    da, g["w_o"] = R.rapt_linear_bwd(dy.view(-1, DM), c["a"].view(-1, H * D), p["w_o"])
    dq, dk, dv, g["gq"], g["gk"] = R.rapt_prefill_bwd(c["q"], c["k"], c["v"], da.view(B, L, H, D), p["gq"], p["gk"])
    dqkv = torch.cat([t.reshape(B, L, H * D) for t in (dq, dk, dv)], -1)
    dh1, g["w_qkv"] = R.rapt_linear_bwd(dqkv, c["h1"], p["w_qkv"])
    g["x"], _, _, _, _, g["w1"] = R.rapt_residual_norm_bwd(dx, dh1, p["x"], w_pre=p["w1"])
    return g


def _rel(got, ref):
    got, ref = got.detach().double().cpu().numpy(), ref.detach().numpy()
    return float(np.linalg.norm(got - ref) / np.linalg.norm(ref))


def test_block_forward_and_backward(cuda_device, lib):
    host, dr2, dh3 = _parameters()
    p = {k: t.to(cuda_device) for k, t in host.items()}
    ref = {k: t.double().requires_grad_(True) for k, t in host.items()}
    keep = {}
    r2, h3 = _forward(p, keep)
    e2, e3 = _reference(ref)
    assert _rel(r2, e2) <= 12 * 2.0 ** -8 and _rel(h3, e3) <= 12 * 2.0 ** -8
    got = _backward(p, keep, dr2.to(cuda_device), dh3.to(cuda_device))
    ((e2 * dr2.double()).sum() + (e3 * dh3.double()).sum()).backward()
    assert set(got) == set(host)
    for name, t in got.items():
        assert t.shape == host[name].shape and t.dtype == host[name].dtype, name
        assert _rel(t, ref[name].grad) <= 26 * 2.0 ** -8, (name, _rel(t, ref[name].grad))


def test_block_captured_and_replayed_token_by_token(cuda_device, lib):
    """The single-token form (norm, gated feed-forward, join) as one captured graph, replayed on tokens of
    its own, gives each token the bits of a call on it alone, and within rounding of the whole batch."""
    host, _, _ = _parameters()
    p = {k: t.to(cuda_device) for k, t in host.items()}
    x, z = p["x"].view(-1, DM)[:1].clone(), p["z2"].view(-1, DM)[:1].clone()

    def step(x, z):
        _, h = R.rapt_residual_norm_fwd(x, w_pre=p["w2"])
        f = R.rapt_linear_fwd(R.rapt_glu_fwd(h, p["w_gate"], p["w_up"]), p["w_down"])
        return R.rapt_residual_norm_fwd(x, f, gate=z, w_post=p["wp2"], scale=p["s2"], w_pre=p["w3"])

    step(x, z)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x, z)
    whole = step(p["x"].view(-1, DM), p["z2"].view(-1, DM))
    for i in (0, 7, 299):
        xi, zi = p["x"].view(-1, DM)[i:i + 1].contiguous(), p["z2"].view(-1, DM)[i:i + 1].contiguous()
        want = step(xi, zi)
        x.copy_(xi), z.copy_(zi)
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(out, want, whole):
            assert torch.equal(a, b)
            # another kernel forms the products of a batch: they differ by a rounding of h, u, f and the result
            d = (a.float() - c[i:i + 1].float()).norm() / c[i:i + 1].float().norm()
            assert float(d) <= 4 * 2.0 ** -8


def test_binding_refuses_wrong_tensors(cuda_device, lib):
    bf, dev = torch.bfloat16, cuda_device
    x, w = torch.zeros(4, 64, device=dev, dtype=bf), torch.ones(64, device=dev)
    wg = torch.zeros(32, 64, device=dev, dtype=bf)
    wide = torch.zeros(4, 128, device=dev, dtype=bf)
    with pytest.raises(ValueError):
        R.rapt_residual_norm_fwd(wide[:, :64], w_pre=w)                   # strided rows
    with pytest.raises(ValueError):
        R.rapt_residual_norm_fwd(x, x.float(), w_pre=w)                   # another type
    with pytest.raises(ValueError):
        R.rapt_residual_norm_fwd(x, w_pre=w.to(bf))                       # gains are fp32
    with pytest.raises(ValueError):
        R.rapt_residual_norm_fwd(x, x[:2], w_pre=w)
    with pytest.raises(ValueError):
        R.rapt_residual_norm_bwd(x, x, x, w_pre=w, act="tanh")
    with pytest.raises(R._lib.RaptError):
        R.rapt_residual_norm_fwd(x, gate=x, w_pre=w)                      # a gate without a block output
    with pytest.raises(R._lib.RaptError):
        R.rapt_residual_norm_fwd(x, w_pre=w, eps=0.0)
    with pytest.raises(R._lib.RaptError):
        R.rapt_residual_norm_bwd(x, x, x, w_pre=w, workspace=torch.empty(16, device=dev, dtype=torch.uint8))
    with pytest.raises(ValueError):
        R.rapt_glu_fwd(x, wg, wg.t().contiguous())
    with pytest.raises(ValueError):
        R.rapt_glu_fwd(x.float(), wg.float(), wg.float())
    with pytest.raises(R._lib.RaptError):
        R.rapt_glu_fwd(x[:, :60].contiguous(), wg[:, :60].contiguous(), wg[:, :60].contiguous())
    with pytest.raises(ValueError):
        R.rapt_glu_bwd(x, x, wg, wg)                                      # dh has F columns
    with pytest.raises(R._lib.RaptError):
        R.rapt_glu_bwd(x[:, :32].contiguous(), x, wg, wg, need_dx=False, need_dw=False)
    with pytest.raises(R._lib.RaptError):
        R.rapt_glu_bwd(x[:, :32].contiguous(), x, wg, wg, workspace=torch.empty(64, device=dev, dtype=torch.uint8))
    with pytest.raises(ValueError):
        R.rapt_linear_bwd(x, x, wg)                                       # dy has N columns
    with pytest.raises(ValueError):
        R.rapt_linear_bwd(x, x, x, dx=x.cpu())
