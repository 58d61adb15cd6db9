"""A selective state space block as a user assembles it: layer norm, a projection to z | x | B | C | dt, the
convolution over the x | B | C columns of its rows, the scan gated by z, the output projection; a prompt and then
token by token, against the same block in 64 bits.

The reference rounds nothing between the steps. Each bf16 tensor on the way adds a relative error of at most half
a step (2^-8) in the 2-norm; with n of them along the longest way (norm, projection, convolution, score, state,
scan, output: 7, and the scan's products take three of them at a time) the result is held to 10 x 2^-8."""

import numpy as np
import pytest
import torch

from oracle import ssm as OS
from relu_linear_attention_gb300 import binding as R
from ssm_inputs import host

pytestmark = pytest.mark.gpu

DM, H, P, G, N, W = 192, 4, 64, 2, 64, 4
HP, GN = H * P, G * N
WIDTH = 2 * HP + 2 * GN + 16  # z | x | B | C | dt and padding


def _parameters():
    g = torch.Generator().manual_seed(3)
    n = lambda *s, scale=1.0: (torch.randn(s, generator=g) * scale).cuda()
    u = lambda k, lo, hi: (torch.rand((k,), generator=g) * (hi - lo) + lo).cuda()
    return dict(w1=u(DM, 0.6, 1.4), b1=n(DM, scale=0.1), w_in=n(WIDTH, DM, scale=DM ** -0.5).bfloat16(),
                w_out=n(DM, HP, scale=HP ** -0.5).bfloat16(), taps=n(HP + 2 * GN, W, scale=0.5),
                cb=n(HP + 2 * GN, scale=0.1), A=-u(H, 1.0, 16.0), D=u(H, 0.5, 1.5), bias=u(H, -4.0, -1.0))


def _split(p, rows, conv):
    """z, x, B, C, dt of the projection's rows and the convolution's."""
    heads = lambda t, *s: t.unflatten(-1, s)
    return (heads(rows[..., :HP], H, P), heads(conv[..., :HP], H, P), heads(conv[..., HP:HP + GN], G, N),
            heads(conv[..., HP + GN:], G, N), rows[..., 2 * HP + 2 * GN:2 * HP + 2 * GN + H])


def _prompt(p, x, cu=None, lens=None):
    h = R.rapt_layer_norm_fwd(x, p["w1"], p["b1"])
    rows = R.rapt_linear_fwd(h.view(-1, DM), p["w_in"]).view(*x.shape[:-1], WIDTH)
    xbc = rows[..., HP:2 * HP + 2 * GN]
    if cu is None:
        conv, tail = R.rapt_conv_prefill_fwd(xbc, p["taps"], p["cb"], final_state=True)
    else:
        conv, tail = R.rapt_conv_varlen_fwd(xbc, cu, p["taps"], p["cb"], final_state=True)
    z, v, b, c, dt = _split(p, rows, conv)
    kw = dict(D=p["D"], z=z, dt_bias=p["bias"], final_state=True)
    if cu is None:
        y, S = R.rapt_ssm_prefill_fwd(v, dt, p["A"], b, c, **kw)
    else:
        y, S = R.rapt_ssm_varlen_fwd(v, dt, p["A"], b, c, cu, max_seqlen=max(lens), **kw)
    return R.rapt_linear_fwd(y.view(-1, HP), p["w_out"]).view(x.shape), tail, S


def _token(p, x, tail, S):
    h = R.rapt_layer_norm_fwd(x, p["w1"], p["b1"])
    rows = R.rapt_linear_fwd(h, p["w_in"])
    conv = R.rapt_conv_decode_step(rows[..., HP:2 * HP + 2 * GN], tail, p["taps"], p["cb"])
    z, v, b, c, dt = _split(p, rows, conv)
    y = R.rapt_ssm_decode_step(v, dt, p["A"], b, c, S, D=p["D"], z=z, dt_bias=p["bias"])
    return R.rapt_linear_fwd(y.view(-1, HP), p["w_out"])


def _reference(p, x):
    """One document x [n, DM] in fp64: (out, S)."""
    q = {k: host(v) for k, v in p.items()}
    h = OS.layer_norm(host(x), q["w1"], q["b1"])
    rows = h @ q["w_in"].T
    conv, _ = OS.conv(rows[:, HP:2 * HP + 2 * GN], q["taps"], q["cb"])
    n = x.shape[0]
    y, S = OS.scan(conv[:, :HP].reshape(n, H, P), rows[:, 2 * HP + 2 * GN:2 * HP + 2 * GN + H], q["A"],
                   conv[:, HP:HP + GN].reshape(n, G, N), conv[:, HP + GN:].reshape(n, G, N), q["D"],
                   rows[:, :HP].reshape(n, H, P), q["bias"])
    return y.reshape(n, HP) @ q["w_out"].T, S


def _near(a, b, what):
    d = np.linalg.norm(host(a) - b) / np.linalg.norm(b)
    assert d <= 10 * 2.0 ** -8, "%s: %.3g" % (what, d)


def test_prompt_then_tokens(cuda_device):
    p = _parameters()
    x = torch.randn(2, 150, DM, generator=torch.Generator().manual_seed(4)).cuda().bfloat16()
    out, tail, S = _prompt(p, x[:, :143].contiguous())
    outs = [out]
    for t in range(143, 150):
        outs.append(_token(p, x[:, t].contiguous(), tail, S)[:, None])
    got = torch.cat(outs, 1)
    for b in range(2):
        ref, refS = _reference(p, x[b])
        _near(got[b], ref, "out")
        _near(got[b, 143:], ref[143:], "tokens")
        _near(S[b], refS, "state")


def test_packed_prompts(cuda_device):
    p = _parameters()
    lens = [3, 200, 1, 128, 61]
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    x = torch.randn(int(cu[-1]), DM, generator=torch.Generator().manual_seed(5)).cuda().bfloat16()
    out, tail, S = _prompt(p, x, torch.from_numpy(cu).cuda(), lens)
    for i in range(len(lens)):
        ref, refS = _reference(p, x[cu[i]:cu[i + 1]])
        _near(out[cu[i]:cu[i + 1]], ref, "document %d" % i)
        _near(S[i], refS, "state %d" % i)


def test_tokens_in_a_captured_graph(cuda_device):
    """The step of a whole block captured once and replayed: the bits of the calls."""
    p = _parameters()
    x = torch.randn(3, 20, DM, generator=torch.Generator().manual_seed(6)).cuda().bfloat16()
    _, tail, S = _prompt(p, x[:, :10].contiguous())
    tail2, S2 = tail.clone(), S.clone()
    want = [_token(p, x[:, t].contiguous(), tail, S) for t in range(10, 20)]
    now, g = x[:, 10].contiguous(), torch.cuda.CUDAGraph()
    keep = tail2.clone(), S2.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _token(p, now, tail2, S2)
    side.synchronize()
    with torch.cuda.graph(g):
        got = _token(p, now, tail2, S2)
    tail2.copy_(keep[0])
    S2.copy_(keep[1])
    for t in range(10, 20):
        now.copy_(x[:, t])
        g.replay()
        assert torch.equal(got, want[t - 10])
    assert torch.equal(S, S2) and torch.equal(tail, tail2)
