"""Refusals and size queries of the operators around the attention (residual norms, gated
feed-forward, projection gradients): every call here ends on the host, before any CUDA work."""

import ctypes

import pytest
import torch

from relu_linear_attention_gb300 import _lib
from relu_linear_attention_gb300 import binding as R

P = [ctypes.c_void_p(0x7F0000000000 + 0x1000 * i) for i in range(1, 17)]  # aligned, never dereferenced
ODD = ctypes.c_void_p(0x7F0000001004)
BAD, UNSUP, WS, OK = _lib.RAPT_ERR_INVALID_ARG, _lib.RAPT_ERR_UNSUPPORTED, _lib.RAPT_ERR_WORKSPACE, _lib.RAPT_OK
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), UNSUP), (dict(act=5), UNSUP), (dict(act=-1), UNSUP), (dict(D=16385), UNSUP),
    (dict(T=-1), BAD), (dict(D=0), BAD), (dict(eps=0.0), BAD), (dict(eps=-1.0), BAD), (dict(eps=NAN), BAD),
    (dict(eps=INF), BAD), (dict(eps=1e-39), BAD), (dict(x=None), BAD), (dict(r=None, h=None), BAD), (dict(w_pre=None), BAD),
    (dict(y=None), BAD), (dict(y=None, gate=None), BAD), (dict(y=None, gate=None, w_post=None), BAD),
    (dict(x=ODD), BAD), (dict(w_post=ODD), BAD), (dict(h=ODD), BAD), (dict(h=P[10]), BAD),
    (dict(T=0), OK), (dict(T=0, x=None, r=None, h=None), OK),
])
def test_residual_norm_fwd_refuses(lib, kw, code):
    a = dict(x=P[0], y=P[1], gate=P[2], dt=1, T=4, D=64, act=4, w_post=P[3], scale=P[4], w_pre=P[5], eps=1e-6,
             r=P[10], h=P[11])
    a.update(kw)
    assert lib.rapt_residual_norm_fwd(a["x"], a["y"], a["gate"], a["dt"], a["T"], a["D"], a["act"], a["w_post"],
                                      a["scale"], a["w_pre"], a["eps"], a["r"], a["h"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dt=9), UNSUP), (dict(act=7), UNSUP), (dict(D=20000), UNSUP), (dict(T=-2), BAD), (dict(eps=NAN), BAD),
    (dict(dr=None, dh=None), BAD), (dict(x=None), BAD), (dict(w_pre=None), BAD), (dict(y=None), BAD),
    (dict(y=None, gate=None, w_post=None, scale=None, dgate=None, dw_post=None, dscale=None), BAD),  # dy without y
    (dict(gate=None), BAD), (dict(w_post=None), BAD), (dict(scale=None), BAD), (dict(dh=None), BAD),
    (dict(dx=P[9]), BAD), (dict(dw_pre=P[11]), BAD), (dict(dscale=P[5]), BAD), (dict(dy=ODD), BAD),
    (dict(ws=None), WS), (dict(wsb=63), WS), (dict(ws=ODD), WS),
])
def test_residual_norm_bwd_refuses(lib, kw, code):
    a = dict(dr=P[0], dh=P[1], x=P[2], y=P[3], gate=P[4], dt=0, T=4, D=64, act=1, w_post=P[5], scale=P[6],
             w_pre=P[7], eps=1e-6, dx=P[8], dy=P[9], dgate=P[10], dw_post=P[11], dscale=P[12], dw_pre=P[13], ws=P[14],
             wsb=1 << 30)
    a.update(kw)
    assert lib.rapt_residual_norm_bwd(*[a[k] for k in (
        "dr dh x y gate dt T D act w_post scale w_pre eps dx dy dgate dw_post dscale dw_pre ws wsb").split()],
        None) == code


def test_workspace_queries(lib):
    q = lib.rapt_residual_norm_bwd_workspace_size
    assert q(0, 64, 1) == 0 and q(1, 64, 1) == 2 * 64 * 4
    assert q(1 << 20, 2048, 1) == q(1 << 21, 2048, 1) > 0  # bounded by the GPU, not by the rows
    assert q(4, 16385, 1) == 0 and q(4, 64, 3) == 0 and q(-1, 64, 1) == 0
    g = lib.rapt_glu_bwd_workspace_size
    assert g(0, 64, 64) == 0 and g(5, 63, 64) == 0 and g(5, 64, 4) == 0
    assert g(16384, 5504, 2048) >= 2 * 16384 * 5504 * 2
    w = lib.rapt_linear_bwd_workspace_size
    assert w(0, 64, 64) == 0 and w(4, 12, 64) == 0
    assert w(65521, 512, 520) > 0  # a long sum of few tiles is split


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), BAD), (dict(F=0), BAD), (dict(K=-8), BAD), (dict(F=60), UNSUP), (dict(K=20), UNSUP),
    (dict(act=5), UNSUP), (dict(x=None), BAD), (dict(wg=None), BAD), (dict(wu=None), BAD), (dict(h=None), BAD),
    (dict(x=ODD), BAD), (dict(h=ODD), BAD), (dict(h=P[1]), BAD), (dict(st=ctypes.c_void_p(0x7F0000001001)), BAD),
    (dict(M=2 ** 31 - 1, F=2 ** 30), BAD), (dict(K=2 ** 31 - 8), BAD), (dict(K=2 ** 24 + 8), BAD),
    (dict(F=2 ** 24 + 8), BAD), (dict(M=2 ** 26 + 1), BAD), (dict(M=0), OK), (dict(M=0, x=None, h=None), OK),
])
def test_glu_fwd_refuses(lib, kw, code):
    a = dict(x=P[0], wg=P[1], wu=P[2], M=4, F=64, K=64, act=1, h=P[3], st=None)
    a.update(kw)
    assert lib.rapt_glu_fwd(a["x"], a["wg"], a["wu"], a["M"], a["F"], a["K"], a["act"], a["h"], a["st"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), BAD), (dict(F=12), UNSUP), (dict(K=4), UNSUP), (dict(act=-3), UNSUP), (dict(dh=None), BAD),
    (dict(x=None), BAD), (dict(wu=None), BAD), (dict(dx=None, dwg=None, dwu=None), BAD), (dict(dwg=None), BAD),
    (dict(dwu=None), BAD), (dict(dwu=P[5]), BAD), (dict(dx=P[1]), BAD), (dict(dwg=P[2]), BAD), (dict(dx=ODD), BAD),
    (dict(ws=None), WS), (dict(ws=ODD), WS), (dict(wsb=1023), WS),
])
def test_glu_bwd_refuses(lib, kw, code):
    a = dict(dh=P[0], x=P[1], wg=P[2], wu=P[3], M=4, F=64, K=64, act=1, dx=P[4], dwg=P[5], dwu=P[6], ws=P[7],
             wsb=1 << 30)
    a.update(kw)
    assert lib.rapt_glu_bwd(a["dh"], a["x"], a["wg"], a["wu"], a["M"], a["F"], a["K"], a["act"], a["dx"], a["dwg"],
                            a["dwu"], None, a["ws"], a["wsb"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), BAD), (dict(N=0), BAD), (dict(M=2 ** 27, N=8, K=8), BAD), (dict(N=12), UNSUP), (dict(K=9), UNSUP), (dict(dy=None), BAD),
    (dict(x=None), BAD), (dict(w=None), BAD), (dict(dx=None, dw=None), BAD), (dict(dx=P[4]), BAD),
    (dict(dx=P[0]), BAD), (dict(dw=P[2]), BAD), (dict(dw=ODD), BAD), (dict(ws=None), WS), (dict(wsb=64), WS),
    (dict(st=ctypes.c_void_p(0x7F0000001002)), BAD),
])
def test_linear_bwd_refuses(lib, kw, code):
    a = dict(dy=P[0], x=P[1], w=P[2], M=65521, N=512, K=520, dx=P[3], dw=P[4], st=None, ws=P[5], wsb=1 << 40)
    a.update(kw)
    assert lib.rapt_linear_bwd(a["dy"], a["x"], a["w"], a["M"], a["N"], a["K"], a["dx"], a["dw"], a["st"], a["ws"],
                               a["wsb"], None) == code


def test_binding_refuses_host_tensors_and_wrong_arguments():
    x, w = torch.zeros(4, 64), torch.ones(64)
    b = torch.zeros(4, 64, dtype=torch.bfloat16)
    wb = torch.zeros(32, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        R.rapt_residual_norm_fwd(x, w_pre=w)
    with pytest.raises(ValueError):
        R.rapt_residual_norm_fwd(x.double(), w_pre=w.double())
    with pytest.raises(ValueError):
        R.rapt_residual_norm_fwd(x, h=x)
    with pytest.raises(ValueError):
        R.rapt_residual_norm_bwd(None, None, x)
    with pytest.raises(ValueError):
        R.rapt_glu_fwd(b, wb, wb)
    with pytest.raises(ValueError):
        R.rapt_glu_bwd(b, b, wb, wb)
    with pytest.raises(ValueError):
        R.rapt_linear_bwd(b, None, None)
    with pytest.raises(ValueError):
        R.rapt_linear_bwd(b, b, None)
    with pytest.raises(ValueError):
        R._act_code("tanh")


@pytest.mark.parametrize("call", [
    lambda lib: lib.rapt_glu_fwd(P[0], P[1], P[2], 4, 60, 64, 1, P[3], None, None),            # F % 8
    lambda lib: lib.rapt_linear_bwd(P[0], P[1], P[2], 4, 64, 20, P[3], P[4], None, P[5], 1 << 40, None),  # K % 8
    lambda lib: lib.rapt_residual_norm_fwd(P[0], P[1], P[2], 1, 4, 16392, 4, P[3], P[4], P[5], 1e-6, P[6], P[7], None),
    lambda lib: lib.rapt_glu_fwd(P[0], P[1], P[2], 4, 64, 64, 9, P[3], None, None),            # activation
])
def test_what_an_unsupported_call_says_names_no_head(lib, call):
    """The operators without heads report sizes and activations by the same code."""
    with pytest.raises(_lib.RaptError) as e:
        _lib.check("f", call(lib))
    assert e.value.code == UNSUP
    assert "head" not in str(e.value) and "size" in str(e.value) and "activation" in str(e.value)
