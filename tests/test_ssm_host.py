"""Host-only checks of the selective state space block's C ABI: refusals before anything is launched, calls
without rows, workspace sizes, and the binding's checks of layouts. No GPU is needed."""

import ctypes

import pytest
import torch

from relu_linear_attention_gb300 import _lib, binding as R

BAD, NOT, WS = _lib.RAPT_ERR_INVALID_ARG, _lib.RAPT_ERR_UNSUPPORTED, _lib.RAPT_ERR_WORKSPACE
P = [0x7F0000000000 + (i << 20) for i in range(16)]  # 16-byte aligned, never dereferenced
F32, BF16 = _lib.RAPT_F32, _lib.RAPT_BF16


def inputs(**kw):
    a = dict(x=P[0], dt=P[1], B=P[2], C=P[3], z=None, x_stride=512, dt_stride=8, B_stride=128, C_stride=128,
             z_stride=0, A=P[4], D=None, dt_bias=None, H=8, P=64, G=2, Ns=64, dt_softplus=1, dtype=BF16)
    a.update(kw)
    return _lib.rapt_ssm_inputs(**a)


def prefill(lib, rows=1, L=8, S0=None, out=P[5], Sf=None, st=None, ws=P[9], wsb=1 << 40, **kw):
    return lib.rapt_ssm_prefill_fwd(ctypes.byref(inputs(**kw)), rows, L, S0, out, Sf, st, ws, wsb, None)


REFUSED = [
    (dict(P=48), NOT), (dict(Ns=256), NOT), (dict(dtype=2), NOT), (dict(H=0), BAD), (dict(G=0), BAD), (dict(G=3), BAD),
    (dict(x=None), BAD), (dict(dt=None), BAD), (dict(B=None), BAD), (dict(C=None), BAD), (dict(A=None), BAD),
    (dict(out=None), BAD), (dict(x=P[0] + 8), BAD), (dict(B=P[2] + 4), BAD), (dict(z=P[6] + 2, z_stride=512), BAD),
    (dict(dt=P[1] + 1), BAD), (dict(A=P[4] + 4), BAD), (dict(x_stride=504), BAD), (dict(x_stride=516), BAD),
    (dict(C_stride=64), BAD), (dict(dt_stride=7), BAD), (dict(z=P[6], z_stride=0), BAD), (dict(x_stride=1 << 38), BAD),
    (dict(out=P[0]), BAD), (dict(out=P[2]), BAD), (dict(S0=P[7], Sf=P[7]), BAD), (dict(Sf=P[5]), BAD),
    (dict(S0=P[7] + 8), BAD), (dict(st=P[8] + 2), BAD), (dict(B_stride=-128), BAD),
]


@pytest.mark.parametrize("kw,code", REFUSED)
def test_scan_refuses(lib, kw, code):
    assert prefill(lib, **kw) == code


def test_scan_refuses_sizes(lib):
    assert prefill(lib, L=-1) == BAD
    assert lib.rapt_ssm_prefill_fwd(None, 1, 8, None, P[5], None, None, None, 0, None) == BAD
    for B, L in ((0, 8), (1 << 20, 1 << 11), (1 << 23, 1)):
        assert lib.rapt_ssm_prefill_fwd(ctypes.byref(inputs()), B, L, None, P[5], None, None, P[9], 1 << 40, None) == BAD


def test_scan_without_tokens_does_nothing(lib):
    assert prefill(lib, L=0, x=None, dt=None, out=None) == _lib.RAPT_OK


def test_scan_varlen_refuses(lib):
    def call(T=64, cu=P[6], N=2, longest=64, **kw):
        return lib.rapt_ssm_varlen_fwd(ctypes.byref(inputs(**kw)), T, cu, N, longest, None, P[5], None, None, P[9],
                                       1 << 40, None)
    for kw in (dict(T=-1), dict(cu=None), dict(cu=P[6] + 2), dict(N=0), dict(longest=-1), dict(T=(1 << 30) + 1), dict(H=0)):
        assert call(**kw) == BAD, kw
    assert call(P=8) == NOT


def test_scan_step_refuses(lib):
    def call(N=4, S=P[7], out=P[5], **kw):
        return lib.rapt_ssm_decode_step(ctypes.byref(inputs(**kw)), N, S, out, None)
    for kw in (dict(N=0), dict(S=None), dict(S=P[7] + 4), dict(S=P[0]), dict(out=None), dict(out=P[3]), dict(S=P[5]),
               dict(x_stride=100), dict(dt=None)):
        assert call(**kw) == BAD, kw
    assert call(Ns=8) == NOT


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scan_workspace(lib, dtype):
    """Few heads and a long document are cut, and refuse a workspace that is missing, small or misaligned."""
    a = inputs(dtype=dtype)
    need = lib.rapt_ssm_prefill_workspace_size(ctypes.byref(a), 1, 32768)
    assert need >= 8 * 64 * 64 * 4
    assert need == lib.rapt_ssm_varlen_workspace_size(ctypes.byref(a), 32768, 1, 32768)
    for ws, wsb in ((None, need), (P[9], need - 1), (P[9] + 8, need)):
        assert prefill(lib, L=32768, dtype=dtype, ws=ws, wsb=wsb) == WS
    assert lib.rapt_ssm_prefill_workspace_size(ctypes.byref(a), 1, 8) == 0
    assert lib.rapt_ssm_prefill_workspace_size(ctypes.byref(inputs(P=40)), 1, 32768) == 0


CONV = [P[0], 64, BF16, 2, 8, 64, P[1], P[2], 4, 1, P[3], P[4], P[5], None]


@pytest.mark.parametrize("at,v,code", [
    (0, None, BAD), (0, P[0] + 4, BAD), (1, 63, BAD), (2, 3, NOT), (3, 0, BAD), (4, -1, BAD), (5, 0, BAD),
    (5, 1 << 25, BAD), (6, None, BAD), (6, P[1] + 4, BAD), (7, P[2] + 8, BAD), (8, 1, NOT), (8, 5, NOT), (9, 9, NOT),
    (10, P[3] + 2, BAD), (11, None, BAD), (11, P[0], BAD), (11, P[3], BAD), (12, P[4], BAD), (12, P[3], BAD),
    (4, (1 << 30) + 1, BAD),
])
def test_conv_refuses(lib, at, v, code):
    a = list(CONV)
    a[at] = v
    assert lib.rapt_conv_prefill_fwd(*a) == code


def test_conv_varlen_and_step_refuse(lib):
    a = [P[0], 64, BF16, 16, 64, P[6], 2, P[1], P[2], 4, 1, P[3], P[4], P[5], None, None]
    for at, v in ((5, None), (5, P[6] + 2), (6, 0), (3, -1), (3, (1 << 30) + 1), (14, P[7] + 1), (12, P[0]), (13, P[12 - 9])):
        b = list(a)
        b[at] = v
        assert lib.rapt_conv_varlen_fwd(*b) == BAD, (at, v)
    s = [P[0], 64, BF16, 4, 64, P[1], P[2], 4, 1, P[3], P[4], None]
    for at, v in ((0, None), (3, 0), (5, None), (9, None), (9, P[0]), (10, P[3]), (10, None), (1, 8)):
        b = list(s)
        b[at] = v
        assert lib.rapt_conv_decode_step(*b) == BAD, (at, v)


def test_conv_without_tokens_does_nothing(lib):
    a = list(CONV)
    a[0], a[4], a[11], a[12] = None, 0, None, None
    assert lib.rapt_conv_prefill_fwd(*a) == _lib.RAPT_OK


@pytest.mark.parametrize("at,v,code", [
    (0, None, BAD), (0, P[0] + 2, BAD), (1, 5, NOT), (2, -1, BAD), (3, 0, BAD), (3, 16385, NOT), (4, P[1] + 4, BAD),
    (5, P[2] + 4, BAD), (6, 0.0, BAD), (6, float("nan"), BAD), (6, 1e-39, BAD), (7, None, BAD), (7, P[3] + 4, BAD),
    (7, P[1], BAD), (7, P[2], BAD)])
def test_layer_norm_refuses(lib, at, v, code):
    a = [P[0], BF16, 4, 64, P[1], P[2], 1e-5, P[3], None]
    a[at] = v
    assert lib.rapt_layer_norm_fwd(*a) == code


@pytest.mark.parametrize("at,v,code", [
    (0, None, BAD), (1, None, BAD), (2, 5, NOT), (3, -1, BAD), (4, 16385, NOT), (5, P[2] + 4, BAD), (6, -1.0, BAD),
    (7, P[4], BAD), (7, P[2], BAD), (8, P[2], BAD), (8, P[5], BAD), (9, P[1], BAD), (10, None, WS), (11, 0, WS),
    (10, P[6] + 4, WS)])
def test_layer_norm_backward_refuses(lib, at, v, code):
    a = [P[0], P[1], BF16, 4, 64, P[2], 1e-5, P[3], P[4], P[5], P[6], 1 << 30, None]
    a[at] = v
    assert lib.rapt_layer_norm_bwd(*a) == code


def test_a_size_past_32_bits_is_refused(lib):
    for at in (3, 4, 5, 8, 9, 2):
        a = list(CONV)
        a[4] = 0
        a[at] += 1 << 32
        assert lib.rapt_conv_prefill_fwd(*a) in (BAD, NOT), at
    n = [P[0], BF16, 0, 64, P[1], P[2], 1e-5, P[3], None]
    assert lib.rapt_layer_norm_fwd(*n) == _lib.RAPT_OK
    for at in (1, 2, 3):
        b = list(n)
        b[at] += 1 << 32
        assert lib.rapt_layer_norm_fwd(*b) in (BAD, NOT), at
    for B, L in ((1 + (1 << 32), 0), (1, 1 << 32)):
        assert prefill_raw(lib, B, L) == BAD


def prefill_raw(lib, B, L):
    return lib.rapt_ssm_prefill_fwd(ctypes.byref(inputs()), B, L, None, P[5], P[6], None, None, 0, None)


def test_rows_of_a_wider_matrix():
    """The binding takes column slices as they are, at the stride of their rows, and refuses what has none."""
    m = torch.zeros(2, 5, 96)
    at = lambda t, lead, index=-1: R._rows("t", t, torch.float32, torch.Size(lead), t.shape[len(lead):], index)
    class Fake:  # a CPU tensor that says that it is on device 0
        def __init__(self, t): self.t = t
        def __getattr__(self, k): return getattr(self.t, k)
        def get_device(self): return 0
    rows = lambda t, lead: R._rows("t", Fake(t), torch.float32, torch.Size(lead), t.shape[len(lead):], 0)
    assert rows(m[..., 32:64], (2, 5))[1] == 96
    assert rows(m[..., 32:64].unflatten(-1, (4, 8)), (2, 5))[1] == 96
    assert rows(m[:1, :1, :32], (1, 1))[1] == 32          # a single row has no stride
    assert rows(m[:, :1, :32], (2, 1))[1] == 480
    assert rows(m[:0, :, :32], (0, 5))[1] == 32
    for t, lead in ((m.transpose(0, 1), (5, 2)), (m[:, ::2, :32][..., ::2], (2, 3)), (m[:, :3, :32], (2, 3)),
                    (m[..., :32].unflatten(-1, (4, 8)).transpose(-1, -2), (2, 5))):
        with pytest.raises(ValueError):
            rows(t, lead)
    with pytest.raises(ValueError):
        at(m, (2, 5))  # not on a GPU
