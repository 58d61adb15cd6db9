"""The activations of the gates and their derivatives over their whole range, relative to their own size.

In fp32, with x = 0, y = 1 and no gains, the residual norm's r is act(z) itself; of dr = 1 its backward's dy
is act(z) and its dgate act'(z). Bounds in half steps of fp32 (2^-24), from the arithmetic: the exponent
z log2(e) is off by 1.5 |z| of them (the constant's and the product's rounding), z^2 log2(e) / 2 by 1.25 z^2;
the hardware's 2^x by 4, its 1/x by 2, every other operation by 1.
"""

import numpy as np
import pytest
import torch
from scipy.special import erfc, expit

from relu_linear_attention_gb300 import binding as R

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
Z = np.unique(np.concatenate([np.linspace(-12.5, 16.0, 60001), np.geomspace(1e-6, 1, 2000),
                              -np.geomspace(1e-6, 1, 2000)]).astype(np.float32))


def _gates(z, act, device):
    """(act(z) of the forward, act(z) and act'(z) of the backward) in fp32."""
    n = z.size
    z = torch.from_numpy(z).to(device).view(1, -1)
    z = torch.nn.functional.pad(z, (0, -z.shape[1] % 1024)).view(-1, 1024)
    one, zero = torch.ones_like(z), torch.zeros_like(z)
    r, _ = R.rapt_residual_norm_fwd(zero, one, gate=z, act=act)
    _, dy, dz = R.rapt_residual_norm_bwd(one, None, zero, one, gate=z, act=act)[:3]
    return [t.flatten()[:n].double().cpu().numpy() for t in (r, dy, dz)]


def _near(got, ref, budget, what, z=Z):
    bad = ~(np.abs(got - ref) <= budget)
    if bad.any():
        i = np.argmax(np.where(bad, np.abs(got - ref) / budget, 0))
        raise AssertionError("%s: %d outside, worst at z = %g: got %r, want %r, %.3g of the bound" % (
            what, bad.sum(), z[i], got[i], ref[i], abs(got[i] - ref[i]) / budget[i]))


def _truth(act, z=Z):
    """z, act(z), act'(z) and the magnitudes of the terms of act', in 64 bits without a difference of near
    values."""
    z = z.astype(np.float64)
    s, t = expit(z), expit(-z)
    if act == "sigmoid":
        return z, s, s * t, s * t
    if act == "silu":
        return z, z * s, s * (1 + z * t), s * (1 + np.abs(z) * t)
    cdf, bell = 0.5 * erfc(-z / np.sqrt(2)), np.exp(-0.5 * z * z) / np.sqrt(2 * np.pi)
    return z, z * cdf, cdf + z * bell, cdf + np.abs(z) * bell


FAR = np.unique(np.concatenate([np.linspace(-86.0, -12.0, 20001), np.linspace(12.0, 80.0, 20001)]).astype(np.float32))


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("at", [Z, FAR], ids=["near", "far"])
def test_sigmoid_gates_keep_their_relative_accuracy(cuda_device, lib, at, act):
    """sigmoid' = s (1 - s) and 1 - s are small where s is near one: formed as e^-z s they keep all bits."""
    z, a, da, mag = _truth(act, at)
    r, dy, dz = _gates(at, act, cuda_device)
    one = (1.5 * np.abs(z) + 8) * U  # s: the exponent, 2^x, 1 + e, 1/x, and z s
    _near(r, a, one * np.abs(a), "forward", at)
    _near(dy, a, one * np.abs(a), "backward's act(z)", at)
    # s, e and s again, and four operations
    _near(dz, da, (3 * one + 4 * U) * mag, "derivative", at)


def test_gelu_keeps_its_relative_accuracy(cuda_device, lib):
    """Phi(z) falls to 1e-36 on the left: its bound is relative all the way."""
    z, a, da, mag = _truth("gelu")
    r, dy, dz = _gates(Z, "gelu", cuda_device)
    # the exponential; the fit and its steps, which lose up to 1.25 |z| where their terms cancel; z Phi
    phi = (1.25 * z * z + 4 + 4 * np.abs(z) + 12) * U
    _near(r, a, phi * np.abs(a), "forward")
    _near(dy, a, phi * np.abs(a), "backward's act(z)")
    _near(dz, da, (phi + 4 * U) * mag, "derivative")


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M", [1, 20])
def test_gated_feed_forward_in_the_tails(cuda_device, lib, act, M):
    """g = z and u = 1 exactly: h is act(z) with one rounding to bf16, for few tokens and in tiles."""
    z = torch.linspace(-12, 12, 4096, device=cuda_device).to(torch.bfloat16)
    x = torch.zeros(M, 8, device=cuda_device, dtype=torch.bfloat16)
    x[:, 0] = 1
    wg, wu = (torch.zeros(4096, 8, device=cuda_device, dtype=torch.bfloat16) for _ in range(2))
    wg[:, 0], wu[:, 0] = z, 1
    h = R.rapt_glu_fwd(x, wg, wu, act=act).double()
    d = z.double()
    ref = d * torch.sigmoid(d) if act == "silu" else d * 0.5 * torch.erfc(-d / 2 ** 0.5)
    assert bool(((h - ref).abs() <= (2.0 ** -8 + 300 * U) * ref.abs()).all())


@pytest.mark.parametrize("act,top", [("sigmoid", [0, 1, 0, 1]), ("silu", [0, 1e30, 0, 3e38]), ("gelu", [0, 1e30, 0, 3e38]),
                                     ("relu", [0, 1e30, 0, 3e38])])
def test_gates_at_the_ends_of_their_range(cuda_device, lib, act, top):
    """Far out a gate is closed or open, its derivative 0 or 1 (sigmoid: 0); a NaN stays one."""
    z = torch.tensor([-1e30, 1e30, -3e38, 3e38, float("nan"), 0.0, 0.0, 0.0], device=cuda_device).view(1, 8)
    one, zero = torch.ones_like(z), torch.zeros_like(z)
    r, _ = R.rapt_residual_norm_fwd(zero, one, gate=z, act=act)
    _, dy, dz = R.rapt_residual_norm_bwd(one, None, zero, one, gate=z, act=act)[:3]
    want = torch.tensor(top, device=cuda_device, dtype=torch.float32)
    assert torch.equal(r[0, :4], want) and torch.equal(dy[0, :4], want)
    assert torch.isnan(r[0, 4]) and torch.isnan(dy[0, 4]) and (act == "relu" or torch.isnan(dz[0, 4]))
    assert dz[0, :4].tolist() == ([0, 0, 0, 0] if act == "sigmoid" else [0, 1, 0, 1])
    inf = torch.full_like(z, float("inf"))
    assert torch.isinf(R.rapt_residual_norm_fwd(zero, one, gate=inf, act=act)[0]).all() or act == "sigmoid"
