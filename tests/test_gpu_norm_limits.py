"""Residual norm backward of rows whose mean of r^2 leaves fp32's range: h is zero there, and the gradients are
those of r alone. Without dh no gradient depends on r at all.

The row sums with r in them (sum t.r, sum e.r; e the joined term, t = w_pre dh) overflow as well then.
"""

import numpy as np
import pytest
import torch

import block_bounds as BB
from gpu_helpers import to_host
from relu_linear_attention_gb300 import binding as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
NAMES = ("x", "y", "gate", "w_post", "scale", "w_pre")
# 8 lanes a row, a warp a row, a CTA a row; with a ring and without; whole vectors and not
SIZES = [(70, 24), (37, 192), (9, 520), (5, 1001), (5, 5120), (3, 8195), (3, 16384)]


def _inputs(T, D, dtype, device, gate=1.0):
    g = torch.Generator().manual_seed(T + D)
    n = lambda s=1.0: (torch.randn((T, D), generator=g) * s).to(DT[dtype]).to(device)
    u = lambda lo, hi: (torch.rand((D,), generator=g) * (hi - lo) + lo).to(device)
    return (dict(x=n(), y=n(), gate=n(gate), w_post=u(0.5, 1.5), scale=u(0.5, 1.0), w_pre=u(0.5, 1.5)), n(), n())


def _against_the_oracle(kw, dr, dh, act, dtype, skip=()):
    got = R.rapt_residual_norm_bwd(dr, dh, **kw, act=act, eps=EPS)
    h = {k: None if v is None else to_host(v) for k, v in {**kw, "dr": dr, "dh": dh}.items()}
    with np.errstate(over="ignore"):  # e^-z of a closed gate
        ref, bud = BB.residual_norm_bwd(dtype, *[h.get(k) for k in ("dr", "dh") + NAMES], act, EPS)
    for name, t in zip(("dx", "dy", "dgate", "dw_post", "dscale", "dw_pre"), got):
        if t is not None and name not in skip:
            BB.within(to_host(t), ref[name], bud[name], name)
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("T,D", SIZES)
def test_a_joined_term_of_1e25_without_dh(cuda_device, lib, T, D, act, dtype):
    """e . r would overflow; nothing depends on it."""
    kw, dr, _ = _inputs(T, D, dtype, cuda_device, gate=1e25)
    got = _against_the_oracle(kw, dr, None, act, dtype)
    assert torch.equal(got[0], dr)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D", SIZES)
def test_a_residual_of_1e25(cuda_device, lib, T, D, dtype):
    """The mean of r^2 overflows: h and the gradients through it are zero, those of r stay."""
    kw, dr, dh = _inputs(T, D, dtype, cuda_device, gate=1e25)
    _against_the_oracle(kw, dr, dh, "none", dtype, skip=("dw_pre",))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D", SIZES)
def test_rows_beside_one_that_overflows_keep_their_bits(cuda_device, lib, T, D, dtype):
    """The rows of a warp (D <= 256) are summed together; every third one overflows."""
    kw, dr, dh = _inputs(T, D, dtype, cuda_device)
    want = R.rapt_residual_norm_bwd(dr, dh, **kw, act="silu", eps=EPS)[:3]
    bad = torch.arange(0, T, 3, device=cuda_device)
    ill = {k: v.clone() for k, v in kw.items()}
    ill["gate"][bad] = 1e25
    ill["x"][bad[1:]] = 1e30
    dhi = dh.clone()
    dhi[bad] = 1e30
    got = R.rapt_residual_norm_bwd(dr, dhi, **ill, act="silu", eps=EPS)[:3]
    rest = torch.ones(T, dtype=torch.bool, device=cuda_device)
    rest[bad] = False
    for a, b in zip(want, got):
        assert torch.equal(a[rest], b[rest]) and torch.isfinite(b[bad].float()).all()
