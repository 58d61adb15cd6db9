"""The products of the gated feed-forward's and the projections' gradients, every element and exactly.

Operands are small whole numbers, so that every product and every partial sum is a whole number below 2^24
in any order: fp32 sums are exact, and a result differs from the plain product's, rounded once, only where a
slice of a sum was lost, taken twice or added elsewhere. Shapes take every way of dealing the tiles out to
the 76 pairs: whole tiles alone; all tiles cut; whole rounds and then cut tiles; cuts at the same places of
every tile or shares that run from one tile into the next; for dx and dw together.

A bound on single elements that grows with the sum cannot see one lost slice of a long sum, so random
operands at layer size are held in the 2-norm as well.
"""

import numpy as np
import pytest
import torch

from gpu_helpers import to_host
from oracle import block as OB
from relu_linear_attention_gb300 import binding as R

pytestmark = pytest.mark.gpu


def _whole(shape, most, seed, device, zero=True):
    """Whole numbers in [-most, most]."""
    g = torch.Generator(device=device).manual_seed(seed)
    t = torch.randint(-most, most + 1, shape, generator=g, device=device)
    if not zero:
        t = torch.where(t == 0, 1, t)
    return t.to(torch.bfloat16)


def _rounded(t):
    assert float(t.abs().max()) < 2 ** 24
    return t.to(torch.float32).to(torch.bfloat16)


def _same(got, want, name):
    bad = got != want
    if bad.any():
        at = [int(i) for i in bad.nonzero()[0]]
        raise AssertionError("%s: %d of %d differ, first at %s: got %g, want %g" % (
            name, int(bad.sum()), bad.numel(), at, float(got[tuple(at)]), float(want[tuple(at)])))


# (M, N, K): how dx's tiles are dealt out, how dw's
LINEAR = [(5, 80, 1384),         # whole, whole
          (43, 6896, 8),         # cut alike, whole
          (3682, 5400, 8),       # both cut alike, shares that end behind their tile in dw
          (9999, 10296, 8),      # both cut, shares across tiles
          (1518, 1712, 2736),    # whole, whole rounds and cut alike
          (3271, 4944, 296),     # shares across tiles, whole
          (2586, 1496, 1736),    # whole rounds and cut alike, whole
          (1669, 1672, 2704),    # whole rounds and cut alike, both
          (6130, 9912, 552),     # whole, whole rounds and shares across tiles
          (14813, 7792, 280),    # whole rounds and shares across tiles, whole
          (5674, 5736, 1192),    # whole rounds and shares across tiles, both
          (65521, 512, 520), (2048, 6144, 2048), (1, 2048, 2048), (257, 264, 776)]


@pytest.mark.parametrize("M,N,K", LINEAR)
def test_linear_gradients_are_exact_sums(cuda_device, lib, M, N, K):
    dy, x, w = (_whole(s, 2, 7 * i + M, cuda_device) for i, s in enumerate(((M, N), (M, K), (N, K))))
    dx, dw = R.rapt_linear_bwd(dy, x, w)
    _same(dx, _rounded(dy.double() @ w.double()), "dx")
    _same(dw, _rounded(dy.double().t() @ x.double()), "dw")


# (M, F, K), as above with two terms in dx and two products in dw
GLU = [(1, 8, 8), (7, 2744, 1032), (16, 1024, 264),  # the kernel of few tokens forward
       (20, 80, 136), (226, 264, 776),
       (139, 3088, 8),           # cut alike, whole
       (5169, 2312, 8),          # both cut alike
       (12947, 5144, 8),         # both cut, shares across tiles
       (817, 888, 2512),         # whole rounds and cut alike, whole
       (1837, 864, 2472),        # whole rounds and cut alike, both
       (6330, 7400, 288),        # shares across tiles, whole rounds and shares across tiles
       (7208, 3672, 784),        # whole rounds and shares across tiles, both
       (1531, 2744, 1032)]


@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("M,F,K", GLU)
def test_glu_and_its_gradients_are_exact_sums(cuda_device, lib, M, F, K, act):
    x, wg, wu = (_whole(s, 1, 5 * i + M, cuda_device) for i, s in enumerate(((M, K), (F, K), (F, K))))
    dh = _whole((M, F), 1, 3, cuda_device, zero=False)
    g, u = x.double() @ wg.double().t(), x.double() @ wu.double().t()
    assert float(g.abs().max()) <= 256 and float(u.abs().max()) <= 256  # whole numbers that bf16 has
    a, da = (g, torch.ones_like(g)) if act == "none" else (g.clamp(min=0), (g > 0).double())
    dg, du = dh.double() * u * da, dh.double() * a
    _same(R.rapt_glu_fwd(x, wg, wu, act=act), _rounded(a * u), "h")
    dx, dwg, dwu = R.rapt_glu_bwd(dh, x, wg, wu, act=act)
    _same(dx, _rounded(dg @ wg.double() + du @ wu.double()), "dx")
    _same(dwg, _rounded(dg.t() @ x.double()), "dw_gate")
    _same(dwu, _rounded(du.t() @ x.double()), "dw_up")


def _rel(got, ref):
    return float(np.linalg.norm(to_host(got) - ref) / np.linalg.norm(ref))


# A rounding to bf16 is off by at most 2^-8 of a value of mantissa 1, and uniformly so: 2^-8 / sqrt(3) in the
# mean square at most. Sums of many such terms keep that ratio, so a result is off by one rounding, or, where
# its terms were rounded as well, by sqrt(2) of it; 5 % for the sample and the fp32 sums (a step of 2^-23 in
# each of 16384 / 16 additions would be 1.2e-4). One 64-deep slice of 16384 terms is 6 % of a sum.
ONE = 2.0 ** -8 / 3 ** 0.5 * 1.05


def test_layer_size_gradients_in_the_2_norm(cuda_device, lib):
    M, F, K, N = 16384, 5504, 2048, 6144
    n = lambda *s, scale=1.0: (torch.randn(s, generator=g, device=cuda_device) * scale).to(torch.bfloat16)
    g = torch.Generator(device=cuda_device).manual_seed(5)
    dh, x, wg, wu = n(M, F), n(M, K), n(F, K, scale=K ** -0.5), n(F, K, scale=K ** -0.5)
    h, (dx, dwg, dwu) = R.rapt_glu_fwd(x, wg, wu), R.rapt_glu_bwd(dh, x, wg, wu)
    rows = torch.tensor([0, 127, 128, 8191, 16127, 16128, 16383], device=cuda_device)
    hx, hg, hu, hd = to_host(x[rows]), to_host(wg), to_host(wu), to_host(dh[rows])
    assert _rel(h[rows], OB.glu(hx, hg, hu)) <= ONE
    assert _rel(dx[rows], OB.glu_bwd(hd, hx, hg, hu)[0]) <= 2 ** 0.5 * ONE
    cols = torch.tensor([0, 255, 256, 2751, 5375, 5376, 5503], device=cuda_device)
    ref = OB.glu_bwd(to_host(dh[:, cols]), to_host(x), to_host(wg[cols]), to_host(wu[cols]))
    assert _rel(dwg[cols], ref[1]) <= 2 ** 0.5 * ONE and _rel(dwu[cols], ref[2]) <= 2 ** 0.5 * ONE
    dy, w = n(M, N), n(N, K)
    dx, dw = R.rapt_linear_bwd(dy, x, w)
    assert _rel(dx[rows], to_host(dy[rows]) @ to_host(w)) <= ONE
    a, b = to_host(dy[:, cols]), to_host(x)
    assert _rel(dw[cols], a.T @ b) <= ONE
    # a slice of 64 tokens left out of the reference is seen
    assert _rel(dw[cols], a[64:].T @ b[64:]) > 10 * ONE
