"""Pins of the fp64 oracle of the operators around the attention (oracle/block.py): closed forms,
invariances, and every gradient against central differences of the forward."""

import numpy as np
import pytest

from oracle import block as OB


def _rng(seed):
    return np.random.default_rng(seed)


def _directional(f, args, grads, seed, step=1e-6):
    """(sum of grad . direction, central difference of f) over a random direction in each argument."""
    g = _rng(seed)
    out = []
    for i, gr in enumerate(grads):
        if gr is None:
            continue
        d = g.standard_normal(np.shape(args[i]))
        hi, lo = list(args), list(args)
        hi[i], lo[i] = args[i] + step * d, args[i] - step * d
        out.append((float((gr * d).sum()), (f(*hi) - f(*lo)) / (2 * step)))
    return out


@pytest.mark.parametrize("name", OB.ACTS)
def test_activation_derivative_is_the_difference_quotient(name):
    z = _rng(1).standard_normal(200) * 3
    z = z[np.abs(z) > 1e-3]
    a, da = OB.act(name, z)
    num = (OB.act(name, z + 1e-6)[0] - OB.act(name, z - 1e-6)[0]) / 2e-6
    assert np.abs(da - num).max() <= 1e-8
    if name == "silu":
        assert np.allclose(a, z * OB.act("sigmoid", z)[0], rtol=1e-15)
    if name == "gelu":
        assert np.allclose(a - OB.act(name, -z)[0], z, rtol=1e-12)  # z Phi(z) + z Phi(-z) = z


def test_norms_have_unit_mean_square_and_ignore_scale():
    g = _rng(2)
    x, y, w = g.standard_normal((3, 7, 40))
    one = np.ones(40)
    r, h = OB.residual_norm(x, y, None, one, None, one, eps=1e-30)
    assert np.allclose((h * h).mean(-1), 1.0)
    assert np.allclose(r, x + y / np.sqrt((y * y).mean(-1, keepdims=True)))
    r2, h2 = OB.residual_norm(3 * x, 3 * y, None, None, None, one, eps=1e-30)
    assert np.allclose(h2, OB.residual_norm(x, y, None, None, None, one, eps=1e-30)[1])
    assert OB.residual_norm(x)[0] is x
    assert np.array_equal(OB.residual_norm(x, y, w, act_name="none")[0], x + w * y)


@pytest.mark.parametrize("name", OB.ACTS)
@pytest.mark.parametrize("parts", ["all", "no_post", "no_gate", "no_scale", "pre_only", "r_only", "h_only"])
def test_residual_norm_gradients_are_differences(name, parts):
    g = _rng(3)
    T, D = 5, 24
    x, y, z, dr, dh = g.standard_normal((5, T, D))
    wpost, sc, wpre = g.uniform(0.5, 1.5, (3, D))
    if parts == "no_post":
        wpost = None
    if parts == "no_gate":
        z = None
    if parts == "no_scale":
        sc = None
    if parts == "pre_only":
        y = z = wpost = sc = None
    if parts == "r_only":
        dh = None
    if parts == "h_only":
        dr = None
    got = OB.residual_norm_bwd(dr, dh, x, y, z, wpost, sc, wpre, name)

    def f(x, y, z, wpost, sc, wpre):
        r, h = OB.residual_norm(x, y, z, wpost, sc, wpre, name)
        return (0 if dr is None else (dr * r).sum()) + (0 if dh is None else (dh * h).sum())

    grads = [got.get(k) for k in ("dx", "dy", "dgate", "dw_post", "dscale", "dw_pre")]
    for a, b in _directional(f, [x, y, z, wpost, sc, wpre], grads, 4):
        assert abs(a - b) <= 1e-7 * (1 + abs(b))


@pytest.mark.parametrize("name", OB.ACTS)
def test_glu_and_linear_gradients_are_differences(name):
    g = _rng(5)
    x, wg, wu, dh = (g.standard_normal(s) for s in ((6, 10), (8, 10), (8, 10), (6, 8)))
    got = OB.glu_bwd(dh, x, wg, wu, name)
    for a, b in _directional(lambda *p: (dh * OB.glu(*p, name)).sum(), [x, wg, wu], got, 6):
        assert abs(a - b) <= 1e-7 * (1 + abs(b))
    got = OB.linear_bwd(dh, x, wg)
    for a, b in _directional(lambda x, w: (dh * (x @ w.T)).sum(), [x, wg], got, 7):
        assert abs(a - b) <= 1e-7 * (1 + abs(b))


def test_glu_closed_forms():
    g = _rng(8)
    x, wg, wu = (g.standard_normal(s) for s in ((4, 6), (5, 6), (5, 6)))
    assert np.allclose(OB.glu(x, wg, wu, "none"), (x @ wg.T) * (x @ wu.T))
    assert np.allclose(OB.glu(x, 0 * wg, wu, "sigmoid"), 0.5 * (x @ wu.T))
    assert not OB.glu(x, -np.abs(wg), np.abs(wu), "relu")[np.all(x > 0, axis=1)].any()
