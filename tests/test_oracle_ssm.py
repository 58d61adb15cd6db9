"""The fp64 oracle of the selective state space block against what mathematics fixes: the recurrence is the
quadratic sum, a split document is the whole one, no decay is a plain sum, gradients are differences."""

import numpy as np
import pytest

from oracle import ssm as OS


def _inputs(seed, n=23, H=4, P=3, G=2, N=5):
    g = np.random.default_rng(seed)
    r = g.standard_normal
    return dict(x=r((n, H, P)), dt=r((n, H)), A=-g.uniform(0.5, 8, H), B=r((n, G, N)), C=r((n, G, N)), D=r(H),
                z=r((n, H, P)), dt_bias=r(H), S0=r((H, N, P)))


@pytest.mark.parametrize("softplus", [True, False])
def test_recurrence_is_the_quadratic_sum(softplus):
    k = _inputs(1)
    if not softplus:
        k["dt"] = np.abs(k["dt"]) + np.abs(k["dt_bias"])
    for a, b in zip(OS.scan(**k, dt_softplus=softplus), OS.scan_quadratic(**k, dt_softplus=softplus)):
        np.testing.assert_allclose(a, b, rtol=1e-12, atol=1e-12)


def test_a_split_document_is_the_whole_one():
    k = _inputs(2)
    whole, S = OS.scan(**k)
    a = {n: v[:9] if n in ("x", "dt", "B", "C", "z") else v for n, v in k.items()}
    b = {n: v[9:] if n in ("x", "dt", "B", "C", "z") else v for n, v in k.items()}
    first, mid = OS.scan(**a)
    b["S0"] = mid
    second, end = OS.scan(**b)
    np.testing.assert_allclose(np.concatenate([first, second]), whole, rtol=1e-13, atol=1e-13)
    np.testing.assert_allclose(end, S, rtol=1e-13, atol=1e-13)


def test_without_decay_it_is_a_sum():
    k = _inputs(3, H=2, G=2)
    k.update(A=np.zeros(2), D=None, z=None, S0=None)
    d = OS.steps(k["dt"], k["dt_bias"])
    S = OS.scan(**k)[1]
    np.testing.assert_allclose(S, np.einsum("th,thn,thp->hnp", d, k["B"], k["x"]), rtol=1e-12, atol=1e-12)


def test_softplus_at_both_ends():
    v = np.array([-800.0, -50.0, 0.0, 50.0, 800.0])
    np.testing.assert_allclose(OS.softplus(v), [0.0, np.exp(-50.0), np.log(2.0), 50.0, 800.0], rtol=1e-14)


def test_convolution_by_hand():
    x, w = np.arange(1.0, 6.0)[:, None], np.array([[100.0, 10.0, 1.0]])
    y, last = OS.conv(x, w, np.array([0.5]), "none", np.array([[7.0], [9.0]]))
    np.testing.assert_array_equal(y[:, 0], [791.5, 912.5, 123.5, 234.5, 345.5])
    np.testing.assert_array_equal(last[:, 0], [4.0, 5.0])
    y, last = OS.conv(x[:1], w, None, "none", np.array([[7.0], [9.0]]))
    np.testing.assert_array_equal(last[:, 0], [9.0, 1.0])


def test_layer_norm_rows_and_differences():
    g = np.random.default_rng(4)
    x, w, b, dy = g.standard_normal((5, 7)), g.standard_normal(7), g.standard_normal(7), g.standard_normal((5, 7))
    y = OS.layer_norm(x)
    np.testing.assert_allclose(y.mean(-1), 0, atol=1e-15)
    np.testing.assert_allclose((y * y).mean(-1), 1, rtol=1e-4)
    np.testing.assert_allclose(OS.layer_norm(3.0 * x + 2.0, eps=9e-5), y, rtol=1e-12, atol=1e-12)
    dx, dw, db = OS.layer_norm_bwd(dy, x, w)
    f = lambda x, w, b: (dy * OS.layer_norm(x, w, b)).sum()
    h = 1e-6
    for v, grad, at in ((x, dx, 0), (w, dw, 1), (b, db, 2)):
        for i in np.ndindex(v.shape):
            hi, lo = v.copy(), v.copy()
            hi[i] += h
            lo[i] -= h
            p = [x, w, b]
            p[at] = hi
            up = f(*p)
            p[at] = lo
            assert abs((up - f(*p)) / (2 * h) - grad[i]) < 1e-7
