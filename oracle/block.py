"""The operators around the attention in fp64: residual norms, gated feed-forward, projection gradients.

Plain restatements of the formulas that include/rapt.h gives for rapt_residual_norm_*, rapt_glu_* and
rapt_linear_bwd; numpy's matmul and scipy's erf are the only building blocks.
"""

import numpy as np
from scipy.special import erf

ACTS = ("none", "silu", "gelu", "relu", "sigmoid")


def act(name, z):
    """act(z) and act'(z)."""
    z = np.asarray(z, dtype=np.float64)
    if name == "none":
        return z, np.ones_like(z)
    if name == "relu":
        return np.where(z > 0, z, 0.0), (z > 0).astype(np.float64)
    if name == "gelu":
        cdf = 0.5 * (1.0 + erf(z / np.sqrt(2.0)))
        return z * cdf, cdf + z * np.exp(-0.5 * z * z) / np.sqrt(2.0 * np.pi)
    s = 1.0 / (1.0 + np.exp(-z))
    if name == "sigmoid":
        return s, s * (1.0 - s)
    if name == "silu":
        return z * s, s * (1.0 + z * (1.0 - s))
    raise ValueError(name)


def rms(x, eps):
    """(mean(x^2) + eps)^(-1/2) of every row."""
    return 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def residual_norm(x, y=None, gate=None, w_post=None, scale=None, w_pre=None, act_name="sigmoid", eps=1e-6):
    """(r, h) of rapt_residual_norm_fwd; h is None without w_pre."""
    r = x
    if y is not None:
        n = y if w_post is None else w_post * y * rms(y, eps)
        a = 1.0 if gate is None else act(act_name, gate)[0]
        r = x + (1.0 if scale is None else scale) * a * n
    return r, None if w_pre is None else w_pre * r * rms(r, eps)


def residual_norm_bwd(dr, dh, x, y=None, gate=None, w_post=None, scale=None, w_pre=None, act_name="sigmoid",
                      eps=1e-6):
    """Gradients of sum(dr r) + sum(dh h): a dict of dx, dy, dgate, dw_post, dscale, dw_pre."""
    out = {}
    s = 1.0 if scale is None else scale
    a, da, n, sg = 1.0, 0.0, None, None
    if y is not None:
        if gate is not None:
            a, da = act(act_name, gate)
        sg = rms(y, eps)
        n = y if w_post is None else w_post * y * sg
    g = 0.0 if dr is None else dr
    if dh is not None:
        r = residual_norm(x, y, gate, w_post, scale, None, act_name, eps)[0]
        rho = rms(r, eps)
        t, rh = w_pre * dh, r * rho
        g = g + rho * (t - rh * (t * rh).mean(-1, keepdims=True))
        out["dw_pre"] = (dh * rh).sum(0)
    out["dx"] = g
    if y is not None:
        dn = s * a * g
        if gate is not None:
            out["dgate"] = s * n * da * g
        if scale is not None:
            out["dscale"] = (a * n * g).sum(0)
        if w_post is None:
            out["dy"] = dn
        else:
            yh = y * sg
            u = w_post * dn
            out["dw_post"] = (dn * yh).sum(0)
            out["dy"] = sg * (u - yh * (u * yh).mean(-1, keepdims=True))
    return out


def glu(x, w_gate, w_up, act_name="silu"):
    """h = act(x w_gate^T) (x w_up^T)."""
    return act(act_name, x @ w_gate.T)[0] * (x @ w_up.T)


def glu_bwd(dh, x, w_gate, w_up, act_name="silu"):
    """(dx, dw_gate, dw_up) of sum(dh h)."""
    a, da = act(act_name, x @ w_gate.T)
    dg, du = dh * (x @ w_up.T) * da, dh * a
    return dg @ w_gate + du @ w_up, dg.T @ x, du.T @ x


def linear_bwd(dy, x, w):
    """(dx, dw) of sum(dy y) for y = x w^T."""
    return dy @ w, dy.T @ x
