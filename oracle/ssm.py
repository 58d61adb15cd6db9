"""The selective state space block in fp64: causal convolution, selective scan, layer norm.

Plain restatements of the formulas that include/rapt.h gives for rapt_conv_*, rapt_ssm_* and
rapt_layer_norm_*; numpy alone. The scan comes as its recurrence and as the quadratic sum over earlier
tokens that the recurrence stands for.
"""

import numpy as np

from .block import act


def conv(x, w, bias=None, act_name="silu", state=None):
    """One document x [n, D], w [D, W]: (y [n, D], the last W - 1 inputs)."""
    W = w.shape[1]
    head = np.zeros((W - 1, x.shape[1])) if state is None else state
    long = np.concatenate([head, x])
    z = sum(long[k:k + x.shape[0]] * w[:, k] for k in range(W)) + (0.0 if bias is None else bias)
    return act(act_name, z)[0], long[x.shape[0]:]


def softplus(v):
    return np.maximum(v, 0.0) + np.log1p(np.exp(-np.abs(v)))


def steps(dt, dt_bias=None, dt_softplus=True):
    v = dt + (0.0 if dt_bias is None else dt_bias)
    return softplus(v) if dt_softplus else v


def silu(z):
    return act("silu", z)[0]


def _finish(y, x, D, z):
    y = y if D is None else y + D[:, None] * x
    return y if z is None else y * silu(z)


def scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=True, S0=None):
    """One document, by its recurrence: x [n, H, P], dt [n, H], B and C [n, G, Ns]. Returns (out, S [H, Ns, P])."""
    n, H, P = x.shape
    R = H // B.shape[1]
    d = steps(dt, dt_bias, dt_softplus)
    S = np.zeros((H, B.shape[2], P)) if S0 is None else S0.copy()
    y = np.zeros_like(x)
    for t in range(n):
        b, c = np.repeat(B[t], R, 0), np.repeat(C[t], R, 0)
        S = np.exp(d[t] * A)[:, None, None] * S + (d[t][:, None] * b)[:, :, None] * x[t][:, None, :]
        y[t] = np.einsum("hn,hnp->hp", c, S)
    return _finish(y, x, D, z), S


def scan_quadratic(x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=True, S0=None):
    """The same as a sum over earlier tokens: y_t = sum_{i<=t} e^(A sum_{i<j<=t} dt_j) dt_i (C_t . B_i) x_i + ..."""
    n, H, P = x.shape
    R = H // B.shape[1]
    d = steps(dt, dt_bias, dt_softplus)
    b, c = np.repeat(B, R, 1), np.repeat(C, R, 1)
    cum = np.cumsum(d * A, 0)
    y = np.zeros_like(x)
    for t in range(n):
        w = np.exp(cum[t] - cum[:t + 1]) * d[:t + 1]
        y[t] = np.einsum("ih,hn,ihn,ihp->hp", w, c[t], b[:t + 1], x[:t + 1])
        if S0 is not None:
            y[t] += np.exp(cum[t])[:, None] * np.einsum("hn,hnp->hp", c[t], S0)
    S = np.zeros((H, B.shape[2], P)) if S0 is None else S0.copy()
    if n:
        S = np.exp(cum[-1])[:, None, None] * S + np.einsum(
            "ih,ihn,ihp->hnp", np.exp(cum[-1] - cum) * d, b, x)
    return _finish(y, x, D, z), S


def layer_norm(x, w=None, b=None, eps=1e-5):
    xc = x - x.mean(-1, keepdims=True)
    y = xc / np.sqrt((xc * xc).mean(-1, keepdims=True) + eps)
    return (y if w is None else y * w) + (0.0 if b is None else b)


def layer_norm_bwd(dy, x, w=None, eps=1e-5):
    """(dx, dw, db) of sum(dy y)."""
    xc = x - x.mean(-1, keepdims=True)
    r = 1.0 / np.sqrt((xc * xc).mean(-1, keepdims=True) + eps)
    xh = xc * r
    g = dy if w is None else dy * w
    dx = r * (g - g.mean(-1, keepdims=True) - xh * (g * xh).mean(-1, keepdims=True))
    return dx, (dy * xh).reshape(-1, x.shape[-1]).sum(0), dy.reshape(-1, x.shape[-1]).sum(0)
