"""Error budgets for the operators around the attention: how far a computed value may be from the
fp64 oracle's, element by element, from the arithmetic alone.

U32 = 2^-24 is half a step of fp32, HALF[dtype] half a step of the output's type (bf16 2^-8, fp32
2^-24). A stored value is off by HALF |value| plus the error of the fp32 value before its rounding,
which the functions below bound by counting roundings: C of them on every term of a sum of few terms
(C = 128 covers the ~20 operations of a term, the partial sums of a row's mean square, the hardware
exponential at |z| <= 10 and the division), and one per addition in a long sum.
"""

import numpy as np

from oracle import block as OB

U32 = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
C = 128 * U32


def within(got, ref, budget, what=""):
    """Asserts |got - ref| <= budget for every element (a NaN fails)."""
    bad = ~(np.abs(got - ref) <= budget)
    if bad.any():
        at = np.unravel_index(np.argmax(np.where(bad, np.abs(got - ref) / budget, 0)), got.shape)
        raise AssertionError("%s: %d of %d outside, worst at %s: got %r, want %r, budget %.3g" % (
            what, bad.sum(), bad.size, at, got[at], ref[at], budget[at]))


def residual_norm(dtype, x, y, gate, w_post, scale, w_pre, act, eps):
    """Oracle (r, h) and their budgets. The error of r before rounding is C (|x| + |s a n|); h = w r rho
    carries it times |w| rho, and C |h|."""
    r, h = OB.residual_norm(x, y, gate, w_post, scale, w_pre, act, eps)
    er = C * (np.abs(x) + (np.abs(r - x) if y is not None else 0))
    br = HALF[dtype] * np.abs(r) + er
    if h is None:
        return r, None, br, None
    bh = (HALF[dtype] + C) * np.abs(h) + np.abs(w_pre) * OB.rms(r, eps) * er
    return r, h, br, bh


def residual_norm_bwd(dtype, dr, dh, x, y, gate, w_post, scale, w_pre, act, eps):
    """Oracle gradients and budgets: every formula of the backward with absolute values in place of
    values bounds the sum of the magnitudes of its terms."""
    ref = OB.residual_norm_bwd(dr, dh, x, y, gate, w_post, scale, w_pre, act, eps)
    T = (dr if dr is not None else dh).shape[0]
    ab = np.abs
    s = 1.0 if scale is None else ab(scale)
    a = da = 1.0
    if gate is not None:
        a, da = OB.act(act, gate)
        # a' is itself a sum of terms: its magnitude is not less than the terms' own
        a, da = ab(a), ab(da) + ab(a) + 0.5
    n = sg = None
    g = np.zeros_like(dr if dr is not None else dh) if dr is None else ab(dr)
    rh = None
    if y is not None:
        sg = OB.rms(y, eps)
        n = ab(y) if w_post is None else ab(w_post * y) * sg
    if dh is not None:
        r = OB.residual_norm(x, y, gate, w_post, scale, None, act, eps)[0]
        rho = OB.rms(r, eps)
        rh = ab(x) * rho + (0 if y is None else s * a * n * rho)  # terms of r, before they cancel
        t = ab(w_pre * dh)
        g = g + rho * (t + rh * (t * rh).mean(-1, keepdims=True) + rh * rh.mean(-1, keepdims=True) * t)
    mag = {"dx": g}
    long = 1.0 + T / 128.0  # a column sum adds T rounded terms one after another
    if dh is not None:
        mag["dw_pre"] = long * (ab(dh) * rh).sum(0)
    if y is not None:
        dn = s * a * g
        mag["dgate"], mag["dscale"] = s * n * da * g, long * (a * n * g).sum(0)
        mag["dy"] = dn
        if w_post is not None:
            yh, u = ab(y) * sg, ab(w_post) * dn
            mag["dw_post"] = long * (dn * yh).sum(0)
            mag["dy"] = sg * (u + yh * (u * yh).mean(-1, keepdims=True))
    half = lambda k: U32 if k in ("dw_post", "dscale", "dw_pre") else HALF[dtype]
    return ref, {k: half(k) * ab(v) + 2 * C * mag[k] for k, v in ref.items()}


def _sum_err(k):
    """Relative to the sum of its terms' magnitudes: a sum of k exact products added in fp32 blocks."""
    return (k + 8) * U32 * 2  # the tensor core truncates where fp32 addition rounds: a whole step


def linear_bwd(dy, x, w):
    """Oracle (dx, dw) and budgets."""
    dx, dw = OB.linear_bwd(dy, x, w)
    ab = np.abs
    bx = HALF["bf16"] * ab(dx) + _sum_err(w.shape[0]) * (ab(dy) @ ab(w))
    bw = HALF["bf16"] * ab(dw) + _sum_err(x.shape[0]) * (ab(dy).T @ ab(x))
    return dx, dw, bx, bw


def _gate_errors(x, w_gate, w_up, act):
    """act(g), act'(g), u and the errors of their fp32 values. Every activation here has |act'| <= 1.13
    and |act''| <= 1.13, except relu's derivative, which may be decided either way within g's error."""
    e = _sum_err(x.shape[1])
    g, u = x @ w_gate.T, x @ w_up.T
    eg, eu = e * (np.abs(x) @ np.abs(w_gate).T), e * (np.abs(x) @ np.abs(w_up).T)
    a, da = OB.act(act, g)
    ea = 1.13 * eg + C * (np.abs(a) + np.abs(g) * 2.0 ** -10)
    eda = (1.13 * eg + C * 1.5) if act != "relu" else (np.abs(g) <= eg).astype(np.float64)
    if act == "none":
        eda = np.zeros_like(g)
    return g, u, a, da, eu, ea, eda


def glu(x, w_gate, w_up, act):
    """Oracle h and its budget."""
    _, u, a, _, eu, ea, _ = _gate_errors(x, w_gate, w_up, act)
    h = a * u
    return h, (HALF["bf16"] + C) * np.abs(h) + (np.abs(u) + eu) * ea + np.abs(a) * eu


def glu_bwd(dh, x, w_gate, w_up, act):
    """Oracle (dx, dw_gate, dw_up) and budgets: dg and du are rounded to bf16 before the products that
    sum them, so each is off by half a bf16 step and its fp32 error, and so is every term."""
    _, u, a, da, eu, ea, eda = _gate_errors(x, w_gate, w_up, act)
    ab = np.abs
    dg, du = dh * u * da, dh * a
    edg = (HALF["bf16"] + C) * ab(dg) + ab(dh) * (ab(u) * eda + (ab(da) + eda) * eu)
    edu = (HALF["bf16"] + C) * ab(du) + ab(dh) * ea
    dx, dwg, dwu = OB.glu_bwd(dh, x, w_gate, w_up, act)
    kx, kw = _sum_err(2 * w_gate.shape[0]), _sum_err(x.shape[0])
    bx = HALF["bf16"] * ab(dx) + edg @ ab(w_gate) + edu @ ab(w_up) + kx * (ab(dg) @ ab(w_gate) + ab(du) @ ab(w_up))
    bg = HALF["bf16"] * ab(dwg) + edg.T @ ab(x) + kw * (ab(dg).T @ ab(x))
    bu = HALF["bf16"] * ab(dwu) + edu.T @ ab(x) + kw * (ab(du).T @ ab(x))
    return (dx, dwg, dwu), (bx, bg, bu)
