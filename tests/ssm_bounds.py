"""Error budgets of the selective state space block: how far a computed value may be from the fp64 oracle's,
element by element, from the arithmetic alone. U32 and HALF as in block_bounds.

Recurrence in fp32. A state is a sum of terms w B x (and w S0), w a product of decays and a step size. A decay
exp(dt A) is off by 2 U32 (expf) and by |dt A| times the relative error of its argument: 8 U32 for the softplus
(expf and log1pf of 2 units each, two sums, the bias's), 1 for the product. Over the n steps a term has seen that
is at most (9 |A| sum dt + 2 n) U32, and w e^(-|A| sum dt) with |A| sum dt in it has its largest value where
that sum is 1, so that the first part adds at most 9 U32 of the term's magnitude WITHOUT its decay; the state's
own fused update adds a rounding a step, n U32, and the step size 9, the products 2. So S is off by at most
(4 n + 32) U32 of the sum of its terms' magnitudes, undecayed terms counted for the 9, and y, a sum of N such
products, by N U32 of its terms' magnitudes more. The budgets take (8 n + N + 64) U32 of magnitudes that the oracle
forms with absolute values in place of values; n is the document's length.

Chunks on the tensor cores: the decayed score, the state that C reads and each product's operands are rounded to
bf16 once (half a step, 2^-8, of a term's magnitude); scores and sums are held to the recurrence's budget; two
bf16 parts of the state's update leave 2^-16. The logarithms of decays add up over a chunk: 128 roundings of at
most the chunk's sum, whose effect on a term e^-s is at most s e^-s 128 U32.
"""

import numpy as np

from block_bounds import HALF, U32
from oracle import ssm as OS


def scan(dtype, x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=True, S0=None, chunks=False):
    """Oracle (out, S) of a document and their budgets. chunks: bf16 on the tensor cores."""
    out, S = OS.scan(x, dt, A, B, C, D, z, dt_bias, dt_softplus, S0)
    ab = np.abs
    a0 = None if S0 is None else ab(S0)
    y, mag = OS.scan(ab(x), dt, A, ab(B), ab(C), None, None, dt_bias, dt_softplus, a0)
    n, N = x.shape[0], B.shape[2]
    c = (8 * n + N + 64) * U32
    ey, eS = c * y, c * mag
    if chunks:
        ey = ey + 2.0 ** -8 * y
        eS = eS + 2.0 ** -16 * mag
    # terms as they enter: a decay's argument is off by parts of |A| dt, seen where the decay is near e^-1
    floor = 16 * U32 * (ab(x).max(initial=0) * ab(B).max(initial=0) + (0 if S0 is None else ab(S0).max(initial=0)))
    eS = eS + floor
    ey = ey + floor * ab(C).sum(-1).max(initial=0)
    if D is not None:
        ey = ey + 2 * U32 * ab(D)[:, None] * ab(x)
    if z is not None:
        g = OS.silu(z)
        pre = y if D is None else y + ab(D)[:, None] * ab(x)
        ey = ey * ab(g) + (1.5 * ab(z) + 16) * U32 * ab(g) * pre
    return out, S, HALF[dtype] * ab(out) + ey, eS


def conv(dtype, x, w, bias, act_name, state):
    """Oracle (y, last inputs) of a document and y's budget."""
    y, last = OS.conv(x, w, bias, act_name, state)
    z, _ = OS.conv(x, w, bias, "none", state)
    mag, _ = OS.conv(np.abs(x), np.abs(w), None if bias is None else np.abs(bias), "none",
                     None if state is None else np.abs(state))
    # an activation of slope at most 1.2 passes the sum's error on; its own by rapt_act's bounds
    e = 1.2 * 8 * U32 * mag + (1.25 * z * z + 4 * np.abs(z) + 20) * U32 * np.abs(y)
    return y, last, HALF[dtype] * np.abs(y) + e
