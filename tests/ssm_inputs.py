"""Seeded inputs of the selective state space block on the GPU, as column slices of wider rows, and the same in
fp64 for the oracle."""

import numpy as np
import torch

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def host(t):
    return None if t is None else t.detach().double().cpu().numpy()


def scan_inputs(seed, rows, H, P, G, N, dtype, z=True, D=True, bias=True, sliced=True, decay=(1.0, 16.0)):
    """x, dt, A, B, C and the options of a scan over rows (a tuple) of tokens."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda").to(DT[dtype])
    u = lambda k, lo, hi: torch.rand((k,), generator=g, device="cuda") * (hi - lo) + lo
    rows = tuple(rows)
    if sliced:
        pad = 16
        xbc = n(*rows, H * P + 2 * G * N + pad)
        zdt = n(*rows, (H * P + H + pad + 15) // 16 * 16)
        x, b, c = (v.unflatten(-1, s) for v, s in zip(xbc[..., pad:].split((H * P, G * N, G * N), -1),
                                                      ((H, P), (G, N), (G, N))))
        zz, dt = zdt[..., :H * P].unflatten(-1, (H, P)), zdt[..., H * P:H * P + H]
    else:
        x, b, c, zz, dt = n(*rows, H, P), n(*rows, G, N), n(*rows, G, N), n(*rows, H, P), n(*rows, H)
    args = dict(x=x, dt=dt, A=-u(H, *decay), B=b, C=c)
    opts = dict(D=u(H, 0.5, 1.5) if D else None, z=zz if z else None, dt_bias=u(H, -6.0, -2.0) if bias else None)
    return args, opts


def document(args, opts, at):
    """fp64 inputs of the tokens `at` (an index of the leading dimensions)."""
    per_head = ("A", "D", "dt_bias")
    return {k: host(v) if v is None or k in per_head else host(v[at]) for k, v in {**args, **opts}.items()}


def state(seed, n, H, N, P):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((n, H, N, P), generator=g, device="cuda")
