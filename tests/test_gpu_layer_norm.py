"""Layer norm and its gradients on the GPU against the fp64 oracle.

Budgets as in block_bounds: C = 128 U32 covers the ~20 operations of a term, the hardware's root and the row sums'
partial sums. The mean is corrected by the mean of the differences to it, so xh carries C (|xh| + 1) whatever the
row's mean; a column sum adds T rounded terms one after another, at most 1 + T / 128 times C of their magnitudes."""

import numpy as np
import pytest
import torch

from block_bounds import C, HALF, U32, within
from oracle import ssm as OS
from relu_linear_attention_gb300 import binding as R
from ssm_inputs import DT, host

pytestmark = pytest.mark.gpu
EPS = 1e-5


def inputs(seed, T, D, dtype, mean=0.5, scale=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")
    return (n(T, D) * scale + mean).to(DT[dtype]), n(T, D).to(DT[dtype]), n(D) + 1.0, n(D) * 0.2


def check_fwd(y, x, w, b, dtype):
    hx, hw, hb = host(x), 1.0 if w is None else host(w), 0.0 if b is None else host(b)
    ref = OS.layer_norm(hx, hw, hb, EPS)
    xh = OS.layer_norm(hx, eps=EPS)
    within(host(y), ref, HALF[dtype] * np.abs(ref) + C * (np.abs(hw) * (np.abs(xh) + 1) + np.abs(hb)), "y")


def check_bwd(got, dy, x, w, dtype):
    hx, hd, hw = host(x), host(dy), 1.0 if w is None else host(w)
    ref = OS.layer_norm_bwd(hd, hx, hw, EPS)
    xc = hx - hx.mean(-1, keepdims=True)
    r = 1.0 / np.sqrt((xc * xc).mean(-1, keepdims=True) + EPS)
    h, g = np.abs(xc * r) + 1, np.abs(hd * hw)
    long = 1.0 + hx.shape[0] / 128.0
    mags = (r * (g + g.mean(-1, keepdims=True) + h * (g * h).mean(-1, keepdims=True)), long * (np.abs(hd) * h).sum(0),
            long * np.abs(hd).sum(0))
    for name, v, want, mag, half in zip(("dx", "dw", "db"), got, ref, mags, (HALF[dtype], U32, U32)):
        if v is not None:
            within(host(v), want, half * np.abs(want) + 2 * C * mag + 1e-30, name)


WIDTHS = [1, 2, 3, 7, 8, 31, 64, 65, 127, 250, 256, 257, 511, 512, 1000, 1001, 2047, 2048, 4090, 4096, 4097, 5120, 5121, 8185,
          8192, 8193, 12288, 12290, 16383, 16384]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", WIDTHS)
def test_widths(cuda_device, dtype, D):
    for T in (1, 5, 37) if D > 300 else (1, 9, 700):
        x, dy, w, b = inputs(D + T, T, D, dtype)
        check_fwd(R.rapt_layer_norm_fwd(x, w, b, eps=EPS), x, w, b, dtype)
        check_bwd(R.rapt_layer_norm_bwd(dy, x, w, eps=EPS), dy, x, w, dtype)


@pytest.mark.parametrize("dtype,D", [("bf16", 2048), ("bf16", 1001), ("f32", 1536), ("f32", 257), ("f32", 8192),
                                     ("bf16", 64), ("bf16", 16384)])
def test_more_rows_than_the_gpu_holds(cuda_device, dtype, D):
    T = 3001 if D > 300 else 40001
    x, dy, w, b = inputs(1, T, D, dtype)
    check_fwd(R.rapt_layer_norm_fwd(x, w, b, eps=EPS), x, w, b, dtype)
    got = R.rapt_layer_norm_bwd(dy, x, w, eps=EPS)
    check_bwd(got, dy, x, w, dtype)
    assert all(torch.equal(a, c) for a, c in zip(got, R.rapt_layer_norm_bwd(dy, x, w, eps=EPS)))


@pytest.mark.parametrize("dtype,D", [("f32", 1000), ("f32", 65), ("bf16", 2048)])
def test_missing_inputs_and_outputs(cuda_device, dtype, D):
    x, dy, w, b = inputs(2, 50, D, dtype)
    for ww, bb in ((None, None), (w, None), (None, b)):
        check_fwd(R.rapt_layer_norm_fwd(x, ww, bb, eps=EPS), x, ww, bb, dtype)
    check_bwd(R.rapt_layer_norm_bwd(dy, x, None, eps=EPS), dy, x, None, dtype)
    whole = R.rapt_layer_norm_bwd(dy, x, w, eps=EPS)
    for need in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (0, 1, 1), (1, 0, 1)):
        got = R.rapt_layer_norm_bwd(dy, x, w, eps=EPS, need_dx=need[0], need_dw=need[1], need_db=need[2])
        for k in range(3):
            assert (got[k] is None) == (not need[k])
            assert got[k] is None or torch.equal(got[k], whole[k])


@pytest.mark.parametrize("dtype,D", [("f32", 1001), ("bf16", 2048), ("bf16", 77)])
def test_in_place(cuda_device, dtype, D):
    x, dy, w, b = inputs(3, 300, D, dtype)
    y, (dx, dw, db) = R.rapt_layer_norm_fwd(x, w, b), R.rapt_layer_norm_bwd(dy, x, w)
    a, c = dy.clone(), x.clone()
    assert torch.equal(R.rapt_layer_norm_bwd(a, x, w, dx=a)[0], dx)
    got = R.rapt_layer_norm_bwd(dy, c, w, dx=c)
    assert torch.equal(got[0], dx) and torch.equal(got[1], dw) and torch.equal(got[2], db)
    c = x.clone()
    assert R.rapt_layer_norm_fwd(c, w, b, y=c) is c and torch.equal(c, y)


@pytest.mark.parametrize("D", [64, 1001, 2048, 8192])
def test_a_mean_far_from_zero(cuda_device, D):
    """The mean 1e4 times the deviation: the values' own differences decide, and they are exact."""
    x, dy, w, b = inputs(4, 40, D, "f32", mean=2e4)
    check_fwd(R.rapt_layer_norm_fwd(x, w, b, eps=EPS), x, w, b, "f32")
    check_bwd(R.rapt_layer_norm_bwd(dy, x, w, eps=EPS), dy, x, w, "f32")


def test_equal_values_and_single_columns(cuda_device):
    for D in (1, 8, 33, 2048):
        x = torch.full((5, D), 3.0, device="cuda")
        w, b = torch.randn(D, device="cuda"), torch.randn(D, device="cuda")
        assert torch.equal(R.rapt_layer_norm_fwd(x, w, b), b.expand(5, D))
        dx, dw, db = R.rapt_layer_norm_bwd(torch.ones_like(x), x, w)
        assert torch.isfinite(dx).all() and torch.equal(dw, torch.zeros(D, device="cuda"))
        assert torch.equal(db, torch.full((D,), 5.0, device="cuda"))


def test_a_row_depends_on_no_other(cuda_device):
    for D in (40, 1001, 2048):
        x, dy, w, b = inputs(5, 2000, D, "f32")
        y, dx = R.rapt_layer_norm_fwd(x, w, b), R.rapt_layer_norm_bwd(dy, x, w)[0]
        x[700] = float("nan")
        x[701, 5] = float("inf")
        y2, dx2 = R.rapt_layer_norm_fwd(x, w, b), R.rapt_layer_norm_bwd(dy, x, w)[0]
        rest = torch.ones(2000, dtype=torch.bool, device="cuda")
        rest[700:702] = False
        assert torch.equal(y[rest], y2[rest]) and torch.equal(dx[rest], dx2[rest])
        assert torch.isnan(y2[700]).all()


def test_no_rows(cuda_device):
    x = torch.empty(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    assert R.rapt_layer_norm_fwd(x, w).shape == (0, 64)
    dx, dw, db = R.rapt_layer_norm_bwd(x, x, w)
    assert dx.shape == (0, 64) and torch.equal(dw, torch.zeros_like(w)) and torch.equal(db, torch.zeros_like(w))


def test_gradients_are_differences(cuda_device):
    """Central differences of the library's own forward in fp32: steps of 2^-4 in values near 1 leave 2^-16 of
    roundings (2^-20 of y over the step) and a curvature of the step's square, 2^-8, times third derivatives of
    order r^3."""
    T, D = 3, 24
    x, dy, w, b = inputs(6, T, D, "f32", scale=8.0)
    dx, dw, db = R.rapt_layer_norm_bwd(dy, x, w, eps=EPS)
    f = lambda *a: (dy.double() * R.rapt_layer_norm_fwd(*a, eps=EPS).double()).sum().item()
    h = 2.0 ** -4
    for v, grad in ((x, dx), (w, dw), (b, db)):
        for i in range(0, v.numel(), 5):
            flat, keep = v.view(-1), v.view(-1)[i].item()
            flat[i] = keep + h
            up = f(x, w, b)
            flat[i] = keep - h
            down = f(x, w, b)
            flat[i] = keep
            # 2 y values of each of D columns, their rounding 2^-22 of |y| < 8, over 2 h; dy below 4
            assert abs((up - down) / (2 * h) - grad.view(-1)[i].item()) < 2 * D * 4 * 8 * 2.0 ** -22 / h + h * h


@pytest.mark.parametrize("dtype,D", [("bf16", 2048), ("f32", 1001)])
def test_streams_and_graphs(cuda_device, dtype, D):
    """Two graphs captured with one workspace, replayed in turn with new inputs, and two streams at once."""
    x, dy, w, b = inputs(6, 500, D, dtype)
    x2, dy2, _, _ = inputs(7, 500, D, dtype)
    want = [(R.rapt_layer_norm_fwd(p, w, b), *R.rapt_layer_norm_bwd(q, p, w)) for p, q in ((x, dy), (x2, dy2))]
    same = lambda got, k: all(torch.equal(u, v) for u, v in zip(got, want[k]))
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    p, q = x.clone(), dy.clone()
    graphs, outs = [], []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                outs.append((R.rapt_layer_norm_fwd(p, w, b), *R.rapt_layer_norm_bwd(q, p, w, workspace=ws)))
            graphs.append(g)
    torch.cuda.current_stream().wait_stream(side)
    for k, (a, c) in enumerate(((x, dy), (x2, dy2), (x, dy))):
        p.copy_(a)
        q.copy_(c)
        for g in graphs:
            g.replay()
        assert same(outs[0], k % 2) and same(outs[1], k % 2)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    got = [None, None]
    for _ in range(5):
        got[0] = (R.rapt_layer_norm_fwd(x, w, b), *R.rapt_layer_norm_bwd(dy, x, w))
        got[1] = (R.rapt_layer_norm_fwd(x2, w, b, stream=other), *R.rapt_layer_norm_bwd(dy2, x2, w, stream=other))
    torch.cuda.synchronize()
    assert same(got[0], 0) and same(got[1], 1)
