"""GPU parity of the gated feed-forward (rapt_glu_fwd / _bwd) and of the projection gradients
(rapt_linear_bwd) against the fp64 oracle, element by element within the budgets of block_bounds: one
row and one tile's edge in every dimension, sums split into parts, every activation."""

import threading

import numpy as np
import pytest
import torch

import block_bounds as BB
from gpu_helpers import to_host
from oracle import block as OB
from relu_linear_attention_gb300 import binding as R

pytestmark = pytest.mark.gpu


def _normal(shape, seed, device, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16).to(device)


def _glu_inputs(M, F, K, seed, device):
    return (_normal((M, F), seed, device), _normal((M, K), seed + 1, device),
            _normal((F, K), seed + 2, device, K ** -0.5), _normal((F, K), seed + 3, device, K ** -0.5))


def _status(device):
    return torch.zeros(1, dtype=torch.int32, device=device)


SHAPES = [(1, 8, 8), (1, 128, 64), (2, 136, 72), (7, 2744, 1032), (8, 64, 512), (9, 200, 264), (16, 1024, 256),
          (31, 40, 2048), (33, 264, 136), (64, 512, 512), (65, 512, 128), (100, 1000, 200), (128, 128, 64),
          (129, 136, 72), (256, 256, 256), (257, 264, 520), (500, 72, 1000), (1000, 520, 72), (300, 2048, 96)]


@pytest.mark.parametrize("M,F,K", SHAPES)
def test_glu_forward_matches_the_oracle(cuda_device, lib, M, F, K):
    _, x, wg, wu = _glu_inputs(M, F, K, 1000 + M, cuda_device)
    st = _status(cuda_device)
    h = R.rapt_glu_fwd(x, wg, wu, dev_status=st)
    ref, bud = BB.glu(to_host(x), to_host(wg), to_host(wu), "silu")
    BB.within(to_host(h), ref, bud, "h")
    assert int(st.item()) == 0
    assert torch.equal(h, R.rapt_glu_fwd(x, wg, wu))


@pytest.mark.parametrize("M,F,K", SHAPES)
def test_glu_backward_matches_the_oracle(cuda_device, lib, M, F, K):
    dh, x, wg, wu = _glu_inputs(M, F, K, 2000 + M, cuda_device)
    st = _status(cuda_device)
    got = R.rapt_glu_bwd(dh, x, wg, wu, dev_status=st)
    ref, bud = BB.glu_bwd(to_host(dh), to_host(x), to_host(wg), to_host(wu), "silu")
    for name, a, b, c in zip(("dx", "dw_gate", "dw_up"), got, ref, bud):
        BB.within(to_host(a), b, c, name)
    assert int(st.item()) == 0
    assert all(torch.equal(a, b) for a, b in zip(got, R.rapt_glu_bwd(dh, x, wg, wu)))


@pytest.mark.parametrize("M", [3, 150])
@pytest.mark.parametrize("act", OB.ACTS)
def test_glu_every_activation(cuda_device, lib, act, M):
    dh, x, wg, wu = _glu_inputs(M, 136, 264, 30, cuda_device)
    hx, hg, hu = to_host(x), to_host(wg), to_host(wu)
    BB.within(to_host(R.rapt_glu_fwd(x, wg, wu, act=act)), *BB.glu(hx, hg, hu, act), "h")
    ref, bud = BB.glu_bwd(to_host(dh), hx, hg, hu, act)
    for a, b, c in zip(R.rapt_glu_bwd(dh, x, wg, wu, act=act), ref, bud):
        BB.within(to_host(a), b, c, act)


@pytest.mark.parametrize("M,N,K", [(1, 8, 8), (1, 1024, 64), (5, 24, 40), (64, 64, 64), (65, 72, 56), (130, 264, 520),
                                   (128, 256, 256), (129, 257 * 8, 264), (1000, 40, 1000), (3000, 256, 136),
                                   (20000, 64, 72), (4099, 520, 264),
                                   (300, 192, 320), (200, 128, 1088)])
def test_linear_backward_matches_the_oracle(cuda_device, lib, M, N, K):
    dy, x, w = (_normal(s, 40 + i, cuda_device) for i, s in enumerate(((M, N), (M, K), (N, K))))
    st = _status(cuda_device)
    dx, dw = R.rapt_linear_bwd(dy, x, w, dev_status=st)
    rx, rw, bx, bw = BB.linear_bwd(to_host(dy), to_host(x), to_host(w))
    BB.within(to_host(dx), rx, bx, "dx")
    BB.within(to_host(dw), rw, bw, "dw")
    assert int(st.item()) == 0
    a, b = R.rapt_linear_bwd(dy, x, None, need_dx=False), R.rapt_linear_bwd(dy, None, w, need_dw=False)
    assert a[0] is None and b[1] is None and torch.equal(a[1], dw) and torch.equal(b[0], dx)
    assert all(torch.equal(p, q) for p, q in zip((dx, dw), R.rapt_linear_bwd(dy, x, w)))


def test_glu_backward_parts(cuda_device, lib):
    dh, x, wg, wu = _glu_inputs(200, 264, 136, 50, cuda_device)
    dx, dwg, dwu = R.rapt_glu_bwd(dh, x, wg, wu)
    a, b = R.rapt_glu_bwd(dh, x, wg, wu, need_dw=False), R.rapt_glu_bwd(dh, x, wg, wu, need_dx=False)
    assert a[1] is None and a[2] is None and torch.equal(a[0], dx)
    assert b[0] is None and torch.equal(b[1], dwg) and torch.equal(b[2], dwu)


def test_no_tokens(cuda_device, lib):
    dh, x, wg, wu = _glu_inputs(0, 64, 128, 60, cuda_device)
    assert R.rapt_glu_fwd(x, wg, wu).shape == (0, 64)
    dx, dwg, dwu = R.rapt_glu_bwd(dh, x, wg, wu)
    assert dx.shape == (0, 128) and not dwg.any() and not dwu.any()
    dx, dw = R.rapt_linear_bwd(dh, x, wg)
    assert dx.shape == (0, 128) and not dw.any() and dw.shape == (64, 128)


@pytest.mark.parametrize("M", [20, 300])
def test_a_row_of_tokens_depends_on_no_other(cuda_device, lib, M):
    dh, x, wg, wu = _glu_inputs(M, 264, 136, 70, cuda_device)
    h, dx = R.rapt_glu_fwd(x, wg, wu), R.rapt_glu_bwd(dh, x, wg, wu, need_dw=False)[0]
    bad = x.clone()
    bad[2, 3], bad[M - 1, 0] = float("nan"), float("inf")
    h2, dx2 = R.rapt_glu_fwd(bad, wg, wu), R.rapt_glu_bwd(dh, bad, wg, wu, need_dw=False)[0]
    rest = [i for i in range(M) if i not in (2, M - 1)]
    assert torch.equal(h[rest], h2[rest]) and torch.equal(dx[rest], dx2[rest])
    assert torch.isnan(h2[2]).all()


@pytest.mark.parametrize("M", [5, 200])
def test_nothing_is_written_behind_the_last_row_or_column(cuda_device, lib, M):
    """Outputs inside larger buffers: the guard bytes before and behind keep their values."""
    F, K = 72, 136
    dh, x, wg, wu = _glu_inputs(M, F, K, 80, cuda_device)

    def guarded(rows, cols):
        n = rows * cols
        buf = torch.full((n + 4096,), 7.0, device=cuda_device, dtype=torch.bfloat16)
        return buf, buf[2048:2048 + n].view(rows, cols)

    bufs = [guarded(M, F), guarded(M, K), guarded(F, K), guarded(F, K)]
    h = R.rapt_glu_fwd(x, wg, wu, h=bufs[0][1])
    dx, dwg, dwu = R.rapt_glu_bwd(dh, x, wg, wu, dx=bufs[1][1], dw_gate=bufs[2][1], dw_up=bufs[3][1])
    assert torch.equal(h, R.rapt_glu_fwd(x, wg, wu))
    assert all(torch.equal(a, b) for a, b in zip((dx, dwg, dwu), R.rapt_glu_bwd(dh, x, wg, wu)))
    for buf, t in bufs:
        assert (buf[:2048] == 7).all() and (buf[2048 + t.numel():] == 7).all()


def test_captured_graphs_and_streams(cuda_device, lib):
    """Two captured graphs with workspaces of their own, replayed one after the other on other inputs,
    and a call on another stream."""
    ins = [_glu_inputs(M, 264, 520, 90 + M, cuda_device) for M in (150, 9)]
    lin = [(_normal((2000, 64), 95, cuda_device), _normal((2000, 72), 96, cuda_device), _normal((64, 72), 97, cuda_device))]
    run = lambda i: (R.rapt_glu_fwd(*ins[i][1:]), *R.rapt_glu_bwd(*ins[i]), *R.rapt_linear_bwd(*lin[0]))
    run(0), run(1)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in (0, 1):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(i))
        graphs.append(g)
    for i in (0, 1):
        for t in ins[i]:
            t.copy_(t.flip(0))
    want = [run(0), run(1)]
    graphs[1].replay(), graphs[0].replay(), graphs[1].replay()
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(a, b) for a, b in zip(want[i], outs[i]))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = R.rapt_glu_fwd(*ins[0][1:], stream=s), *R.rapt_glu_bwd(*ins[0], stream=s), *R.rapt_linear_bwd(*lin[0], stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want[0], got))


def test_two_threads_on_streams_of_their_own(cuda_device, lib):
    ins = _glu_inputs(700, 520, 264, 110, cuda_device)
    want = R.rapt_glu_bwd(*ins)
    torch.cuda.synchronize()
    got = [None, None]

    def work(i):
        s = torch.cuda.Stream()
        for _ in range(5):
            got[i] = R.rapt_glu_bwd(*ins, stream=s)
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(want, g))


def test_layer_sizes_on_sampled_rows(cuda_device, lib):
    """16384 tokens, d_model 2048, hidden 5504: sampled rows of h and dx, sampled rows of the weight
    gradients (each a sum over all tokens), as exact products in 64 bits."""
    M, F, K = 16384, 5504, 2048
    dh, x, wg, wu = _glu_inputs(M, F, K, 120, cuda_device)
    h, (dx, dwg, dwu) = R.rapt_glu_fwd(x, wg, wu), R.rapt_glu_bwd(dh, x, wg, wu)
    rows = torch.tensor([0, 1, 127, 128, 4095, 8191, 16383], device=cuda_device)
    hx, hg, hu, hd = to_host(x[rows]), to_host(wg), to_host(wu), to_host(dh[rows])
    BB.within(to_host(h[rows]), *BB.glu(hx, hg, hu, "silu"), "h")
    ref, bud = BB.glu_bwd(hd, hx, hg, hu, "silu")
    BB.within(to_host(dx[rows]), ref[0], bud[0], "dx")
    cols = torch.tensor([0, 63, 127, 128, 2751, 5503], device=cuda_device)
    ref, bud = BB.glu_bwd(to_host(dh[:, cols]), to_host(x), to_host(wg[cols]), to_host(wu[cols]), "silu")
    BB.within(to_host(dwg[cols]), ref[1], bud[1], "dw_gate")
    BB.within(to_host(dwu[cols]), ref[2], bud[2], "dw_up")
