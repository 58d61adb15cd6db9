"""GPU parity of rapt_residual_norm_fwd / _bwd against the fp64 oracle, element by element within the
budgets of block_bounds, over widths that take every path (one warp a row, one CTA a row, eight and
sixteen columns a thread, rows that are not 16-byte aligned), both types, every activation and every
subset of the optional inputs."""

import numpy as np
import pytest
import torch

import block_bounds as BB
from gpu_helpers import to_host
from oracle import block as OB
from relu_linear_attention_gb300 import binding as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
GRADS = ("dx", "dy", "dgate", "dw_post", "dscale", "dw_pre")


def _inputs(T, D, dtype, seed, device):
    g = torch.Generator().manual_seed(seed)
    n = lambda s=1.0: (torch.randn((T, D), generator=g) * s).to(DT[dtype]).to(device)
    u = lambda lo, hi: (torch.rand((D,), generator=g) * (hi - lo) + lo).to(device)
    return dict(x=n(2.0), y=n(), gate=n(2.0), w_post=u(0.5, 1.5), scale=u(-1.0, 1.0), w_pre=u(0.5, 1.5)), n(), n()


def _host(kw):
    return {k: None if v is None else to_host(v) for k, v in kw.items()}


def _check_fwd(kw, act, dtype):
    r, h = R.rapt_residual_norm_fwd(**kw, act=act, eps=EPS)
    rr, rh, br, bh = BB.residual_norm(dtype, *[_host(kw)[k] for k in ("x", "y", "gate", "w_post", "scale", "w_pre")],
                                      act, EPS)
    BB.within(to_host(r), rr, br, "r")
    assert (h is None) == (rh is None)
    if h is not None:
        BB.within(to_host(h), rh, bh, "h")
    return r, h


def _check_bwd(dr, dh, kw, act, dtype):
    got = R.rapt_residual_norm_bwd(dr, dh, **kw, act=act, eps=EPS)
    h = _host({**kw, "dr": dr, "dh": dh})
    ref, bud = BB.residual_norm_bwd(dtype, *[h[k] for k in ("dr", "dh", "x", "y", "gate", "w_post", "scale", "w_pre")],
                                    act, EPS)
    for name, t in zip(GRADS, got):
        assert (t is None) == (name not in ref), name
        if t is not None:
            BB.within(to_host(t), ref[name], bud[name], name)
    return got


SIZES = [(1, 1), (1, 8), (3, 7), (5, 64), (33, 96), (17, 256), (9, 257), (4, 264), (3, 1000), (2, 1537), (700, 520),
         (5, 2048), (3, 2056), (3, 4096), (2, 4100), (2, 5121), (3, 8192), (2, 8200), (2, 12288), (2, 16383), (1, 16384)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D", SIZES)
def test_forward_and_backward_match_the_oracle(cuda_device, lib, T, D, dtype):
    kw, dr, dh = _inputs(T, D, dtype, 100 + T + D, cuda_device)
    _check_fwd(kw, "sigmoid", dtype)
    _check_bwd(dr, dh, kw, "sigmoid", dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", OB.ACTS)
def test_every_activation(cuda_device, lib, act, dtype):
    kw, dr, dh = _inputs(37, 200, dtype, 5, cuda_device)
    _check_fwd(kw, act, dtype)
    _check_bwd(dr, dh, kw, act, dtype)


PARTS = ["no_gate", "no_post", "no_scale", "plain_join", "pre_only", "no_pre", "dr_only", "dh_only"]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [72, 75, 1032])
@pytest.mark.parametrize("parts", PARTS)
def test_every_subset_of_the_inputs(cuda_device, lib, parts, D, dtype):
    kw, dr, dh = _inputs(21, D, dtype, 7, cuda_device)
    drop = dict(no_gate=["gate"], no_post=["w_post"], no_scale=["scale"], plain_join=["gate", "w_post", "scale"],
                pre_only=["y", "gate", "w_post", "scale"], no_pre=["w_pre"]).get(parts, [])
    for k in drop:
        kw[k] = None
    if parts == "dh_only":
        dr = None
    if parts in ("dr_only", "no_pre"):
        dh = None
    r, _ = _check_fwd(kw, "silu", dtype)
    assert (r is kw["x"]) == (parts == "pre_only")
    _check_bwd(dr, dh, kw, "silu", dtype)


def test_backward_without_dh_needs_no_x(cuda_device, lib):
    kw, dr, _ = _inputs(6, 128, "f32", 8, cuda_device)
    want = R.rapt_residual_norm_bwd(dr, None, **kw)
    got = R.rapt_residual_norm_bwd(dr, None, **{**kw, "x": None})
    assert got[5] is None and all(torch.equal(a, b) for a, b in zip(want[:5], got[:5]))


def test_many_rows_give_column_sums_within_their_budget(cuda_device, lib):
    """More rows than CTAs: every CTA sums several, and the warps of a CTA join theirs (D <= 256)."""
    for T, D, dtype in ((6000, 64, "bf16"), (5001, 250, "f32"), (3000, 1024, "bf16")):
        kw, dr, dh = _inputs(T, D, dtype, 9, cuda_device)
        a = _check_bwd(dr, dh, kw, "sigmoid", dtype)
        b = R.rapt_residual_norm_bwd(dr, dh, **kw, act="sigmoid", eps=EPS)
        assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("D", [64, 65, 2048])
def test_outputs_in_place(cuda_device, lib, D):
    kw, dr, dh = _inputs(50, D, "bf16", 10, cuda_device)
    r, h = R.rapt_residual_norm_fwd(**kw)
    k2 = {k: v.clone() for k, v in kw.items()}
    r2, h2 = R.rapt_residual_norm_fwd(**k2, r=k2["x"], h=k2["y"])
    assert r2 is k2["x"] and h2 is k2["y"] and torch.equal(r, r2) and torch.equal(h, h2)
    want = R.rapt_residual_norm_bwd(dr, dh, **kw)
    k2 = {k: v.clone() for k, v in kw.items()}
    got = R.rapt_residual_norm_bwd(dr, dh, **k2, dx=dr, dy=k2["y"], dgate=k2["gate"])
    assert got[0] is dr and all(torch.equal(a, b) for a, b in zip(want, got))


def test_no_rows(cuda_device, lib):
    kw, dr, dh = _inputs(0, 96, "bf16", 11, cuda_device)
    r, h = R.rapt_residual_norm_fwd(**kw)
    assert r.shape == (0, 96) and h.shape == (0, 96)
    got = R.rapt_residual_norm_bwd(dr, dh, **kw)
    assert all(not t.any() for t in got[3:]) and got[0].shape == (0, 96)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_row_depends_on_no_other(cuda_device, lib, dtype):
    """Zeros, the largest values, infinities and NaN in some rows leave the others' bits alone."""
    kw, dr, dh = _inputs(40, 192, dtype, 12, cuda_device)
    clean = R.rapt_residual_norm_fwd(**kw), R.rapt_residual_norm_bwd(dr, dh, **kw)[:3]
    bad = {k: v.clone() if k in ("x", "y", "gate") else v for k, v in kw.items()}
    bad["x"][3], bad["y"][3] = 0.0, 0.0
    bad["y"][7, 5] = float("nan")
    bad["x"][11, 0] = float("inf")
    bad["gate"][13] = -1e30
    bad["gate"][14] = 1e30
    bad["x"][20] = torch.finfo(DT[dtype]).max
    rest = [i for i in range(40) if i not in (3, 7, 11, 13, 14, 20)]
    got = R.rapt_residual_norm_fwd(**bad), R.rapt_residual_norm_bwd(dr, dh, **bad)[:3]
    for a, b in zip(clean[0] + clean[1], got[0] + got[1]):
        assert torch.equal(a[rest], b[rest])
    r, h = got[0]
    assert not r[3].any() and not h[3].any()          # rows of zeros: 0 eps^(-1/2) = 0
    assert torch.isnan(r[7]).all()                     # a NaN in y reaches its whole row
    assert torch.equal(r[13], bad["x"][13])            # sigmoid(-1e30) = 0 exactly
    assert torch.isfinite(r[14].float()).all()


def test_leading_dimensions_and_another_stream(cuda_device, lib):
    kw, dr, dh = _inputs(24, 128, "bf16", 13, cuda_device)
    want = R.rapt_residual_norm_fwd(**kw), R.rapt_residual_norm_bwd(dr, dh, **kw)
    v = {k: t.view(2, 3, 4, 128) if t.dim() == 2 else t for k, t in kw.items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = R.rapt_residual_norm_fwd(**v, stream=s), R.rapt_residual_norm_bwd(dr.view(2, 3, 4, 128), dh.view(2, 3, 4, 128),
                                                                            **v, stream=s)
    s.synchronize()
    for a, b in zip(want[0] + want[1], got[0] + got[1]):
        assert torch.equal(a, b.view(a.shape))


def test_captured_and_replayed(cuda_device, lib):
    kw, dr, dh = _inputs(300, 512, "bf16", 14, cuda_device)
    other, dr2, dh2 = _inputs(300, 512, "bf16", 15, cuda_device)
    R.rapt_residual_norm_fwd(**kw), R.rapt_residual_norm_bwd(dr, dh, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f, b = R.rapt_residual_norm_fwd(**kw), R.rapt_residual_norm_bwd(dr, dh, **kw)
    for k in kw:
        kw[k].copy_(other[k])
    dr.copy_(dr2), dh.copy_(dh2)
    want = R.rapt_residual_norm_fwd(**other), R.rapt_residual_norm_bwd(dr2, dh2, **other)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want[0] + want[1], f + b))


def test_rows_past_32_bit_offsets(cuda_device, lib):
    """T D over 2^31: the last rows' values against the same rows computed alone."""
    D, T = 16384, 131076
    x = torch.zeros((T, D), device=cuda_device, dtype=torch.bfloat16)
    g = torch.Generator(device=cuda_device).manual_seed(3)
    tail = torch.randn((4, D), generator=g, device=cuda_device).to(torch.bfloat16)
    x[-4:] = tail
    w = torch.ones(D, device=cuda_device)
    _, h = R.rapt_residual_norm_fwd(x, w_pre=w)
    assert torch.equal(h[-4:], R.rapt_residual_norm_fwd(tail, w_pre=w)[1])
    assert not h[:-4].any()


# Rows that start at different places of a 16-byte vector: a thread's rows have to start at the same one,
# so that many more rows than CTAs (or rows of a CTA) are in question, and their neighbours' values.
@pytest.mark.parametrize("T,D", [(9001, 1), (6001, 3), (5003, 65), (6001, 257), (3001, 1001), (1201, 1538), (701, 4093),
                                 (353, 4099), (331, 8190), (331, 8195), (307, 16381)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_rows_of_odd_widths(cuda_device, lib, T, D, dtype):
    kw, dr, dh = _inputs(T, D, dtype, T + D, cuda_device)
    _check_fwd(kw, "silu", dtype)
    got = _check_bwd(dr, dh, kw, "silu", dtype)
    for a, b in zip(got, R.rapt_residual_norm_bwd(dr, dh, **kw, act="silu", eps=EPS)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,D", [(301, 257), (901, 1001), (170, 8195)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_row_leaves_its_neighbours(cuda_device, lib, T, D, dtype):
    """NaN and infinite rows reach no other row, in place too: the pieces that rows share are split."""
    kw, dr, dh = _inputs(T, D, dtype, 3, cuda_device)
    r, h = R.rapt_residual_norm_fwd(**kw, act="gelu", eps=EPS)
    grads = R.rapt_residual_norm_bwd(dr, dh, **kw, act="gelu", eps=EPS)[:3]
    bad = torch.arange(1, T, 3, device=cuda_device)
    rest = torch.ones(T, dtype=torch.bool, device=cuda_device)
    rest[bad] = False
    ill = {k: v.clone() if v.dim() == 2 else v for k, v in kw.items()}
    for k in ("x", "y", "gate"):
        ill[k][bad] = float("nan") if k != "y" else float("inf")
    dri, dhi = dr.clone(), dh.clone()
    dri[bad] = float("nan")
    dhi[bad] = float("-inf")
    gi = R.rapt_residual_norm_bwd(dri, dhi, **ill, act="gelu", eps=EPS)[:3]
    for a, b in zip(grads, gi):
        assert torch.equal(a[rest], b[rest])
    ri, hi = R.rapt_residual_norm_fwd(**ill, act="gelu", eps=EPS, r=ill["x"], h=ill["y"])
    assert ri.data_ptr() == ill["x"].data_ptr()
    assert torch.equal(ri[rest], r[rest]) and torch.equal(hi[rest], h[rest])
    assert torch.isnan(ri[bad]).all()


# Every choice of columns a thread and of ring, with more rows than are in flight at once.
@pytest.mark.parametrize("T,D", [(12000, 300), (9000, 512), (5000, 768), (4000, 1536), (1500, 2052), (1500, 2560), (800, 3600),
                                 (700, 4100), (700, 5120), (640, 6144), (640, 7000), (480, 8200), (480, 9300), (480, 10800),
                                 (480, 12296), (480, 16384)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rings_of_every_width(cuda_device, lib, T, D, dtype):
    kw, dr, dh = _inputs(T, D, dtype, T * D, cuda_device)
    _check_fwd(kw, "sigmoid", dtype)
    _check_bwd(dr, dh, kw, "sigmoid", dtype)


@pytest.mark.parametrize("T,D", [(1400, 300), (700, 2560), (400, 6400), (400, 9300)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("parts", PARTS)
def test_rings_without_some_of_the_inputs(cuda_device, lib, parts, T, D, dtype):
    kw, dr, dh = _inputs(T, D, dtype, 7, cuda_device)
    drop = dict(no_gate=["gate"], no_post=["w_post"], no_scale=["scale"], plain_join=["gate", "w_post", "scale"],
                pre_only=["y", "gate", "w_post", "scale"], no_pre=["w_pre"]).get(parts, [])
    kw.update((k, None) for k in drop)
    _check_fwd(kw, "silu", dtype)
    _check_bwd(None if parts == "dh_only" else dr, None if parts in ("dr_only", "no_pre") else dh, kw, "silu", dtype)


@pytest.mark.parametrize("T,D", [(1400, 300), (700, 2560), (400, 6400), (400, 9300), (300, 12401)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rings_in_place(cuda_device, lib, T, D, dtype):
    kw, dr, dh = _inputs(T, D, dtype, 12, cuda_device)
    grads = R.rapt_residual_norm_bwd(dr, dh, **kw, act="relu", eps=EPS)
    own = {k: v.clone() for k, v in kw.items()}
    got = R.rapt_residual_norm_bwd(dr, dh, **own, act="relu", eps=EPS, dx=own["y"], dy=own["gate"], dgate=own["x"])
    for a, b in zip(grads, got):
        assert torch.equal(a, b)
    r, h = R.rapt_residual_norm_fwd(**kw, act="relu", eps=EPS)
    own = {k: v.clone() for k, v in kw.items()}
    ri, hi = R.rapt_residual_norm_fwd(**own, act="relu", eps=EPS, r=own["gate"], h=own["x"])
    assert torch.equal(r, ri) and torch.equal(h, hi)
