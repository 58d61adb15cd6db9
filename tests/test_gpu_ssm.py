"""The selective scan on the GPU against the fp64 oracle: prompts (dense, packed) and single tokens."""

import numpy as np
import pytest
import torch

import ssm_bounds as SB
from block_bounds import within
from relu_linear_attention_gb300 import binding as R
from ssm_inputs import document, host, scan_inputs, state

pytestmark = pytest.mark.gpu


def on_chunks(dtype, P, N):
    return dtype == "bf16" and P >= 64 and N >= 64


def check(got, S, args, opts, at, dtype, what, S0=None, softplus=True):
    """One document's out and final state against the oracle."""
    k = document(args, opts, at)
    chunks = on_chunks(dtype, k["x"].shape[-1], k["B"].shape[-1])
    ref, refS, eo, eS = SB.scan(dtype, **k, dt_softplus=softplus, S0=None if S0 is None else host(S0), chunks=chunks)
    within(host(got), ref, eo + 1e-30, what + " out")
    if S is not None:
        within(host(S), refS, eS + 1e-30, what + " S")


# (H, P, G, N): every head size with every state size, heads alone in a group and in odd numbers
SHAPES = [(2, 16, 1, 16), (3, 16, 3, 128), (4, 32, 2, 16), (1, 32, 1, 32), (2, 64, 2, 32), (3, 64, 1, 64), (5, 64, 1, 128),
          (4, 64, 2, 64), (6, 64, 3, 128), (2, 128, 1, 64), (3, 128, 3, 128), (1, 128, 1, 16), (2, 16, 1, 64),
          (4, 128, 2, 128), (2, 64, 2, 128), (2, 32, 1, 128)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(cuda_device, shape, dtype):
    H, P, G, N = shape
    args, opts = scan_inputs(1, (2, 150), H, P, G, N, dtype)
    S0 = state(2, 2, H, N, P)
    keep = S0.clone()
    out, S = R.rapt_ssm_prefill_fwd(**args, **opts, S0=S0, final_state=True)
    assert torch.equal(S0, keep)
    for b in range(2):
        check(out[b], S[b], args, opts, b, dtype, "row %d" % b, S0[b])


@pytest.mark.parametrize("shape,dtype", [((2, 64, 1, 128), "bf16"), ((3, 128, 3, 64), "bf16"), ((2, 32, 1, 16), "f32"),
                                         ((3, 16, 1, 32), "bf16"), ((2, 64, 2, 64), "f32")])
@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 385, 640])
def test_lengths(cuda_device, shape, dtype, L):
    args, opts = scan_inputs(L, (1, L), *shape, dtype)
    out, S = R.rapt_ssm_prefill_fwd(**args, **opts, final_state=True)
    check(out[0], S[0], args, opts, 0, dtype, "L %d" % L)


@pytest.mark.parametrize("shape,dtype", [((2, 64, 1, 128), "bf16"), ((2, 128, 1, 128), "bf16"), ((2, 32, 1, 16), "f32")])
@pytest.mark.parametrize("missing", ["z", "D", "bias", "all"])
def test_options(cuda_device, shape, dtype, missing):
    kw = {k: missing not in (k, "all") for k in ("z", "D", "bias")}
    args, opts = scan_inputs(7, (1, 200), *shape, dtype, sliced=missing != "z", **kw)
    softplus = missing != "all"
    if not softplus:
        args["dt"] = torch.rand_like(args["dt"], dtype=torch.float32).to(args["dt"].dtype) * 0.1
    out, S = R.rapt_ssm_prefill_fwd(**args, **opts, dt_softplus=softplus)
    assert S is None
    check(out[0], None, args, opts, 0, dtype, missing, softplus=softplus)


@pytest.mark.parametrize("dtype,shape", [("bf16", (2, 64, 1, 128)), ("bf16", (1, 128, 1, 64)), ("f32", (2, 16, 2, 16))])
@pytest.mark.parametrize("decay", [(1e-6, 1e-5), (200.0, 4000.0), (0.0, 0.0)])
def test_decays(cuda_device, dtype, shape, decay):
    """States that forget nothing, and ones that forget all at once: logarithms of decays down to -1e5 a chunk."""
    args, opts = scan_inputs(8, (1, 300), *shape, dtype, decay=decay)
    out, S = R.rapt_ssm_prefill_fwd(**args, **opts, final_state=True)
    check(out[0], S[0], args, opts, 0, dtype, "decay")


@pytest.mark.parametrize("dtype,shape", [("bf16", (2, 64, 1, 128)), ("f32", (2, 32, 1, 16))])
def test_steps_far_out(cuda_device, dtype, shape):
    """Raw steps at both ends of the softplus: tokens that change nothing, and ones that wipe the state."""
    args, opts = scan_inputs(9, (1, 260), *shape, dtype)
    dt = args["dt"] = args["dt"].contiguous()
    dt[0, 3::7] = -200.0
    dt[0, 5::11] = 90.0
    out, S = R.rapt_ssm_prefill_fwd(**args, **opts, final_state=True)
    assert torch.isfinite(out.float()).all() and torch.isfinite(S).all()
    check(out[0], S[0], args, opts, 0, dtype, "far out")


@pytest.mark.parametrize("dtype,shape", [("bf16", (3, 64, 1, 64)), ("bf16", (4, 64, 2, 128)), ("bf16", (2, 128, 1, 128)),
                                         ("bf16", (2, 32, 1, 16)), ("f32", (2, 64, 1, 32))])
def test_packed(cuda_device, dtype, shape):
    H, P, G, N = shape
    lens = [0, 1, 130, 0, 128, 5, 127, 300, 0, 33, 0]
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    args, opts = scan_inputs(10, (int(cu[-1]),), H, P, G, N, dtype)
    S0 = state(11, len(lens), H, N, P)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, S = R.rapt_ssm_varlen_fwd(**args, **opts, cu_seqlens=torch.from_numpy(cu).cuda(), max_seqlen=300, S0=S0,
                                   final_state=True, dev_status=status)
    assert status.item() == 0
    for i, n in enumerate(lens):
        check(out[cu[i]:cu[i + 1]], S[i], args, opts, slice(cu[i], cu[i + 1]), dtype, "document %d" % i, S0[i])


@pytest.mark.parametrize("dtype,shape", [("bf16", (2, 64, 1, 128)), ("bf16", (1, 128, 1, 64)), ("f32", (2, 16, 1, 32))])
@pytest.mark.parametrize("packed", [False, True])
def test_segments(cuda_device, dtype, shape, packed):
    """Few heads and long documents, cut into segments: the workspace says so. Against the oracle's last state and
    against the same tokens given in pieces, each from the state of the one before."""
    H, P, G, N = shape
    L = 3000
    args, opts = scan_inputs(12, (L,) if packed else (1, L), H, P, G, N, dtype)
    S0 = state(13, 1, H, N, P)
    if packed:
        cu = torch.tensor([0, L], dtype=torch.int32, device="cuda")
        call = lambda **kw: R.rapt_ssm_varlen_fwd(**args, **opts, cu_seqlens=cu, max_seqlen=L, **kw)
    else:
        call = lambda **kw: R.rapt_ssm_prefill_fwd(**args, **opts, **kw)
    with pytest.raises(R._lib.RaptError):  # there are segments: their records want room
        call(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    out, S = call(S0=S0, final_state=True)
    check(out if packed else out[0], S[0], args, opts, slice(None) if packed else 0, dtype, "segments", S0[0])
    out2, S2 = call(S0=S0, final_state=True)
    assert torch.equal(out, out2) and torch.equal(S, S2)


def test_malformed_documents_are_reported(cuda_device):
    """Bounds that go back or do not end at T: reported, and what lies outside the good documents is left alone."""
    for dtype, shape in (("bf16", (2, 64, 1, 64)), ("f32", (2, 16, 1, 16))):
        args, opts = scan_inputs(14, (64,), *shape, dtype)
        for cu in ([0, 20, 10, 64], [0, 30, 60, 63], [1, 30, 60, 64], [0, 30, 70, 64]):
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            out = torch.full((64,) + tuple(args["x"].shape[1:]), 7.0, dtype=args["x"].dtype, device="cuda")
            R.rapt_ssm_varlen_fwd(**args, **opts, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"),
                                  max_seqlen=64, out=out, dev_status=status)
            assert status.item() == 1, cu
        assert torch.all(out[30:60] == 7.0) or torch.isfinite(out.float()).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("n", [1, 3, 70])
def test_single_tokens(cuda_device, shape, dtype, n):
    H, P, G, N = shape
    args, opts = scan_inputs(15, (n,), H, P, G, N, dtype)
    S = state(16, n, H, N, P)
    S0 = S.clone()
    out = R.rapt_ssm_decode_step(**args, **opts, S=S)
    for i in range(n) if n < 8 else (0, 31, n - 1):
        k = document(args, opts, slice(i, i + 1))
        ref, refS, eo, eS = SB.scan(dtype, **k, S0=host(S0[i]))
        within(host(out[i:i + 1]), ref, eo + 1e-30, "token %d out" % i)
        within(host(S[i]), refS, eS + 1e-30, "token %d S" % i)


@pytest.mark.parametrize("dtype,shape", [("bf16", (4, 64, 2, 64)), ("f32", (2, 32, 1, 16))])
def test_tokens_after_a_prompt(cuda_device, dtype, shape):
    """A prompt, then single tokens on its state: the document as a whole."""
    H, P, G, N = shape
    args, opts = scan_inputs(17, (3, 140), H, P, G, N, dtype)
    part = lambda s: ({k: v if k == "A" else v[:, s].contiguous() for k, v in args.items()},
                      {k: v[:, s].contiguous() if k == "z" else v for k, v in opts.items()})
    a, o = part(slice(0, 133))
    outs, S = R.rapt_ssm_prefill_fwd(**a, **o, final_state=True)
    outs = [outs]
    for t in range(133, 140):
        a, o = part(t)
        outs.append(R.rapt_ssm_decode_step(**a, **o, S=S)[:, None])
    out = torch.cat(outs, 1)
    for b in range(3):
        check(out[b], S[b], args, opts, b, dtype, "row %d" % b)


def test_no_tokens(cuda_device):
    args, opts = scan_inputs(18, (2, 0), 2, 64, 1, 64, "bf16", sliced=False)
    S0 = state(19, 2, 2, 64, 64)
    out, S = R.rapt_ssm_prefill_fwd(**args, **opts, S0=S0, final_state=True)
    assert out.shape == (2, 0, 2, 64) and torch.equal(S, S0)
    assert torch.equal(R.rapt_ssm_prefill_fwd(**args, **opts, final_state=True)[1], torch.zeros_like(S0))


@pytest.mark.parametrize("dtype,shape", [("bf16", (4, 64, 1, 128)), ("f32", (2, 16, 1, 16))])
def test_streams_and_graphs(cuda_device, dtype, shape):
    """A call on a stream of its own, and two captured graphs of calls that each hold their workspace, replayed in
    turn on new inputs, give the bits of a plain call."""
    args, opts = scan_inputs(20, (1, 900), *shape, dtype)
    want = R.rapt_ssm_prefill_fwd(**args, **opts, final_state=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = R.rapt_ssm_prefill_fwd(**args, **opts, final_state=True, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):
        mine = {k: v.clone() for k, v in args.items()}
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = R.rapt_ssm_prefill_fwd(**mine, **opts, final_state=True)
        graphs.append((g, mine, res))
    for turn in range(3):
        fresh = [scan_inputs(30 + 2 * turn + i, (1, 900), *shape, dtype)[0] for i in range(2)]
        for (g, mine, res), new in zip(graphs, fresh):
            for k in ("x", "dt", "B", "C"):
                mine[k].copy_(new[k])
            g.replay()
        for (g, mine, res), new in zip(graphs, fresh):
            new["A"] = args["A"]
            ref = R.rapt_ssm_prefill_fwd(**new, **opts, final_state=True)
            assert all(torch.equal(a, b) for a, b in zip(res, ref))


def test_refuses_layouts(cuda_device):
    args, opts = scan_inputs(21, (2, 16), 2, 64, 1, 64, "bf16")
    for k, v in (("x", args["x"][:, ::2]), ("x", args["x"].transpose(2, 3)), ("dt", args["dt"].float()),
                 ("B", args["B"][..., :32]), ("A", args["A"][:1]), ("C", args["C"].cpu())):
        with pytest.raises(ValueError):
            R.rapt_ssm_prefill_fwd(**{**args, k: v}, **opts)
    odd = torch.empty(2, 16, 2 * 64 + 4, dtype=torch.bfloat16, device="cuda")[..., :128].unflatten(-1, (2, 64))
    with pytest.raises(R._lib.RaptError):  # rows at no multiple of 16 bytes
        R.rapt_ssm_prefill_fwd(**{**args, "x": odd}, **opts)
