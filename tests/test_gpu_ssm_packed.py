"""Packed documents on the ways that the scan's plans take: whole and the longest first, cut into segments, more
documents than are sorted. The size of the workspace tells which; against the fp64 oracle, and what a call may not
touch."""

import ctypes

import numpy as np
import pytest
import torch

import ssm_bounds as SB
from block_bounds import within
from oracle import ssm as OS
from relu_linear_attention_gb300 import _lib, binding as R
from ssm_inputs import document, host, scan_inputs, state

pytestmark = pytest.mark.gpu


def plan_bytes(args, T, N, longest):
    """The workspace of a packed call, without its inputs' addresses."""
    x, b = args["x"], args["B"]
    a = _lib.rapt_ssm_inputs(H=x.shape[1], P=x.shape[2], G=b.shape[1], Ns=b.shape[2], dt_softplus=1,
                             dtype=_lib.RAPT_BF16 if x.dtype == torch.bfloat16 else _lib.RAPT_F32)
    return _lib.load().rapt_ssm_varlen_workspace_size(ctypes.byref(a), T, N, longest)


def pack(lens):
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    return cu, torch.from_numpy(cu).cuda()


def check(out, S, args, opts, cu, i, dtype, S0=None, chunks=True):
    """Document i. Its state in chunks: w = w1 + w2 + 2^-16 w, hi = bf16(x w1) leaves an exact remainder of 2^-8 of
    the term, x w2 is another 2^-8, their sum is rounded to 2^-8 of itself: 2^-16 + 2^-15 of a term's magnitude."""
    at = slice(cu[i], cu[i + 1])
    k = document(args, opts, at)
    first = None if S0 is None else host(S0[i])
    ref, refS, eo, eS = SB.scan(dtype, **k, S0=first, chunks=chunks)
    if chunks:
        mag = OS.scan(np.abs(k["x"]), k["dt"], k["A"], np.abs(k["B"]), np.abs(k["C"]), dt_bias=k["dt_bias"],
                      S0=None if S0 is None else np.abs(first))[1]
        eS = eS + 1.5 * 2.0 ** -15 * mag
    within(host(out[at]), ref, eo + 1e-30, "document %d out" % i)
    if S is not None:
        within(host(S[i]), refS, eS + 1e-30, "document %d S" % i)


# lengths, (H, P, G, N), type: whole and sorted (an odd head of a group among them, heads of 128), in segments of
# which some documents have fewer than the plan's, none or no token
RNG = np.random.RandomState(1)
MANY = [int(n) for n in RNG.randint(0, 500, 40)] + [0, 1, 128, 500]
FEW = [0, 2500, 130, 900, 0, 1, 257]
WAYS = {
    "sorted": (MANY, (8, 64, 4, 64), "bf16"),
    "sorted, odd heads": (MANY, (9, 64, 3, 128), "bf16"),
    "sorted, heads of 128": (MANY, (4, 128, 2, 64), "bf16"),
    "segments": (FEW, (2, 64, 1, 64), "bf16"),
    "segments, odd heads": (FEW, (3, 64, 1, 128), "bf16"),
    "segments, heads of 128": (FEW, (2, 128, 1, 128), "bf16"),
    "segments on CUDA cores": (FEW, (2, 32, 1, 16), "f32"),
}


def make(way, seed=1):
    lens, (H, P, G, N), dtype = WAYS[way]
    cu, dev = pack(lens)
    args, opts = scan_inputs(seed, (int(cu[-1]),), H, P, G, N, dtype)
    need = plan_bytes(args, int(cu[-1]), len(lens), max(lens))
    # the order of the documents, or records of the states
    assert need == 4 * len(lens) if way.startswith("sorted") else need >= H * N * P * 4 * 3, "another plan"
    return lens, cu, dev, args, opts, state(seed + 1, len(lens), H, N, P), dtype


@pytest.mark.parametrize("way", WAYS)
def test_ways_of_the_plan(cuda_device, way):
    lens, cu, dev, args, opts, S0, dtype = make(way)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, S = R.rapt_ssm_varlen_fwd(**args, **opts, cu_seqlens=dev, max_seqlen=max(lens), S0=S0, final_state=True,
                                   dev_status=status)
    assert status.item() == 0
    for i in range(len(lens)):
        check(out, S, args, opts, cu, i, dtype, S0, chunks=dtype == "bf16")


@pytest.mark.parametrize("way", WAYS)
def test_malformed_documents_touch_nothing(cuda_device, way):
    """Bounds that go back, leave [0, T], exceed the longest or do not end at T: reported; the good documents are
    right, and the rows and final states of the others keep what was there."""
    lens, cu, dev, args, opts, S0, dtype = make(way)
    T, N, longest = int(cu[-1]), len(lens), max(lens)
    H, P = args["x"].shape[1:]
    k = int(np.argmax(lens))
    for change in ({k + 1: cu[k] - 1}, {N: T - 1}, {0: 1}, {2: T + 5}, {3: -7}, {k + 1: cu[k + 1] + 1}):
        bad = cu.copy()
        for at, v in change.items():
            bad[at] = v
        ok = [i for i in range(N) if 0 <= bad[i] <= bad[i + 1] <= T and bad[i + 1] - bad[i] <= longest
              and (bad[i - 1] <= bad[i] if i else bad[i] == 0) and (i < N - 1 or bad[N] == T)]
        assert len(ok) < N
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((T, H, P), 7.0, dtype=args["x"].dtype, device="cuda")
        S = torch.full_like(S0, 7.0)
        R.rapt_ssm_varlen_fwd(**args, **opts, cu_seqlens=torch.from_numpy(bad).cuda(), max_seqlen=longest, S0=S0,
                              out=out, S_final=S, dev_status=status)
        assert status.item() == 1, change
        rest = torch.ones(T, dtype=torch.bool, device="cuda")
        for i in ok:
            rest[bad[i]:bad[i + 1]] = False
        assert torch.all(out[rest] == 7.0), change
        for i in range(N):
            if i not in ok:
                assert torch.all(S[i] == 7.0), (change, i)
        for i in ok[:6]:
            check(out, S, args, opts, bad, i, dtype, S0, chunks=dtype == "bf16")


@pytest.mark.parametrize("way", ["sorted", "segments", "segments on CUDA cores"])
def test_bounds_that_change_between_replays(cuda_device, way):
    """A packed call captured once, replayed with other bounds and inputs (as many tokens and documents): the bits of
    a plain call each time."""
    lens, cu, dev, args, opts, S0, dtype = make(way)
    longest = max(lens)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = lambda a, c: R.rapt_ssm_varlen_fwd(**a, **opts, cu_seqlens=c, max_seqlen=longest, S0=S0, final_state=True,
                                              dev_status=status)
    mine, bounds = {k: v.clone() for k, v in args.items()}, dev.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, S = call(mine, bounds)
    for turn in range(4):
        other = list(np.roll(lens, 3 * turn + 1))
        bounds.copy_(torch.from_numpy(np.concatenate([[0], np.cumsum(other)]).astype(np.int32)))
        for k in ("x", "dt", "B", "C"):
            mine[k].copy_(scan_inputs(20 + turn, (int(cu[-1]),), *WAYS[way][1], dtype)[0][k])
        g.replay()
        bounds2 = bounds.clone()
        want = call({k: v.clone() for k, v in mine.items()}, bounds2)
        assert torch.equal(out, want[0]) and torch.equal(S, want[1])
    assert status.item() == 0


@pytest.mark.parametrize("dtype,shape", [("bf16", (2, 64, 1, 128)), ("bf16", (1, 128, 1, 64)), ("f32", (2, 16, 2, 16))])
def test_a_prompt_in_pieces(cuda_device, dtype, shape):
    """A prompt cut into segments, and the same tokens in calls that each begin with the state before: both within
    the budget of the oracle."""
    H, P, G, N = shape
    L = 3000
    args, opts = scan_inputs(12, (1, L), H, P, G, N, dtype)
    S = S0 = state(13, 1, H, N, P)
    whole, last = R.rapt_ssm_prefill_fwd(**args, **opts, S0=S0, final_state=True)
    outs = []
    for a, b in ((0, 1), (1, 700), (700, 828), (828, 2999), (2999, L)):
        piece = {k: v if k == "A" else v[:, a:b] for k, v in args.items()}
        rest = {k: v[:, a:b] if k == "z" else v for k, v in opts.items()}
        out, S = R.rapt_ssm_prefill_fwd(**piece, **rest, S0=S, final_state=True)
        outs.append(out)
    flat = lambda d: {k: v[0] if k in ("x", "dt", "B", "C", "z") else v for k, v in d.items()}
    chunks = dtype == "bf16" and P >= 64
    for out, Sf in ((whole, last), (torch.cat(outs, 1), S)):
        check(out[0], Sf, flat(args), flat(opts), [0, L], 0, dtype, S0, chunks=chunks)


@pytest.mark.parametrize("lens", [[3] * 700 + [2000] + [1, 0, 129] * 150, [7] * 1024 + [1200]])
@pytest.mark.parametrize("shape", [(1, 64, 1, 64), (8, 64, 4, 64), (2, 128, 2, 128)])
def test_many_documents(cuda_device, lens, shape):
    """More documents than are sorted, one of them long."""
    H, P, G, N = shape
    cu, dev = pack(lens)
    T = int(cu[-1])
    args, opts = scan_inputs(5, (T,), H, P, G, N, "bf16")
    assert plan_bytes(args, T, len(lens), max(lens)) <= H * (T // 128) * (N * P + 4) * 4
    S0 = state(6, len(lens), H, N, P)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, S = R.rapt_ssm_varlen_fwd(**args, **opts, cu_seqlens=dev, max_seqlen=max(lens), S0=S0, final_state=True,
                                   dev_status=status)
    assert status.item() == 0
    for i in (0, 1, 699, 700, 701, 703, 704, len(lens) - 2, len(lens) - 1):
        check(out, S, args, opts, cu, i, "bf16", S0)
    whole = R.rapt_ssm_varlen_fwd(**args, **opts, cu_seqlens=dev, max_seqlen=T, S0=S0, final_state=True)
    for i in (0, 700, len(lens) - 1):  # a looser bound on the lengths, another plan
        check(*whole, args, opts, cu, i, "bf16", S0)


@pytest.mark.parametrize("shape,dtype", [((2, 64, 1, 64), "bf16"), ((2, 32, 1, 16), "f32")])
def test_short_documents_in_a_plan_of_segments(cuda_device, shape, dtype):
    """A bound on the lengths far above them: segments that no document has; bounds and workspace are overwritten right
    behind the call."""
    H, P, G, N = shape
    lens = [60, 64, 0, 17, 1, 50] * 4
    cu, dev = pack(lens)
    args, opts = scan_inputs(15, (int(cu[-1]),), H, P, G, N, dtype)
    need = plan_bytes(args, int(cu[-1]), len(lens), 1 << 20)
    S0 = state(16, len(lens), H, N, P)
    want = None
    for _ in range(20):
        c, ws = dev.clone(), torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        out, S = R.rapt_ssm_varlen_fwd(**args, **opts, cu_seqlens=c, max_seqlen=1 << 20, S0=S0, final_state=True,
                                       workspace=ws)
        c.zero_()
        ws.zero_()
        want = want or (out, S)
        assert torch.equal(out, want[0]) and torch.equal(S, want[1]) and not ws.any()
    for i in range(len(lens)):
        check(out, S, args, opts, cu, i, dtype, S0, chunks=dtype == "bf16")


@pytest.mark.parametrize("shape,dtype", [((2, 64, 1, 64), "bf16"), ((8, 64, 4, 128), "bf16"), ((2, 32, 1, 16), "f32")])
@pytest.mark.parametrize("longest", [0, 1 << 20])
def test_documents_without_a_token(cuda_device, shape, dtype, longest):
    """T = 0: the final states are the ones before, or zeros; bounds that are not all 0 are reported."""
    H, P, G, N = shape
    args, opts = scan_inputs(17, (0,), H, P, G, N, dtype, sliced=False)
    S0 = state(18, 50, H, N, P)
    cu = torch.zeros(51, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = lambda **kw: R.rapt_ssm_varlen_fwd(**args, **opts, cu_seqlens=cu, max_seqlen=longest, final_state=True,
                                              dev_status=status, **kw)
    out, S = call(S0=S0)
    assert out.shape == (0, H, P) and torch.equal(S, S0)
    assert torch.equal(call()[1], torch.zeros_like(S0)) and status.item() == 0
    cu[7] = 1
    call(S0=S0)
    assert status.item() == 1


@pytest.mark.parametrize("dtype,shape", [("bf16", (2, 64, 1, 64)), ("f32", (2, 32, 1, 16))])
def test_tokens_that_change_nothing(cuda_device, dtype, shape):
    """Padding with a raw step of -infinity at the end of the rows of a batch: the final states are those of the rows
    without it, and the outputs before it their bits."""
    H, P, G, N = shape
    args, opts = scan_inputs(19, (3, 300), H, P, G, N, dtype, sliced=False)
    ends = (300, 131, 1)
    for b, n in enumerate(ends):
        args["dt"][b, n:] = float("-inf")
    S0 = state(20, 3, H, N, P)
    out, S = R.rapt_ssm_prefill_fwd(**args, **opts, S0=S0, final_state=True)
    for b, n in enumerate(ends):
        flat = lambda d: {k: v[b] if k in ("x", "dt", "B", "C", "z") else v for k, v in d.items()}
        check(out[b], S[b:b + 1], flat(args), flat(opts), [0, n], 0, dtype, S0[b:b + 1], chunks=dtype == "bf16")
