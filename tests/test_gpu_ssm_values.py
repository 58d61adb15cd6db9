"""The selective scan at the ends of its inputs' range, and with values that are not finite: the gate, the step
sizes and decays, and tokens that belong to others. Prompts (on the tensor cores and on the CUDA cores) and single
tokens, against the fp64 oracle or against the bits of the same call without such values."""

import numpy as np
import pytest
import torch

import ssm_bounds as SB
from block_bounds import within
from relu_linear_attention_gb300 import binding as R
from ssm_inputs import document, host, scan_inputs, state

pytestmark = pytest.mark.gpu

# tensor cores: pairs of heads, a head alone, heads of 128; CUDA cores
FORMS = [("bf16", (2, 64, 1, 64)), ("bf16", (3, 64, 1, 128)), ("bf16", (2, 128, 1, 64)), ("bf16", (2, 32, 1, 16)),
         ("f32", (2, 64, 1, 64))]


def _pack(lens):
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    return cu, torch.from_numpy(cu).cuda()


@pytest.mark.parametrize("dtype,shape", FORMS)
def test_gate_at_the_ends_of_its_range(cuda_device, dtype, shape):
    """z silu far out: closed (a mask of the type's lowest value) or open, in prompts and single tokens alike."""
    H, P, G, N = shape
    args, opts = scan_inputs(1, (1, 140), H, P, G, N, dtype)
    lowest = torch.finfo(args["x"].dtype).min
    far = torch.tensor([lowest, -1e30, -200.0, -90.0, 90.0, 200.0, 1e30], device="cuda")
    z = opts["z"] = far[torch.arange(140 * H * P, device="cuda") % 7].view(1, 140, H, P).to(args["x"].dtype)
    args["x"] = args["x"].contiguous() * 16  # outputs well above 1
    out = R.rapt_ssm_prefill_fwd(**args, **opts)[0]
    chunks = dtype == "bf16" and P >= 64
    with np.errstate(over="ignore"):
        ref, _, eo, _ = SB.scan(dtype, **document(args, opts, 0), chunks=chunks)
        within(host(out[0]), ref, eo + 1e-30, "prompt")
        assert torch.equal(out[z == lowest], torch.zeros_like(out[z == lowest]))
        # an open gate is its own value: z times what a call without a gate gives, four roundings of the type
        wide = z == z.max()
        plain = (R.rapt_ssm_prefill_fwd(**args, **{**opts, "z": None})[0].double() * z.double())[wide]
        assert plain.abs().max() > 1e30
        assert ((out[wide].double() - plain).abs() <= 2 * torch.finfo(out.dtype).eps * plain.abs()).all()
        S = torch.zeros(140, H, N, P, device="cuda")
        one = {k: v if k == "A" else v[0] for k, v in args.items()}
        tok = {k: v[0] if k == "z" else v for k, v in opts.items()}
        out = R.rapt_ssm_decode_step(**one, **tok, S=S)
        for i in (0, 77, 139):
            ref, _, eo, _ = SB.scan(dtype, **document(one, tok, slice(i, i + 1)))
            within(host(out[i:i + 1]), ref, eo + 1e-30, "token %d" % i)


@pytest.mark.parametrize("dtype,shape", FORMS)
@pytest.mark.parametrize("what", ["x", "B", "C", "dt", "z"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_not_finite_stays_in_its_document(cuda_device, dtype, shape, what, value):
    """Documents that end inside a chunk, the next one's first tokens not finite: the bits of the others are those of
    the call without them, outputs and final states. Packed, and rows of a batch."""
    H, P, G, N = shape
    lens = [5, 130, 1, 127, 128, 300, 17, 33]
    cu, dev = _pack(lens)
    args, opts = scan_inputs(2, (int(cu[-1]),), H, P, G, N, dtype, sliced=False)
    S0 = state(3, len(lens), H, N, P)
    call = lambda: R.rapt_ssm_varlen_fwd(**args, **opts, cu_seqlens=dev, max_seqlen=300, S0=S0, final_state=True)
    out, S = call()
    t = args.get(what, opts.get(what))
    for bad in (1, 3, 5, 7):
        t[cu[bad]:cu[bad] + 3] = value
    out2, S2 = call()
    for i, n in enumerate(lens):
        same, same_S = torch.equal(out[cu[i]:cu[i + 1]], out2[cu[i]:cu[i + 1]]), torch.equal(S[i], S2[i])
        assert (same, same_S) == ((True, True) if i % 2 == 0 else (False, what in ("C", "z"))), i
    args, opts = scan_inputs(4, (3, 150), H, P, G, N, dtype, sliced=False)
    S0 = state(5, 3, H, N, P)
    call = lambda: R.rapt_ssm_prefill_fwd(**args, **opts, S0=S0, final_state=True)
    out, S = call()
    args.get(what, opts.get(what))[1, :100] = value
    out2, S2 = call()
    assert all(torch.equal(out[b], out2[b]) and torch.equal(S[b], S2[b]) for b in (0, 2))
    assert not torch.isfinite(out2[1].float()).all()


@pytest.mark.parametrize("dtype,shape", FORMS)
@pytest.mark.parametrize("what", ["B", "C", "dt", "z"])
def test_not_finite_reaches_no_token_before_it(cuda_device, dtype, shape, what):
    H, P, G, N = shape
    args, opts = scan_inputs(6, (1, 300), H, P, G, N, dtype, sliced=False)
    out = R.rapt_ssm_prefill_fwd(**args, **opts)[0]
    args.get(what, opts.get(what))[0, 200] = float("nan")
    out2 = R.rapt_ssm_prefill_fwd(**args, **opts)[0]
    assert torch.equal(out[0, :200], out2[0, :200]) and torch.isnan(out2[0, 200]).all()
    later = torch.isnan(out2[0, 201:])
    assert not later.any() if what in ("C", "z") else later.all()


@pytest.mark.parametrize("dtype,shape", FORMS)
def test_a_decay_that_forgets_everything(cuda_device, dtype, shape):
    """A = -infinity: every state is its last token's; a document's end inside a chunk changes nothing."""
    H, P, G, N = shape
    lens = [150, 128, 1, 37]
    cu, dev = _pack(lens)
    args, opts = scan_inputs(9, (int(cu[-1]),), H, P, G, N, dtype)
    args["A"][0] = float("-inf")
    S0 = state(10, len(lens), H, N, P)
    out, S = R.rapt_ssm_varlen_fwd(**args, **opts, cu_seqlens=dev, max_seqlen=150, S0=S0, final_state=True)
    for i in range(len(lens)):
        at = slice(cu[i], cu[i + 1])
        k = document(args, opts, at)
        k["A"] = np.maximum(k["A"], -1e6)
        ref, refS, eo, eS = SB.scan(dtype, **k, S0=host(S0[i]), chunks=dtype == "bf16" and P >= 64)
        within(host(out[at]), ref, eo + 1e-30, "document %d out" % i)
        within(host(S[i]), refS, eS + 1e-30, "document %d S" % i)


@pytest.mark.parametrize("dtype,shape", FORMS)
def test_a_parameter_that_is_no_number_shows(cuda_device, dtype, shape):
    """NaN in A: its head's outputs and state are NaN, the others keep their bits; prompts and single tokens."""
    H, P, G, N = shape
    args, opts = scan_inputs(7, (1, 150), H, P, G, N, dtype)
    S0 = state(8, 1, H, N, P)
    res = []
    for bad in (False, True):
        if bad:
            args["A"][1] = float("nan")
        one = {k: v if k == "A" else v[:, 0] for k, v in args.items()}
        tok = {k: v[:, 0] if k == "z" else v for k, v in opts.items()}
        out, Sf = R.rapt_ssm_prefill_fwd(**args, **opts, S0=S0, final_state=True)
        S = S0.clone()
        y = R.rapt_ssm_decode_step(**one, **tok, S=S)
        res.append([v.movedim(d, 0) for v, d in ((out, 2), (Sf, 1), (y, 1), (S, 1))])
    for clean, got in zip(*res):
        assert torch.isnan(got[1]).all()
        assert all(torch.equal(got[h], clean[h]) for h in range(H) if h != 1)


@pytest.mark.parametrize("dtype,shape", FORMS)
@pytest.mark.parametrize("decay", [(1.0, 16.0), (200.0, 4000.0)])
def test_large_values(cuda_device, dtype, shape, decay):
    """Scores and outputs of up to some 2^60 with decays below 2^-64: inside the range that the header gives."""
    H, P, G, N = shape
    args, opts = scan_inputs(11, (1, 300), H, P, G, N, dtype, z=False, decay=decay)
    args["x"], args["B"], args["C"] = (args[k].contiguous() * 2.0 ** e for k, e in (("x", 22), ("B", 16), ("C", 16)))
    S0 = state(12, 1, H, N, P) * 2.0 ** 30
    out, S = R.rapt_ssm_prefill_fwd(**args, **opts, S0=S0, final_state=True)
    ref, refS, eo, eS = SB.scan(dtype, **document(args, opts, 0), S0=host(S0[0]), chunks=dtype == "bf16" and P >= 64)
    assert 2.0 ** 52 < np.abs(ref).max() < 2.0 ** 62
    within(host(out[0]), ref, eo + 1e-30, "out")
    within(host(S[0]), refS, eS + 1e-30, "S")
