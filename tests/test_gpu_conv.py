"""The short causal convolution on the GPU against the fp64 oracle."""

import numpy as np
import pytest
import torch

import ssm_bounds as SB
from block_bounds import within
from relu_linear_attention_gb300 import binding as R
from ssm_inputs import DT, host

pytestmark = pytest.mark.gpu
ACTS = ("none", "silu", "gelu", "relu", "sigmoid")


def inputs(seed, rows, D, W, dtype, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")
    x = n(*rows, D + 2 * pad).to(DT[dtype])[..., pad:pad + D]
    return x, n(D, W) * 0.7, n(D) * 0.3


def check(got, last, x, w, b, act, state, dtype, what):
    y, tail, e = SB.conv(dtype, host(x), host(w), host(b), act, host(state))
    within(host(got), y, e + 1e-30, what)
    if last is not None:
        np.testing.assert_array_equal(host(last), tail, err_msg=what)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("D,pad", [(8, 0), (64, 16), (1, 0), (7, 0), (130, 0), (1032, 8), (200, 1)])
def test_dense(cuda_device, dtype, W, D, pad):
    if pad == 1:
        x, w, b = inputs(1, (2, 9), D, W, dtype, pad)
        with pytest.raises(R._lib.RaptError):  # a slice that begins inside 16 bytes
            R.rapt_conv_prefill_fwd(x, w, b)
        return
    for L in (1, 2, 3, 31, 32, 33, 100):
        x, w, b = inputs(L, (3, L), D, W, dtype, pad)
        state = inputs(L + 50, (3, W - 1), D, W, dtype)[0].contiguous()
        for st, bias in ((None, b), (state, None)):
            out, last = R.rapt_conv_prefill_fwd(x, w, bias, state=st, final_state=True)
            for i in range(3):
                check(out[i], last[i], x[i], w, bias, "silu", None if st is None else st[i], dtype, "L %d" % L)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ACTS)
def test_activations(cuda_device, dtype, act):
    for D in (40, 41):
        x, w, b = inputs(3, (1, 50), D, 4, dtype)
        out, last = R.rapt_conv_prefill_fwd(x, w, b, act=act)
        assert last is None
        check(out[0], None, x[0], w, b, act, None, dtype, act)


@pytest.mark.parametrize("dtype,D", [("bf16", 72), ("bf16", 71), ("f32", 36), ("f32", 5)])
@pytest.mark.parametrize("W", [2, 4])
def test_packed(cuda_device, dtype, D, W):
    """Documents shorter than the window, empty ones, several ends in one tile, a tile that begins at an end."""
    lens = [0, 1, 2, 1, 0, 0, 28, 3, 61, 0, 1, 1, 1, 40, 0]
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    x, w, b = inputs(5, (int(cu[-1]),), D, W, dtype)
    state = inputs(6, (len(lens), W - 1), D, W, dtype)[0]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for st in (None, state):
        out, last = R.rapt_conv_varlen_fwd(x, torch.from_numpy(cu).cuda(), w, b, state=st, final_state=True,
                                           dev_status=status)
        for i in range(len(lens)):
            check(out[cu[i]:cu[i + 1]], last[i], x[cu[i]:cu[i + 1]], w, b, "silu", None if st is None else st[i],
                  dtype, "document %d" % i)
    assert status.item() == 0


def test_malformed_documents_are_reported(cuda_device):
    x, w, b = inputs(7, (64,), 16, 4, "bf16")
    for cu in ([0, 20, 10, 64], [0, 30, 60, 63], [5, 30, 60, 64], [0, 90, 60, 64], [0, -7, 60, 64]):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, _ = R.rapt_conv_varlen_fwd(x, torch.tensor(cu, dtype=torch.int32, device="cuda"), w, b, final_state=True,
                                        dev_status=status)
        assert status.item() == 1, cu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 65, 1])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_single_tokens_continue_a_prompt(cuda_device, dtype, D, W):
    """Token by token on the state that a prompt leaves: the bits of the whole prompt."""
    x, w, b = inputs(8, (5, 20), D, W, dtype)
    whole, last = R.rapt_conv_prefill_fwd(x, w, b, final_state=True)
    out, state = R.rapt_conv_prefill_fwd(x[:, :13].contiguous(), w, b, final_state=True)
    outs = [out]
    for t in range(13, 20):
        outs.append(R.rapt_conv_decode_step(x[:, t].contiguous(), state, w, b)[:, None])
    assert torch.equal(torch.cat(outs, 1), whole) and torch.equal(state, last)
    if D % 8 == 0:  # a column slice of wider rows
        wide = torch.cat((x[:, 0], x[:, 1], x[:, 0]), 1)
        s1, s2 = state.clone(), state.clone()
        assert torch.equal(R.rapt_conv_decode_step(wide[:, D:2 * D], s1, w, b),
                           R.rapt_conv_decode_step(x[:, 1].contiguous(), s2, w, b)) and torch.equal(s1, s2)


def test_not_finite_stays_in_its_channel_and_window(cuda_device):
    x, w, b = inputs(9, (1, 40), 16, 4, "f32")
    clean = R.rapt_conv_prefill_fwd(x, w, b)[0]
    x[0, 10, 3] = float("nan")
    x[0, 20, 5] = float("inf")
    out = R.rapt_conv_prefill_fwd(x, w, b)[0]
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[0, 10:14, 3] = True
    hit[0, 20:24, 5] = True
    assert torch.equal(out[~hit], clean[~hit]) and torch.isnan(out[0, 10:14, 3]).all()


def test_no_tokens_and_streams(cuda_device):
    x, w, b = inputs(10, (2, 0), 16, 4, "bf16")
    state = torch.randn(2, 3, 16, device="cuda").bfloat16()
    out, last = R.rapt_conv_prefill_fwd(x, w, b, state=state, final_state=True)
    assert out.shape == (2, 0, 16) and torch.equal(last, state)
    x, w, b = inputs(11, (2, 100), 16, 4, "bf16")
    want = R.rapt_conv_prefill_fwd(x, w, b)[0]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = R.rapt_conv_prefill_fwd(x, w, b, stream=s)[0]
    s.synchronize()
    assert torch.equal(got, want)
