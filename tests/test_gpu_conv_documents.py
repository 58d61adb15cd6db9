"""The convolution's look at a call's documents: as many as it allows, and bounds that are malformed."""

import pytest
import torch

from relu_linear_attention_gb300 import _lib, binding as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("stride", [16384, 16385])
def test_as_many_documents_as_are_allowed(cuda_device, stride):
    """2^38 documents' channels without states: the bounds are looked at once a document."""
    N, D, W = 1 << 24, 1 << 14, 2
    cu = torch.zeros(N + 1, dtype=torch.int32, device="cuda")
    cu[-1] = 1
    x, w = torch.randn(1, stride, device="cuda"), torch.randn(D, W, device="cuda")
    for bad in (False, True):
        if bad:
            cu[N // 2] = 5
        out, status = torch.zeros(1, D, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        st = _lib.load().rapt_conv_varlen_fwd(x.data_ptr(), stride, _lib.RAPT_F32, 1, D, cu.data_ptr(), N, w.data_ptr(),
                                              None, W, 0, None, out.data_ptr(), None, status.data_ptr(), None)
        assert st == _lib.RAPT_OK and status.item() == bad
        if not bad:
            assert torch.equal(out, x[:, :D] * w[:, 1])


@pytest.mark.parametrize("dtype,D", [(torch.bfloat16, 16), (torch.float32, 7)])
def test_malformed_documents_touch_nothing_else(cuda_device, dtype, D):
    """Whatever the bounds: reported, the final states of documents that are good by themselves are right, those of
    the others keep what was there, and so does what lies around the outputs."""
    T, N, W = 64, 3, 4
    x, w = torch.randn(T, D, device="cuda").to(dtype), torch.randn(D, W, device="cuda")
    for cu in ([0, 20, 10, 64], [0, 30, 60, 63], [5, 30, 60, 64], [0, 90, 60, 64], [0, -7, 60, 64], [64, 0, 0, 64],
               [-(1 << 31), (1 << 31) - 1, 0, 64]):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((T + 128, D), 7.0, dtype=dtype, device="cuda")
        last = torch.full((N + 32, W - 1, D), 7.0, dtype=dtype, device="cuda")
        R.rapt_conv_varlen_fwd(x, torch.tensor(cu, dtype=torch.int32, device="cuda"), w, act="none", out=out[64:64 + T],
                               state_final=last[16:16 + N], dev_status=status)
        assert status.item() == 1, cu
        assert torch.all(out[:64] == 7.0) and torch.all(out[64 + T:] == 7.0), cu
        assert torch.all(last[:16] == 7.0) and torch.all(last[16 + N:] == 7.0), cu
        for i in range(N):
            s, e = cu[i], cu[i + 1]
            good = 0 <= s <= e <= T and (cu[i - 1] <= s if i else s == 0) and (i < N - 1 or e == T)
            want = torch.full((W - 1, D), 7.0, dtype=dtype, device="cuda")
            if good:
                want.zero_()
                n = min(W - 1, e - s)
                if n:
                    want[W - 1 - n:] = x[e - n:e]
            assert torch.equal(last[16 + i], want), (cu, i)


def test_documents_without_a_token(cuda_device):
    x, w = torch.randn(0, 16, device="cuda"), torch.randn(16, 4, device="cuda")
    state, status = torch.randn(50, 3, 16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = torch.zeros(51, dtype=torch.int32, device="cuda")
    out, last = R.rapt_conv_varlen_fwd(x, cu, w, state=state, final_state=True, dev_status=status)
    assert out.shape == (0, 16) and torch.equal(last, state) and status.item() == 0
    assert not R.rapt_conv_varlen_fwd(x, cu, w, final_state=True)[1].any()
    cu[7] = 1
    R.rapt_conv_varlen_fwd(x, cu, w, dev_status=status)
    assert status.item() == 1
