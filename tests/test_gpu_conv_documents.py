"""The convolution's look at a call's documents: as many as it allows, of no tokens but one."""

import pytest
import torch

from relu_linear_attention_gb300 import _lib

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
