"""The scan's workspace over packed documents, from the C ABI alone: no more than a record of each head's state for
every chunk of 128 tokens, however the tokens are spread over the documents. No GPU is needed."""

import ctypes

import pytest

from relu_linear_attention_gb300 import _lib

# tokens, documents, the longest: many documents with one that is long, few, and as many as tokens
CALLS = [(65536, 1025, 32768), (65536, 2000, 60000), (65536, 100, 60000), (65536, 1000, 60000), (65536, 2, 65535),
         (65536, 65536, 1), (65536, 65536, 65536), (1 << 20, 3000, 1 << 19), (300, 4, 297), (1, 1, 1), (0, 5, 0)]


@pytest.mark.parametrize("T,N,longest", CALLS)
@pytest.mark.parametrize("H,P,G,Ns", [(64, 64, 1, 128), (32, 64, 1, 64), (16, 128, 8, 128), (1, 64, 1, 64), (3, 64, 1, 64)])
@pytest.mark.parametrize("dtype", [_lib.RAPT_BF16, _lib.RAPT_F32])
def test_packed_workspace_goes_by_tokens(lib, T, N, longest, H, P, G, Ns, dtype):
    a = _lib.rapt_ssm_inputs(H=H, P=P, G=G, Ns=Ns, dt_softplus=1, dtype=dtype)
    need = lib.rapt_ssm_varlen_workspace_size(ctypes.byref(a), T, N, longest)
    # (fp32 on the CUDA cores: segments of 64 tokens and more)
    each = 128 if dtype == _lib.RAPT_BF16 else 64
    assert need <= max(4 * min(N, 1024), H * (T // each) * (Ns * P + 4) * 4)
    # a looser bound on the lengths needs no more than that either
    need = lib.rapt_ssm_varlen_workspace_size(ctypes.byref(a), T, N, 1 << 30)
    assert need <= max(4 * min(N, 1024), H * (T // each) * (Ns * P + 4) * 4)
