"""Elements more than 2^31 from a tensor's start: the same bits as from small contiguous copies of the same rows."""

import pytest
import torch

from relu_linear_attention_gb300 import binding as R

pytestmark = pytest.mark.gpu
FAR = 1 << 31


def _far_rows(rows, width, dtype):
    """[rows, width] at a stride that puts the last rows more than 2^31 elements from the first."""
    stride = (FAR // (rows - 8) + 63) // 64 * 64
    x = torch.empty((rows - 1) * stride + width, dtype=dtype, device="cuda").as_strided((rows, width), (stride, 1))
    x.copy_(torch.randn(rows, width, device="cuda"))
    return x


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_convolution_and_scan_of_far_rows(cuda_device, dtype):
    torch.manual_seed(1)
    L, H, P, N = 600, 2, 64, 64
    x = _far_rows(L, H * P, dtype)
    near = x.contiguous()
    w, b = torch.randn(H * P, 4, device="cuda"), torch.randn(H * P, device="cuda")
    got, tail = R.rapt_conv_prefill_fwd(x[None], w, b, final_state=True)
    want, tail2 = R.rapt_conv_prefill_fwd(near[None], w, b, final_state=True)
    assert torch.equal(got, want) and torch.equal(tail, tail2)
    cu = torch.tensor([0, 250, L], dtype=torch.int32, device="cuda")
    assert torch.equal(R.rapt_conv_varlen_fwd(x, cu, w, b)[0], R.rapt_conv_varlen_fwd(near, cu, w, b)[0])
    dt, A = torch.randn(1, L, H, device="cuda").to(dtype), -torch.rand(H, device="cuda") - 0.1
    bc = torch.randn(1, L, 1, N, device="cuda").to(dtype)
    z = torch.randn(1, L, H, P, device="cuda").to(dtype)
    outs = []
    for v in (x, near):
        v = v.unflatten(-1, (H, P))
        # the far rows as the scan's x, as its gate and, cut to a group's columns, as B and C
        outs.append(R.rapt_ssm_prefill_fwd(v[None], dt, A, bc, bc, z=z, final_state=True)
                    + R.rapt_ssm_prefill_fwd(z, dt, A, v[None, :, :1], v[None, :, 1:], z=v[None], final_state=True)
                    + R.rapt_ssm_varlen_fwd(v, dt[0], A, bc[0], bc[0], cu, max_seqlen=350, final_state=True))
    assert all(torch.equal(p, q) for p, q in zip(*outs))


def test_steps_of_states_past_32_bits(cuda_device):
    torch.manual_seed(2)
    H, P, N = 16, 64, 128
    n = FAR // (H * N * P) + 44
    S = torch.empty(n, H, N, P, device="cuda").normal_()
    x, dt = torch.randn(n, H, P, device="cuda").bfloat16(), torch.randn(n, H, device="cuda").bfloat16()
    bc, A = torch.randn(n, 1, N, device="cuda").bfloat16(), -torch.rand(H, device="cuda")
    last = S[-40:].clone()  # (640 heads: as many to a CTA as all of them)
    out = R.rapt_ssm_decode_step(x, dt, A, bc, bc, S)
    want = R.rapt_ssm_decode_step(x[-40:], dt[-40:], A, bc[-40:], bc[-40:], last)
    assert torch.equal(out[-40:], want) and torch.equal(S[-40:], last)


def test_layer_norm_past_32_bits(cuda_device):
    torch.manual_seed(3)
    D = 16384
    T = FAR // D + 40
    x = torch.empty(T, D, dtype=torch.bfloat16, device="cuda").normal_()
    w, b = torch.randn(D, device="cuda"), torch.randn(D, device="cuda")
    y = R.rapt_layer_norm_fwd(x, w, b)
    assert torch.equal(y[-37:], R.rapt_layer_norm_fwd(x[-37:].clone(), w, b))
    dx = R.rapt_layer_norm_bwd(y, x, w, need_dw=False, need_db=False)[0]
    assert torch.equal(dx[-37:], R.rapt_layer_norm_bwd(y[-37:].clone(), x[-37:].clone(), w, need_dw=False,
                                                       need_db=False)[0])
