"""Sizes beyond 32 bits at the C boundary: no int32_t argument of any function may lose its upper bits on
the way, whatever the low ones say. Every call here ends on the host, before any CUDA work."""

import ctypes

import pytest

from relu_linear_attention_gb300 import _lib

P = [ctypes.c_void_p(0x7F0000000000 + 0x1000 * i) for i in range(1, 17)]  # aligned, never dereferenced
ARGS = _lib.rapt_params(1e-6, 1e4, 1e-4, 0)
HUGE = 1 << 40  # bytes of a workspace that is large enough

# name -> arguments that the function accepts, but for "rows": a count of rows, queries or sequences of
# which 0 asks for nothing (so that 2^32 with its upper bits lost asks for nothing, too) and the others.
# Every int in the list is an int32_t but the last-but-one size of a workspace.
FN = {
    "rapt_residual_norm_fwd": [P[0], P[1], P[2], 1, 0, 64, 4, P[3], P[4], P[5], 1e-6, P[6], P[7], None],
    "rapt_glu_fwd": [P[0], P[1], P[2], 0, 64, 64, 1, P[3], None, None],
    "rapt_prefill_fwd": [P[0], P[1], P[2], 1, 1, 0, 2, 64, P[3], P[4], ARGS, 0, None, None, P[5], None, None, None,
                         P[6], HUGE, None],
    "rapt_bidir_fwd": [P[0], P[1], P[2], 1, 1, 0, 2, 64, P[3], P[4], ARGS, 0, P[5], None, P[6], HUGE, None],
    "rla_l2_fwd": [P[0], P[1], P[2], 1, 1, 0, 2, 128, 1e-6, P[3], P[4], HUGE, None],
    "rla_l2_readout": [P[0], P[1], 1, 1, 0, 2, 128, 1e-6, P[2], P[3], HUGE, None],
}
CASES = [(fn, i) for fn, a in FN.items() for i, v in enumerate(a) if isinstance(v, int) and v != HUGE]


@pytest.mark.parametrize("fn,i", CASES)
@pytest.mark.parametrize("lost", [1 << 32, -(1 << 32), 1 << 40])
def test_a_size_past_32_bits_is_refused(lib, fn, i, lost):
    assert getattr(lib, fn)(*FN[fn]) == _lib.RAPT_OK
    a = list(FN[fn])
    a[i] += lost
    assert getattr(lib, fn)(*a) in (_lib.RAPT_ERR_INVALID_ARG, _lib.RAPT_ERR_UNSUPPORTED)


def test_the_least_size_past_32_bits_is_refused(lib):
    for M in (1 << 31, (1 << 32) - 1, -(1 << 31) - 1):
        a = list(FN["rapt_glu_fwd"])
        a[3] = M
        assert lib.rapt_glu_fwd(*a) == _lib.RAPT_ERR_INVALID_ARG


@pytest.mark.parametrize("name,sizes", [
    ("rapt_residual_norm_bwd_workspace_size", [4, 64, 1]), ("rapt_glu_bwd_workspace_size", [4, 64, 64]),
    ("rapt_linear_bwd_workspace_size", [65521, 512, 520]), ("rapt_prefill_workspace_size", [4, 4096, 16, 128, 1]),
    ("rapt_prefill_bwd_workspace_size", [4, 4096, 16, 128, 1]), ("rla_l2_workspace_size", [2, 16384, 16, 128, 1]),
    ("rapt_layer_workspace_size", [4, 4096, 16, 128, 2048]),
])
def test_workspace_queries_of_sizes_past_32_bits(lib, name, sizes):
    query = getattr(lib, name)
    assert query(*sizes) > 0
    for i in range(len(sizes)):
        assert query(*[v + ((1 << 32) if i == j else 0) for j, v in enumerate(sizes)]) == 0


def test_what_is_no_int_is_no_size(lib):
    for v in (4.0, "4", None):
        with pytest.raises(ctypes.ArgumentError):
            lib.rapt_glu_bwd_workspace_size(v, 64, 64)
