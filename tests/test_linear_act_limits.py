"""The linear with its epilogue at the ends of its ranges: calls that enqueue nothing
or that the library refuses on the host (fake device addresses, so only where no
GPU is visible)."""
import ctypes

import pytest
import torch

from float8_mixed_precision_amd import ops as E

A = 0x10000
P = lambda v: ctypes.c_void_p(v) if v else None
no_gpu = pytest.mark.skipif(torch.cuda.device_count() != 0,
                            reason="fake-pointer cases run without a GPU only")


@no_gpu
@pytest.mark.parametrize("act", [E.FP8L_ACT_NONE, E.FP8L_ACT_GELU])
@pytest.mark.parametrize("q,scale,amax", [(A, A, A), (A, None, None), (None, A, None),
                                          (None, None, A)])
@pytest.mark.parametrize("y,z", [(A, A), (A, None), (None, A), (None, None)])
def test_codes_of_no_rows(y, z, q, scale, amax, act):
    """M = 0 tokens with the outputs of the serving form in hand (qt and scale_t absent):
    there is nothing to write and nothing is enqueued."""
    for N, K in ((32, 48), (0, 48), (32, 0), (8208, 4112)):
        at = iter(range(A, 1 << 40, 1 << 28))
        new = lambda v: P(next(at)) if v else None
        ok = E.lib().fp8_linear_act_fwd(
            new(A), new(A), new(A), new(A), 0, N, K, E.FP8L_ROWWISE, new(A), E.FP8L_BF16, act,
            None, new(z), new(y), new(q), None, new(scale), None, new(amax), new(A), 1 << 27, None)
        assert ok == E.FP8L_OK, (N, K)
