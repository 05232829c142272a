"""GPU linear with its epilogue at the ends of its ranges."""
import ctypes

import pytest
import torch

from float8_mixed_precision_amd import ops
from tests import gpu_util as G
from tests.test_gpu_linear_act import BF, _bias, _bits, _w, _x

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("stored", [True, False], ids=["y", "z"])
def test_codes_of_no_rows(act, stored):
    """M = 0 tokens with the buffers of a larger batch in hand: nothing is written."""
    N, K, R = 4112, 272, 16
    u8 = lambda *s: torch.full(s, 5, dtype=torch.uint8, device=G.DEV)
    f32 = lambda n: torch.full((n,), 7.0, device=G.DEV)
    xq, wq, q = u8(R, K), u8(N, K), u8(R, N)
    sx, sw, scale, amax, bias = f32(R), f32(N), f32(R), f32(R), f32(N)
    y = torch.full((R, N), 7.0, dtype=BF, device=G.DEV)
    ws = ops.alloc_linear_act_workspace(R, N, True, G.DEV)
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    G.say("linear act codes of no rows", act, stored)
    status = ops.lib().fp8_linear_act_fwd(
        p(xq), p(sx), p(wq), p(sw), 0, N, K, ops.FP8L_ROWWISE, p(bias), ops.FP8L_F32,
        ops.ACTS[act], None, None if stored else p(y), p(y) if stored else None, p(q), None,
        p(scale), None, p(amax), p(ws), ws.numel(), None)
    torch.cuda.synchronize()
    assert status == ops.FP8L_OK
    assert torch.all(y == 7.0) and torch.all(q == 5)
    assert torch.all(scale == 7.0) and torch.all(amax == 7.0)
