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


@pytest.mark.parametrize("stored", [True, False], ids=["y", "z"])
def test_codes_of_more_rows_than_a_launch_takes(stored):
    """2^22 workgroups of 1024 threads are more than HIP launches together."""
    M, N, K = (1 << 22) + 37, 16, 16
    part = 4096
    xq, sx = _x(part, K, True, 111)
    wq, sw = _w(N, K, True, 112)
    bias = _bias(N, BF, 113)
    roll = lambda t, at: torch.roll(t, at, 0)
    reps = M // part + 1
    xs = torch.cat([roll(xq, k % 7) for k in range(reps)])[:M]
    ss = torch.cat([roll(sx, k % 7) for k in range(reps)])[:M]
    q = torch.full((M + 3, N), 5, dtype=torch.uint8, device=G.DEV)
    scale, amax = (torch.full((M + 3,), 7.0, device=G.DEV) for _ in range(2))
    out = ops.Quantized(q[:M], None, scale[:M], None, amax[:M])
    v = torch.empty((M, N), dtype=BF, device=G.DEV)
    G.say("linear act rows past a launch", M, stored)
    y = ops.fp8_linear_act_fwd(xs, ss, wq, sw, bias, "gelu", None, True, y=v if stored else None,
                               z=None if stored else v, out=out, transposed=False)
    torch.cuda.synchronize()
    assert (y is None) == (not stored)
    assert torch.all(q[M:] == 5) and torch.all(scale[M:] == 7.0) and torch.all(amax[M:] == 7.0)
    for at in (0, (1 << 21) - 100, 1 << 21, (1 << 22) - 100, M - 200):
        rows = slice(at, min(at + 200, M))
        n = rows.stop - at
        z, o = (torch.empty((n, N), dtype=BF, device=G.DEV) for _ in range(2))
        want = ops.Quantized(torch.empty((n, N), dtype=torch.uint8, device=G.DEV), None,
                             torch.empty(n, device=G.DEV), None, torch.empty(n, device=G.DEV))
        ops.fp8_linear_act_fwd(xs[rows].clone(), ss[rows].clone(), wq, sw, bias, "gelu", None, True,
                               y=o, z=z, out=want, transposed=False)
        torch.cuda.synchronize()
        assert torch.equal(_bits(v[rows]), _bits(o if stored else z)), at
        assert torch.equal(q[rows], want.q), at
        assert torch.equal(scale[rows], want.scale) and torch.equal(amax[rows], want.amax), at
    if stored:
        assert torch.equal(amax[:M], v.abs().amax(1).float())
        # (one IEEE division of two 32-bit tensors, as the quantize defines the scale)
        top = torch.full((M,), 448.0, device=G.DEV)
        assert torch.equal(scale[:M], torch.div(top, amax[:M].clamp(min=1e-12)))
