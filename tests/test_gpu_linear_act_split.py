"""GPU linear with its epilogue where the contraction is split over workgroups: a
second kernel adds the parts' fp32 sums and finishes the output, and the maxima of
what is quantized come from a pass of their own.

Parts are added in another order than the plain GEMM's: p is within the
instruction's accumulation bound (tests/mfma_model.py), K sequential additions and
at most 64 more, one for each part, of the exact product; what follows is checked
as in test_gpu_linear_act.py."""
import numpy as np
import pytest
import torch

import oracle
from float8_mixed_precision_amd import ops
from tests import gpu_util as G
from tests import mfma_model as MM
from tests.test_gpu_linear_act import (BF, F32, RW, SIZE_ID, U, _bias, _bits, _hq, _residual,
                                       _value, _w, _x, check_y)

pytestmark = pytest.mark.gpu

# (4 parts; 8 of which the last has 2 k-tiles; 8 of a few tokens; 2; 4 of ragged tiles)
SIZES = [(64, 256, 4096), (32, 256, 8208), (16, 512, 8192), (128, 144, 1040), (48, 528, 2064)]


@RW
@pytest.mark.parametrize("mnk", SIZES, ids=SIZE_ID)
def test_split_contraction_with_codes(mnk, rowwise):
    M, N, K = mnk
    xq, sx = _x(M, K, rowwise, 101)
    wq, sw = _w(N, K, rowwise, 102)
    bias, res = _bias(N, F32 if N % 32 else BF, 103), _residual(M, N, 104)
    A, B = G.host(xq), G.host(wq)
    ii, jj = np.divmod(np.arange(M * N), N)
    val = np.nan_to_num(oracle.e4m3_values())
    sa = np.broadcast_to(1 / G.host(sx).astype(np.float64), (M,))[:, None]
    sb = np.broadcast_to(1 / G.host(sw).astype(np.float64), (N,))[None, :]
    p = (val[A] @ val[B].T) * sa * sb
    D = MM.sum_difference_bound(A, B, ii, jj).reshape(M, N)
    D = D + (K + 64) * U * (np.abs(val)[A] @ np.abs(val)[B].T)
    want = p + _value(bias)
    tol = D * sa * sb * (1 + 2.0 ** -20) + 3 * U * np.abs(p) + U * np.abs(want)
    half = lambda v, t: t + 2.0 ** -8 * (np.abs(v) + t)
    new = lambda: torch.empty((M, N), dtype=BF, device=G.DEV)
    codes = lambda: ops.alloc_quantized(M, N, rowwise, G.DEV)
    # the size that is asked for, and no more
    ws = torch.empty(ops.fp8_linear_act_workspace_bytes(M, N, rowwise), dtype=torch.uint8,
                     device=G.DEV)
    first = None
    for act in ops.ACTS:
        G.say("linear act split", mnk, act, "rowwise", rowwise)
        call = lambda **k: ops.fp8_linear_act_fwd(xq, sx, wq, sw, bias, act, rowwise=rowwise,
                                                  workspace=ws.fill_(0x7F), **k)
        for r in (None, res):
            z, q1, q2, q3 = new(), codes(), codes(), codes()
            y = call(residual=r, z=z, y=new(), out=q1)
            y2 = call(residual=r, out=q2)                    # z not stored
            y3 = call(residual=r)                            # nothing else
            torch.cuda.synchronize()
            label = "%s %s %s" % (mnk, act, r is not None)
            first = z if first is None else first
            assert torch.equal(_bits(z), _bits(first)), label
            assert np.all(np.abs(_value(z) - want) <= half(want, tol)), label
            if act == "none":
                v = want if r is None else want + _value(r)
                t = tol if r is None else tol + U * np.abs(v)
                assert np.all(np.abs(_value(y) - v) <= half(v, t)), label
            else:
                check_y(y, z, act, r, label)
            assert torch.equal(_bits(y), _bits(y2)) and torch.equal(_bits(y), _bits(y3)), label
            ref = oracle.quantize(G.host(y), rowwise)
            G.assert_quantize_equal(_hq(q1), ref, "codes " + label)
            G.assert_quantize_equal(_hq(q2), ref, "codes, z not stored " + label)
            if r is None:
                z2 = new()
                assert call(z=z2, out=q3) is None            # y not stored
                torch.cuda.synchronize()
                assert torch.equal(_bits(z2), _bits(first)), label
                G.assert_quantize_equal(_hq(q3), ref, "codes, y not stored " + label)


def test_split_contraction_in_graphs():
    """Two captured graphs that share the workspace, replayed in turn with eager work
    between, give the eager results."""
    M, N, K = 64, 256, 4096
    xq, sx = _x(M, K, False, 105)
    wq, sw = _w(N, K, False, 106)
    bias = _bias(N, F32, 107)
    ws = ops.alloc_linear_act_workspace(M, N, False, G.DEV)
    z = [torch.empty((M, N), dtype=BF, device=G.DEV) for _ in range(2)]
    q = [ops.alloc_quantized(M, N, False, G.DEV) for _ in range(2)]
    calls = [lambda a=a, k=k: ops.fp8_linear_act_fwd(xq, sx, wq, sw, bias, a, z=z[k], out=q[k],
                                                     workspace=ws)
             for k, a in enumerate(("gelu", "relu2"))]
    G.say("linear act split graphs")

    def results():
        torch.cuda.synchronize()
        return [t.clone() for k in range(2) for t in (z[k], q[k].q, q[k].qt, q[k].scale, q[k].amax)]

    for c in calls:
        c()
    torch.cuda.synchronize()
    graphs = []
    for c in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            c()
    for k in range(3):
        bias.add_(0.25 * k)
        for c in calls:
            c()
        want = results()
        for t in z:
            t.zero_()
        for g in graphs[::-1]:
            g.replay()
        assert all(torch.equal(a, b) for a, b in zip(results(), want)), k
