"""GPU gated feed-forward at the borders between its kernels: batches that
shrink under one workspace, token counts and widths on both sides of each
choice of kernel.  Outputs are compared with the plain GEMM's and with calls of
their own workspace, codes with the oracle's quantize."""
import numpy as np
import pytest
import torch

import oracle
from float8_mixed_precision_amd import ops
from float8_mixed_precision_amd import workloads as W
from tests import gpu_util as G
from tests.test_gpu_gated import RW, RW_IDS, _hq, _weights, _x, check_h

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rowwise", RW, ids=RW_IDS)
def test_one_workspace_for_shrinking_batches(rowwise):
    """The workspace of the largest batch serves the smaller ones (small tiles
    take more partial maxima than large ones), and nothing is written behind it."""
    H, K = 4096, 144
    size = ops.fp8_gated_workspace_bytes(1296, H, rowwise)
    buf = torch.full((size + 4096,), 0x5A, dtype=torch.uint8, device=G.DEV)
    (w1, s1), (w3, s3) = _weights(H, K, rowwise, 90)
    w2 = ops.fp8_linear_quantize(G.dev_bf16(W.random_bf16(90, (K, H), 0.02, 3)), rowwise)
    for M in (1296, 1280, 272, 16):
        G.say("gated workspace", M, "rowwise", rowwise)
        xq, sx = _x(M, K, rowwise, 91)
        out = []
        for ws in (buf[:size], ops.alloc_gated_workspace(M, H, rowwise, G.DEV)):
            a, b = (torch.empty((M, H), dtype=torch.bfloat16, device=G.DEV) for _ in range(2))
            z = ops.alloc_quantized(M, H, rowwise, G.DEV)
            h = ops.fp8_gated_fwd(xq, sx, w1, s1, w3, s3, rowwise, a=a, b=b, out=z, workspace=ws)
            da, db, qa, qb = ops.fp8_gated_bwd(xq, sx, w2.qt, w2.scale_t, a, b, rowwise,
                                               workspace=ws)
            torch.cuda.synchronize()
            out.append([G.host(t) for t in (h, da, db)] + [t for q in (z, qa, qb) for t in _hq(q)])
        for p, q in zip(*out):
            assert np.array_equal(p, q), M
        assert torch.all(buf[size:] == 0x5A)
