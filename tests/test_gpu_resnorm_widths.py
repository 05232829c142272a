"""Residual norm's backward with codes at the widths of 320 and 640 threads a row
(2049-2560 and 4097-5120 columns), over several rounds of rows a workgroup: the
gradients against the formulas in 64 bits (bounds of test_gpu_resnorm.py), the same
with and without codes, and the codes the oracle's."""
import pytest
import torch

import oracle
from float8_mixed_precision_amd import ops
from tests import gpu_util as G
from tests.test_gpu_layernorm import BF, F32
from tests.test_gpu_resnorm import Case, _check_grads, _grads64, _hq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("norms", ["both", "post", "pre"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1088, 2064), (1040, 2560), (16, 2064), (784, 4112), (528, 5120)],
                         ids=lambda s: "%dx%d" % s)
def test_backward_with_codes(shape, dtype, norms):
    rows, cols = shape
    rms = rows % 32 == 0
    c = Case(rows, cols, dtype, BF, norms, cols + 7)
    s, _, st = ops.fp8_resnorm_fwd(c.dev["b"], c.dev["x"], alpha=0.9, rms=rms, **c.params())
    args = (c.dev["dy"], c.dev["ds"], c.dev["b"], s, st)
    plain = ops.fp8_resnorm_bwd(*args, alpha=0.9, rms=rms, **c.params())
    torch.cuda.synchronize()
    _check_grads(plain, _grads64(c, s.cpu(), st, 0.9, rms), dtype, "%s" % (shape,))
    for rowwise in (False, True):
        for e5m2 in (False, True):
            G.say("resnorm bwd codes", shape, dtype, norms, "rowwise", rowwise, "e5m2", e5m2)
            ws = torch.full((ops.fp8_resnorm_workspace_bytes(rows, cols, rowwise),), 0x7F,
                            dtype=torch.uint8, device=G.DEV)
            z = ops.alloc_quantized(rows, cols, rowwise, G.DEV)
            grads = ops.fp8_resnorm_bwd(*args, alpha=0.9, rms=rms, out=z, rowwise=rowwise,
                                        e5m2=e5m2, workspace=ws, **c.params())
            torch.cuda.synchronize()
            for n in ops.ResNormGrads.__slots__:
                p, q = getattr(plain, n), getattr(grads, n)
                assert (p is None and q is None) or torch.equal(p, q), n
            quantize = oracle.quantize_e5m2 if e5m2 else oracle.quantize
            G.assert_quantize_equal(_hq(z), quantize(G.host(grads.db), rowwise),
                                    "codes of db %s" % (shape,))
