"""The feed-forward block with its norm and the fused gate launches
(SwiGLUFFNStep with ``norm`` and ``fused``), as a training step runs them:

* every tensor of the step equals, bit for bit, the chain of the entry points
  called one by one (the norm, its quantize from a stored y, the plain
  products, the gate kernels, the quantizes of the written tensors);
* against the separate launches (``fused`` off) on the same inputs, a and b
  are equal and h is within one bf16 step;
* a side stream for the weights' quantizes changes nothing, and a captured
  step replays to the same bits."""
import numpy as np
import pytest
import torch

import oracle
from float8_mixed_precision_amd import ops
from float8_mixed_precision_amd import workloads as W
from tests import gpu_util as G

pytestmark = pytest.mark.gpu

M, D, H = 528, 272, 400
RESULTS = ("a", "b", "h", "out", "da", "db", "grad_x", "grad_w1", "grad_w3", "grad_w2")


def _inputs(seed):
    r = lambda shape, sigma, t: G.dev_bf16(W.random_bf16(seed, shape, sigma, t))
    x = r((M, D), 2.0, 0) + 0.5
    nw = (1 + 0.2 * r((1, D), 1.0, 6).float())[0].to(torch.bfloat16)
    return dict(x=x, w1=r((H, D), 0.08, 1), w3=r((H, D), 0.06, 2), w2=r((D, H), 0.05, 3),
                d_out=r((M, D), 1e-2, 4)), (nw, r((1, D), 0.1, 5)[0].contiguous())


def _snapshot(blk, names):
    torch.cuda.synchronize()
    return {n: getattr(blk, n).clone() for n in names}


@pytest.mark.parametrize("e5m2", [False, True], ids=["e4m3", "e5m2"])
@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
@pytest.mark.parametrize("rowwise", [False, True], ids=["tensorwise", "rowwise"])
def test_block_is_the_chain_of_its_calls(rowwise, rms, e5m2):
    t, (nw, nb) = _inputs(90)
    nb = None if rms else nb
    G.say("norm block", "rowwise", rowwise, "rms", rms, "e5m2", e5m2)
    blk = ops.SwiGLUFFNStep(**t, rowwise=rowwise, e5m2_grad=e5m2, fused=True, norm=(nw, nb),
                            rms=rms)
    blk.run()
    names = RESULTS + ("grad_in", "grad_norm_w") + (() if rms else ("grad_norm_b",))
    got = _snapshot(blk, names)
    # one call after the other, on buffers of their own
    y, mean, rstd = ops.fp8_layernorm_fwd(t["x"], nw, nb, rms=rms)
    q = lambda v, e=False: ops.fp8_linear_quantize(v, rowwise, e5m2=e)
    qx, q1, q3, q2 = q(y), q(t["w1"]), q(t["w3"]), q(t["w2"])
    qd = q(t["d_out"], e5m2)
    c = {"a": ops.fp8_linear_fwd(qx.q, qx.scale, q1.q, q1.scale, rowwise),
         "b": ops.fp8_linear_fwd(qx.q, qx.scale, q3.q, q3.scale, rowwise)}
    c["h"] = ops.fp8_gated_fwd(qx.q, qx.scale, q1.q, q1.scale, q3.q, q3.scale, rowwise)
    qh = q(c["h"])
    c["out"] = ops.fp8_linear_fwd(qh.q, qh.scale, q2.q, q2.scale, rowwise)
    _, c["grad_w2"] = ops.fp8_linear_bwd(None, None, qd.qt, qd.scale_t, None, None, qh.qt,
                                         qh.scale_t, M, D, H, rowwise, want_x=False, e5m2=e5m2)
    c["da"], c["db"], _, _ = ops.fp8_gated_bwd(qd.q, qd.scale, q2.qt, q2.scale_t, c["a"], c["b"],
                                               rowwise, e5m2)
    qa, qb = q(c["da"], e5m2), q(c["db"], e5m2)
    c["grad_x"], c["grad_w1"] = ops.fp8_linear_bwd(
        qa.q, qa.scale, qa.qt, qa.scale_t, q1.qt, q1.scale_t, qx.qt, qx.scale_t, M, H, D, rowwise,
        e5m2=e5m2)
    _, c["grad_w3"] = ops.fp8_linear_bwd(None, None, qb.qt, qb.scale_t, None, None, qx.qt,
                                         qx.scale_t, M, H, D, rowwise, want_x=False, e5m2=e5m2)
    ops.fp8_linear_bwd_x_acc(qb.q, qb.scale, q3.qt, q3.scale_t, M, H, D, c["grad_x"], rowwise,
                             e5m2=e5m2)
    c["grad_in"], c["grad_norm_w"], gb = ops.fp8_layernorm_bwd(c["grad_x"], t["x"], nw, mean, rstd,
                                                               rms, want_b=not rms)
    if not rms:
        c["grad_norm_b"] = gb
    torch.cuda.synchronize()
    for n in names:
        assert torch.equal(got[n], c[n]), n
    # weights' quantizes on a second stream
    blk.run(side=torch.cuda.Stream())
    for n, v in _snapshot(blk, names).items():
        assert torch.equal(got[n], v), n


@pytest.mark.parametrize("rowwise", [False, True], ids=["tensorwise", "rowwise"])
def test_fused_against_separate(rowwise):
    t, norm = _inputs(91)
    G.say("norm block fused against separate", rowwise)
    blks = [ops.SwiGLUFFNStep(**t, rowwise=rowwise, fused=f, norm=norm) for f in (True, False)]
    for b in blks:
        b.run()
    f, s = (_snapshot(b, RESULTS) for b in blks)
    assert torch.equal(f["a"], s["a"]) and torch.equal(f["b"], s["b"])
    hf, hs = (G.host(v["h"]) for v in (f, s))
    assert oracle.bf16_ulp_distance(hf.ravel(), hs.ravel()).max() <= 1


def test_captured_step():
    t, norm = _inputs(92)
    blk = ops.SwiGLUFFNStep(**t, rowwise=True, fused=True, norm=norm)
    names = RESULTS + ("grad_in", "grad_norm_w", "grad_norm_b")
    G.say("norm block graph")
    blk.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        blk.run()
    for k in range(3):
        t["x"].add_(0.25 * k)
        graph.replay()
        got = _snapshot(blk, names)
        blk.run()
        for n, v in _snapshot(blk, names).items():
            assert torch.equal(got[n], v), (k, n)
