"""The biased feed-forward block between two norms of a residual stream
(MLPStep), as a training step runs it:

* every tensor of the step equals, bit for bit, the chain of the entry points
  called one by one, with the quantizes of the written tensors in the place of the
  fused ones;
* its outputs and gradients follow a 64-bit chain of the formulas on the same
  operands (the fp8 copies' own rounding left out: the 64-bit chain starts from the
  values that the codes stand for at each product);
* a captured step replays to the same bits, on two streams in turn."""
import numpy as np
import pytest
import torch

import oracle
from float8_mixed_precision_amd import ops
from float8_mixed_precision_amd import workloads as W
from tests import gpu_util as G
from tests.test_gpu_linear_act import act64

pytestmark = pytest.mark.gpu

M, D, H = 528, 272, 400
BF, F32 = torch.bfloat16, torch.float32


def _block(seed, rowwise, e5m2=False, dtype=BF, act="gelu", post=True, bias=True, rms=False):
    r = lambda shape, sigma, t: G.dev_bf16(W.random_bf16(seed, shape, sigma, t))
    vec = lambda base, sigma, t: (base + r((1, D), sigma, t).float())[0].to(BF)
    qy = ops.fp8_linear_quantize(r((M, D), 1.0, 0), rowwise)
    b1 = r((1, H), 0.3, 1)[0].contiguous() if bias else None
    b2 = r((1, D), 0.3, 2)[0].float() if bias else None
    return ops.MLPStep(qy, (r((M, D), 2.0, 3) + 0.5).to(dtype), r((H, D), 0.06, 4), b1,
                       r((D, H), 0.05, 5), b2, r((M, D), 1e-2, 6).to(dtype), r((M, D), 1e-2, 7),
                       act, (vec(1, 0.2, 8), vec(0, 0.1, 9)) if post else None,
                       (vec(1, 0.2, 10), vec(0, 0.1, 11)), vec(0.5, 0.2, 12), 0.9, rms=rms,
                       rowwise=rowwise, e5m2_grad=e5m2)


def _results(b):
    torch.cuda.synchronize()
    r = {n: getattr(b, n) for n in ("z", "out", "s", "dz", "grad_y", "grad_w1", "grad_w2",
                                    "grad_b1", "grad_b2")}
    r.update({n: getattr(b.grads, n) for n in ops.ResNormGrads.__slots__})
    for n in ("qh", "qs", "qdo", "qdz"):
        q = getattr(b, n)
        r.update({n + "." + k: getattr(q, k) for k in ("q", "qt", "scale", "scale_t", "amax")})
    return {n: v.clone() for n, v in r.items() if v is not None}


CASES = [dict(rowwise=False), dict(rowwise=True, e5m2=True, act="silu", rms=True),
         dict(rowwise=False, e5m2=True, dtype=F32, act="relu2"),
         dict(rowwise=True, post=False, bias=False, act="gelu_tanh")]


@pytest.mark.parametrize("kw", CASES, ids=["tensorwise", "rowwise_rms", "f32_stream", "no_bias"])
def test_block_is_the_chain_of_its_calls(kw):
    b = _block(60, **kw)
    G.say("mlp block", kw)
    b.run()
    got = _results(b)
    rw, e5 = b.rowwise, b.e5m2_grad
    q = lambda v, e=False: ops.fp8_linear_quantize(v, rw, e5m2=e)
    q1, q2 = q(b.w1), q(b.w2)
    c = {"z": torch.empty_like(b.z)}
    h = ops.fp8_linear_act_fwd(b.qy.q, b.qy.scale, q1.q, q1.scale, b.b1, b.act, rowwise=rw,
                               z=c["z"])
    qh = q(h)
    c["out"] = ops.fp8_linear_act_fwd(qh.q, qh.scale, q2.q, q2.scale, b.b2, rowwise=rw)
    c["s"], y, st = ops.fp8_resnorm_fwd(c["out"], b.x, b.post, b.pre, b.gate, b.alpha, b.eps,
                                        b.rms)
    g = ops.fp8_resnorm_bwd(b.d_y, b.d_s, c["out"], c["s"], st, b.post, b.pre, b.gate, b.alpha,
                            b.rms)
    c.update({n: getattr(g, n) for n in ops.ResNormGrads.__slots__ if getattr(g, n) is not None})
    qdo = q(g.db, e5)
    if b.b2 is not None:
        _, _, c["grad_b2"] = ops.fp8_bias_act_bwd(g.db, rowwise=rw, e5m2=e5, bias_dtype=F32)
    c["dz"], _, gb1 = ops.fp8_linear_act_bwd(qdo.q, qdo.scale, q2.qt, q2.scale_t, c["z"], b.act, rw,
                                             e5, bias_dtype=BF)
    if b.b1 is not None:
        c["grad_b1"] = gb1
    qdz = q(c["dz"], e5)
    c["grad_y"], c["grad_w1"] = ops.fp8_linear_bwd(
        qdz.q, qdz.scale, qdz.qt, qdz.scale_t, q1.qt, q1.scale_t, b.qy.qt, b.qy.scale_t, M, H, D,
        rw, e5m2=e5)
    _, c["grad_w2"] = ops.fp8_linear_bwd(None, None, qdo.qt, qdo.scale_t, None, None, qh.qt,
                                         qh.scale_t, M, D, H, rw, want_x=False, e5m2=e5)
    for n, v in (("qh", qh), ("qs", q(y)), ("qdo", qdo), ("qdz", qdz)):
        c.update({n + "." + k: getattr(v, k) for k in ("q", "qt", "scale", "scale_t", "amax")})
    torch.cuda.synchronize()
    assert set(c) == set(got)
    for n in c:
        assert torch.equal(c[n], got[n]), n


def test_against_64_bits():
    """Relative Frobenius errors: each bf16 tensor carries its rounding (2^-9 rms at
    most) and the fp8 products' sums; 1e-2 allows a few of each in a chain."""
    b = _block(61, False)
    G.say("mlp block against 64 bits")
    b.run()
    torch.cuda.synchronize()
    val = lambda q, s, t=None: oracle.e4m3_values()[G.host(q)] / G.host(s).astype(np.float64)
    v = lambda t: t.double().cpu().numpy()

    def close(name, got, want, tol=1e-2):
        e = np.linalg.norm(v(got) - want) / np.linalg.norm(want)
        assert e < tol, (name, e)

    y, w1, w2 = val(b.qy.q, b.qy.scale), val(b.qw1.q, b.qw1.scale), val(b.qw2.q, b.qw2.scale)
    z = y @ w1.T + v(b.b1)
    close("z", b.z, z)
    close("h", torch.from_numpy(val(b.qh.q, b.qh.scale)), act64(z, "gelu")[0], 0.05)   # fp8 codes
    h = val(b.qh.q, b.qh.scale)
    out = h @ w2.T + v(b.b2)
    close("out", b.out, out)

    def norm(t, pair):
        m = t.mean(1, keepdims=True)
        r = 1 / np.sqrt(((t - m) ** 2).mean(1, keepdims=True) + b.eps)
        return (t - m) * r * v(pair[0]) + v(pair[1]), (t - m) * r, r

    t, xh1, r1 = norm(out, b.post)
    s = b.alpha * v(b.x) + v(b.gate) * t
    close("s", b.s, s)
    yn, xh2, r2 = norm(s, b.pre)
    close("y", torch.from_numpy(val(b.qs.q, b.qs.scale)), yn, 0.05)                    # fp8 codes

    def back(g, xh, r):
        return r * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))

    dT = v(b.d_s) + back(v(b.d_y) * v(b.pre[0]), xh2, r2)
    db = back(dT * v(b.gate) * v(b.post[0]), xh1, r1)
    close("dx", b.grads.dx, b.alpha * dT)
    close("db", b.grads.db, db)
    close("dgate", b.grads.dgate, (dT * t).sum(0))
    close("dpre_weight", b.grads.dpre_weight, (v(b.d_y) * xh2).sum(0))
    close("grad_b2", b.grad_b2, db.sum(0))
    dz = (val(b.qdo.q, b.qdo.scale) @ w2) * act64(v(b.z), "gelu")[1]
    close("dz", b.dz, dz)
    close("grad_b1", b.grad_b1, dz.sum(0))
    dzq = val(b.qdz.q, b.qdz.scale)
    close("grad_y", b.grad_y, dzq @ w1)
    close("grad_w1", b.grad_w1, dzq.T @ y)
    close("grad_w2", b.grad_w2, val(b.qdo.q, b.qdo.scale).T @ h)


@pytest.mark.parametrize("rowwise", [False, True], ids=["tensorwise", "rowwise"])
def test_captured_step(rowwise):
    b = _block(62, rowwise)
    G.say("mlp block graph", rowwise)
    b.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.run()
    side = torch.cuda.Stream()
    for k in range(3):
        b.x.add_(0.25 * k)
        graph.replay()
        got = _results(b)
        if k == 1:
            b.run()
        else:                                                # a stream given to the calls
            side.wait_stream(torch.cuda.current_stream())
            b.run(side)
            side.synchronize()
        for n, v in _results(b).items():
            assert torch.equal(got[n], v), (k, n)
