"""GPU gated feed-forward kernels.

* a, b and dh come from the plain GEMM's instructions in its order: for more
  than 16 tokens they equal fp8_linear_fwd's / fp8_linear_bwd's outputs bit
  for bit, and with fewer (the contraction split over 8 waves) they are
  within the instruction's accumulation bound (tests/mfma_model.py) plus 7
  fp32 additions, 7 2^-24 sum |p|, and two bf16 roundings.
* h, da and db are checked in 64 bits from those bf16 a, b and dh.  With
  r = (|a| + 4) 2^-23 the documented relative error of the sigmoid s and of
  u = silu(a): h = u b carries r, one product (2^-24) and the rounding (half a
  bf16 step, 2^-8 |h| at most); silu' = s + u (1 - s) carries r (s + |u|) for
  its parts, r |u| s for 1 - s and three roundings within
  3 2^-24 (s + |u|): r (s + 2 |u|) + 2^-22 (s + |u|) covers both; below
  2^-118 an absolute term allows the flushed tail.
* The codes and scales are the oracle's quantize of the written bf16 values,
  bit for bit."""
import numpy as np
import pytest
import torch

import oracle
from float8_mixed_precision_amd import ops
from float8_mixed_precision_amd import workloads as W
from tests import gpu_util as G
from tests import mfma_model as MM

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TINY = 2.0 ** -118
RW = [False, True]
RW_IDS = ["tensorwise", "rowwise"]


def _value(bits):
    return oracle.bf16_to_f32(np.asarray(bits, np.uint16)).astype(np.float64)


def _sigmoid(a):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-a))


def check_h(h, a, b, label):
    h, a, b = _value(h), _value(a), _value(b)
    s = _sigmoid(a)
    want = a * s * b
    tol = np.abs(want) * ((np.abs(a) + 4) * 2.0 ** -23 + U) + TINY * (1 + np.abs(b))
    tol += 2.0 ** -8 * (np.abs(want) + tol)
    assert np.all(np.isfinite(h)), label
    bad = np.abs(h - want) > tol
    assert not bad.any(), "%s: %d outside, first %s" % (label, bad.sum(), np.argwhere(bad)[0])


def check_dab(da, db, dh, a, b, label):
    da, db, g, a, b = (_value(t) for t in (da, db, dh, a, b))
    s = _sigmoid(a)
    u = a * s
    d = s + u * (1 - s)
    r = (np.abs(a) + 4) * 2.0 ** -23
    wa, wb = g * b * d, g * u
    dt = r * (s + 2 * np.abs(u)) + 2.0 ** -22 * (s + np.abs(u)) + TINY
    ta = np.abs(g * b) * dt + 2 * U * np.abs(wa) + TINY
    tb = np.abs(wb) * (r + U) + TINY * (1 + np.abs(g))
    for name, got, want, tol in (("da", da, wa, ta), ("db", db, wb, tb)):
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
        bad = ~(np.abs(got - want) <= tol)
        assert not bad.any(), "%s %s: %d outside, first %s" % (label, name, bad.sum(),
                                                                np.argwhere(bad)[0])


def _hq(z):
    return tuple(G.host(t) for t in (z.q, z.qt, z.scale, z.scale_t, z.amax))


def _weights(H, K, rowwise, seed):
    ws = [ops.fp8_linear_quantize(G.dev_bf16(W.random_bf16(seed, (H, K), sg, t)), rowwise)
          for t, sg in ((1, 0.05), (2, 0.02))]
    return [(z.q, z.scale) for z in ws]


def _pad16(m):
    return (m + 15) // 16 * 16


def _x(M, K, rowwise, seed):
    """fp8 copy of M tokens (quantized in a matrix padded to 16 rows)."""
    z = ops.fp8_linear_quantize(G.dev_bf16(W.random_bf16(seed, (_pad16(M), K), 1.0, 0)), rowwise)
    return z.q, z.scale


FWD = [(32, 144, 400), (80, 16, 16), (272, 400, 528), (256, 128, 128), (528, 144, 1040), (1040, 784, 304),
       (512, 2048, 256),
       # more than 128 large tiles: those kernels, several tiles a workgroup
       (2064, 4112, 384), (4112, 8208, 144), (4096, 8192, 128)]


@pytest.mark.parametrize("rowwise", RW, ids=RW_IDS)
@pytest.mark.parametrize("mhk", FWD, ids=lambda s: "%dx%dx%d" % s)
def test_forward(mhk, rowwise):
    M, H, K = mhk
    xq, sx = _x(M, K, rowwise, 70)
    (w1, s1), (w3, s3) = _weights(H, K, rowwise, 71)
    G.say("gated fwd", mhk, "rowwise", rowwise)
    a, b = (torch.empty((M, H), dtype=torch.bfloat16, device=G.DEV) for _ in range(2))
    z = ops.alloc_quantized(M, H, rowwise, G.DEV)
    ws = ops.alloc_gated_workspace(M, H, rowwise, G.DEV).fill_(0x7F)
    h = ops.fp8_gated_fwd(xq, sx, w1, s1, w3, s3, rowwise, a=a, b=b, out=z, workspace=ws)
    h2 = ops.fp8_gated_fwd(xq, sx, w1, s1, w3, s3, rowwise)          # neither stored nor quantized
    z3 = ops.alloc_quantized(M, H, rowwise, G.DEV)
    h3 = ops.fp8_gated_fwd(xq, sx, w1, s1, w3, s3, rowwise, out=z3, workspace=ws)
    pa = ops.fp8_linear_fwd(xq, sx, w1, s1, rowwise)
    pb = ops.fp8_linear_fwd(xq, sx, w3, s3, rowwise)
    torch.cuda.synchronize()
    assert np.array_equal(G.host(a), G.host(pa)) and np.array_equal(G.host(b), G.host(pb))
    assert np.array_equal(G.host(h), G.host(h2)) and np.array_equal(G.host(h), G.host(h3))
    check_h(G.host(h), G.host(a), G.host(b), "h %s" % (mhk,))
    ref = oracle.quantize(G.host(h), rowwise)
    G.assert_quantize_equal(_hq(z), ref, "codes of h %s" % (mhk,))
    G.assert_quantize_equal(_hq(z3), ref, "codes of h, a and b not stored %s" % (mhk,))


@pytest.mark.parametrize("rowwise", RW, ids=RW_IDS)
@pytest.mark.parametrize("mhk", [(17, 272, 4112), (50, 1040, 784), (40, 28672, 32), (65, 400, 528), (131, 256, 128), (257, 144, 272),
                                 (769, 2048, 256), (2081, 4112, 144)], ids=lambda s: "%dx%dx%d" % s)
def test_forward_any_number_of_tokens(mhk, rowwise):
    """M tokens give the first M rows of the padded call, and the rows behind
    them stay as they were."""
    M, H, K = mhk
    P = _pad16(M)
    xq, sx = _x(M, K, rowwise, 72)
    (w1, s1), (w3, s3) = _weights(H, K, rowwise, 73)
    G.say("gated fwd ragged", mhk, "rowwise", rowwise)
    want = ops.fp8_gated_fwd(xq, sx, w1, s1, w3, s3, rowwise)
    bufs = [torch.full((P + 16, H), 7.0, dtype=torch.bfloat16, device=G.DEV) for _ in range(3)]
    # (exact-size copies: no readable row behind the operands' last one)
    xs, ss = xq[:M].clone(), sx[:M].clone() if rowwise else sx
    h = ops.fp8_gated_fwd(xs, ss, w1, s1, w3, s3, rowwise, h=bufs[0][:M], a=bufs[1][:M],
                          b=bufs[2][:M])
    torch.cuda.synchronize()
    assert torch.equal(h, want[:M])
    for t in bufs:
        assert torch.all(t[M:] == 7.0)


@pytest.mark.parametrize("rowwise", RW, ids=RW_IDS)
@pytest.mark.parametrize("mhk", [(1, 16, 16), (1, 512, 4096), (2, 144, 1040), (15, 400, 528),
                                 (16, 256, 2048), (17, 256, 1152), (33, 272, 4112), (50, 128, 784),
                                 (64, 528, 3088), (3, 14336, 144)], ids=lambda s: "%dx%dx%d" % s)
def test_few_tokens(mhk, rowwise):
    M, H, K = mhk
    xq, sx = _x(M, K, rowwise, 74)
    xs, ss = xq[:M].clone(), sx[:M].clone() if rowwise else sx
    (w1, s1), (w3, s3) = _weights(H, K, rowwise, 75)
    G.say("gated few tokens", mhk, "rowwise", rowwise)
    bufs = [torch.full((M + 3, H), 7.0, dtype=torch.bfloat16, device=G.DEV) for _ in range(3)]
    h = ops.fp8_gated_fwd(xs, ss, w1, s1, w3, s3, rowwise, h=bufs[0][:M], a=bufs[1][:M],
                          b=bufs[2][:M])
    h2 = ops.fp8_gated_fwd(xs, ss, w1, s1, w3, s3, rowwise)
    torch.cuda.synchronize()
    assert torch.equal(h, h2)
    for t in bufs:
        assert torch.all(t[M:] == 7.0)
    A = G.host(xs)
    ii, jj = np.divmod(np.arange(M * H), H)
    mag = np.abs(np.nan_to_num(oracle.e4m3_values()))
    for t, w, s, name in ((bufs[1], w1, s1, "a"), (bufs[2], w3, s3, "b")):
        B = G.host(w)
        want = _value(oracle.gemm_tn(A, np.atleast_1d(G.host(ss)), B, np.atleast_1d(G.host(s))))
        sa = np.broadcast_to(1 / G.host(ss).astype(np.float64), (M,))[:, None]
        sb = np.broadcast_to(1 / G.host(s).astype(np.float64), (H,))[None, :]
        D = MM.sum_difference_bound(A, B, ii, jj).reshape(M, H)
        D = D + 7 * U * (mag[A] @ mag[B].T)
        tol = D * sa * sb * (1 + 2.0 ** -20)
        tol = tol + 2.0 ** -7 * (np.abs(want) + tol)          # both sides' bf16 rounding
        got = _value(G.host(t[:M]))
        assert np.all(np.abs(got - want) <= tol), (name, mhk)
    check_h(G.host(h), G.host(bufs[1][:M]), G.host(bufs[2][:M]), "h %s" % (mhk,))
    if M % 16 == 0:
        z = ops.alloc_quantized(M, H, rowwise, G.DEV)
        h3 = ops.fp8_gated_fwd(xs, ss, w1, s1, w3, s3, rowwise, out=z)
        torch.cuda.synchronize()
        assert torch.equal(h, h3)
        G.assert_quantize_equal(_hq(z), oracle.quantize(G.host(h), rowwise), "codes %s" % (mhk,))


BWD = [(16, 16, 16), (80, 144, 48), (272, 400, 528), (256, 256, 128), (1040, 784, 304),
       (528, 4112, 400),
       # more than 128 large tiles: those kernels, several tiles a workgroup
       (64, 28672, 48), (2064, 8208, 128), (2064, 4112, 512), (4112, 16400, 272)]


@pytest.mark.parametrize("e5m2", [False, True], ids=["e4m3", "e5m2"])
@pytest.mark.parametrize("rowwise", RW, ids=RW_IDS)
@pytest.mark.parametrize("mhd", BWD, ids=lambda s: "%dx%dx%d" % s)
def test_backward(mhd, rowwise, e5m2):
    M, H, D = mhd
    qdy = ops.fp8_linear_quantize(G.dev_bf16(W.random_bf16(76, (M, D), 1e-2, 0)), rowwise,
                                  e5m2=e5m2)
    qw = ops.fp8_linear_quantize(G.dev_bf16(W.random_bf16(76, (D, H), 0.02, 1)), rowwise)
    a = W.random_bf16(77, (M, H), 3.0, 0)
    b = W.random_bf16(77, (M, H), 1.0, 1)
    a.reshape(-1)[::97] = 0xC2A0                    # -80
    a.reshape(-1)[5::97] = 0x4330                   # 176
    G.say("gated bwd", mhd, "rowwise", rowwise, "e5m2", e5m2)
    ad, bd = G.dev_bf16(a), G.dev_bf16(b)
    ws = ops.alloc_gated_workspace(M, H, rowwise, G.DEV).fill_(0x7F)
    da, db, qa, qb = ops.fp8_gated_bwd(qdy.q, qdy.scale, qw.qt, qw.scale_t, ad, bd, rowwise, e5m2,
                                       workspace=ws)
    dh, _ = ops.fp8_linear_bwd(qdy.q, qdy.scale, None, None, qw.qt, qw.scale_t, None, None, M, D,
                               H, rowwise, want_w=False, e5m2=e5m2)
    torch.cuda.synchronize()
    check_dab(G.host(da), G.host(db), G.host(dh), a, b, "bwd %s" % (mhd,))
    quant = oracle.quantize_e5m2 if e5m2 else oracle.quantize
    G.assert_quantize_equal(_hq(qa), quant(G.host(da), rowwise), "codes of da %s" % (mhd,))
    G.assert_quantize_equal(_hq(qb), quant(G.host(db), rowwise), "codes of db %s" % (mhd,))


@pytest.mark.parametrize("rowwise", RW, ids=RW_IDS)
def test_backward_special_gates(rowwise):
    """Every finite bf16 gate value, and infinities and NaN, against the
    formulas; non-finite results appear where the formulas give them."""
    M, H, D = 4096, 16, 32
    a = np.arange(1 << 16, dtype=np.uint32).astype(np.uint16).reshape(M, H)
    b = W.random_bf16(78, (M, H), 1.0, 1)
    qdy = ops.fp8_linear_quantize(G.dev_bf16(W.random_bf16(78, (M, D), 1.0, 0)), rowwise)
    qw = ops.fp8_linear_quantize(G.dev_bf16(W.random_bf16(78, (D, H), 0.1, 2)), rowwise)
    G.say("gated bwd every gate", "rowwise", rowwise)
    da, db, qa, _ = ops.fp8_gated_bwd(qdy.q, qdy.scale, qw.qt, qw.scale_t, G.dev_bf16(a),
                                      G.dev_bf16(b), rowwise)
    dh, _ = ops.fp8_linear_bwd(qdy.q, qdy.scale, None, None, qw.qt, qw.scale_t, None, None, M, D,
                               H, rowwise, want_w=False)
    torch.cuda.synchronize()
    da, db, dh = G.host(da), G.host(db), G.host(dh)
    # sums of products near the type's limit overflow differently: keep |a| < 2^100
    av = _value(a)
    fin = np.isfinite(av) & (np.abs(av) < 2.0 ** 100)
    z = np.zeros_like(a)
    check_dab(np.where(fin, da, z), np.where(fin, db, z), np.where(fin, dh, z),
              np.where(fin, a, z), np.where(fin, b, z), "every gate")
    nan = np.isnan(av)
    assert np.isnan(_value(da)[nan]).all() and np.isnan(_value(db)[nan]).all()
    neg_inf = a == 0xFF80
    assert np.isnan(_value(db)[neg_inf]).all()      # silu(-inf) = -inf * 0
    am = G.host(qa.amax)
    assert np.isnan(am[0]) if not rowwise else np.isnan(am[:M][nan.any(1)]).all()


@pytest.mark.parametrize("rowwise", RW, ids=RW_IDS)
def test_empty_dimensions(rowwise):
    G.say("gated empty", rowwise)
    E = lambda r, c: torch.empty((r, c), dtype=torch.uint8, device=G.DEV)
    ones = lambda n: torch.ones(n if rowwise else 1, device=G.DEV)
    bf = dict(dtype=torch.bfloat16, device=G.DEV)
    for M in (0, 96, 7):                             # no tokens; an empty contraction
        K = 0 if M else 32
        z = ops.alloc_quantized(M, 48, rowwise, G.DEV) if M % 16 == 0 else None
        a, b, h = (torch.full((M, 48), 3.0, **bf) for _ in range(3))
        ops.fp8_gated_fwd(E(M, K), ones(M), E(48, K).fill_(1), ones(48), E(48, K).fill_(1),
                          ones(48), rowwise, h=h, a=a, b=b, out=z)
        torch.cuda.synchronize()
        for t in (a, b, h):
            assert torch.all(t == 0)
        if z is not None:
            assert torch.all(z.q == 0)
            assert torch.all(z.scale_t == float(oracle.scale_from_amax(0.0)))
    a = torch.full((32, 48), 1.0, **bf)
    da, db, qa, qb = ops.fp8_gated_bwd(E(32, 0), ones(32), E(48, 0), ones(48), a, a, rowwise)
    torch.cuda.synchronize()
    assert torch.all(da == 0) and torch.all(db == 0) and torch.all(qa.q == 0)
    e = torch.empty((0, 48), **bf)
    da, db, qa, qb = ops.fp8_gated_bwd(E(0, 32), ones(0), E(48, 32).fill_(1), ones(48), e, e,
                                       rowwise)
    torch.cuda.synchronize()
    assert torch.all(qb.scale_t == float(oracle.scale_from_amax(0.0)))


def test_nonfinite_scales_reach_the_amax():
    """A NaN in x (its scale is NaN) makes h and the amax of h NaN."""
    M, H, K = 96, 144, 64
    x = W.random_bf16(79, (M, K), 1.0, 0)
    x[5, 5] = 0x7FC0
    z = ops.fp8_linear_quantize(G.dev_bf16(x), True)
    (w1, s1), (w3, s3) = _weights(H, K, True, 79)
    out = ops.alloc_quantized(M, H, True, G.DEV)
    G.say("gated nan")
    h = ops.fp8_gated_fwd(z.q, z.scale, w1, s1, w3, s3, True, out=out)
    torch.cuda.synchronize()
    nan = torch.isnan(h.float()).cpu().numpy()
    assert nan[5].all() and not nan[:5].any() and not nan[6:].any()
    am = G.host(out.amax)
    assert np.isnan(am[5]) and np.isfinite(am[:5]).all() and np.isnan(am[M:]).all()


def test_streams_and_graph():
    """Two calls at once on two streams with workspaces of their own, and a
    captured forward and backward replayed three times on changing inputs."""
    M, H, K = 320, 528, 272
    rw = True
    (w1, s1), (w3, s3) = _weights(H, K, rw, 80)
    w2 = ops.fp8_linear_quantize(G.dev_bf16(W.random_bf16(80, (K, H), 0.02, 3)), rw)
    sets = []
    for k in range(2):
        bf = dict(dtype=torch.bfloat16, device=G.DEV)
        sets.append(dict(x=_x(M, K, rw, 81 + k), dy=_x(M, K, rw, 83 + k),
                         a=torch.empty((M, H), **bf), b=torch.empty((M, H), **bf),
                         h=torch.empty((M, H), **bf), da=torch.empty((M, H), **bf),
                         db=torch.empty((M, H), **bf),
                         z=[ops.alloc_quantized(M, H, rw, G.DEV) for _ in range(3)],
                         ws=ops.alloc_gated_workspace(M, H, rw, G.DEV)))

    def step(s):
        ops.fp8_gated_fwd(*s["x"], w1, s1, w3, s3, rw, h=s["h"], a=s["a"], b=s["b"],
                          out=s["z"][0], workspace=s["ws"])
        ops.fp8_gated_bwd(*s["dy"], w2.qt, w2.scale_t, s["a"], s["b"], rw, da=s["da"],
                          db=s["db"], qa=s["z"][1], qb=s["z"][2], workspace=s["ws"])

    def results(s):
        torch.cuda.synchronize()
        r = [s[n].clone() for n in ("a", "b", "h", "da", "db")]
        for z in s["z"]:
            r += [t.clone() for t in (z.q, z.qt, z.scale, z.scale_t, z.amax)]
        return r

    G.say("gated streams")
    want = []
    for s in sets:
        step(s)
        want.append(results(s))
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for s, st in zip(sets, streams):
        with torch.cuda.stream(st):
            step(s)
    for s, w in zip(sets, want):
        for p, q in zip(results(s), w):
            assert torch.equal(p, q)
    G.say("gated graph")
    s = sets[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(s)
    for k in range(3):
        s["x"][0].copy_(sets[1]["x"][0] if k % 2 else torch.flip(s["x"][0], (0,)))
        graph.replay()
        got = results(s)
        step(s)
        for p, q in zip(results(s), got):
            assert torch.equal(p, q)
