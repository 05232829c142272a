"""GPU layer norm (and its RMS form) against the formulas in 64 bits.

Tolerances (u = 2^-24, one fp32 rounding):

* A row sum of C values takes at most 64 sequential additions per thread, 4
  DPP and 3 scalar steps over a wave and 15 over a row's waves, each within u
  of the running sum: relative to the sum of magnitudes, S = (64 + 22) u.
* mean: S mean|x| + u |mean| (the product with 1/C, 1/C itself within u).
* rstd: the squares carry 3 roundings each, their sum S, the mean's error d
  enters as d^2; square root and reciprocal add 4 u: relative
  (S + 8 u) / 2 + 4 u + d^2 / (2 (var + eps)).
* y: (d + u |x - mean|) rstd |w| for the difference, the relative error of
  rstd and 2 u on xh w, u (|y| + |b|) for the last operation, then the
  rounding to y's type: half a step (bf16 2^-8, fp32 2^-24 of |y|).
* dx: the two row sums S (+ 3 u for the factors), 5 u on each of the three
  terms, the rounding to dx's type.
* dweight, dbias: each thread adds rows in turn, ceil(rows / 256) at most, then
  up to 16 row groups and 16 + 16 partial rows: (rows / 256 + 50) u of the sum
  of magnitudes, 3 u more for xh.
"""
import numpy as np
import pytest
import torch

import oracle
from float8_mixed_precision_amd import ops
from tests import gpu_util as G

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
S = 86 * U
EPS = 1e-5
BF, F32 = torch.bfloat16, torch.float32
SIZES = [(1, 1), (3, 5), (2, 7), (5, 8), (4, 9), (7, 100), (33, 513), (9, 1000), (5, 1025),
         (3, 2050), (2, 4096), (3, 5001), (2, 8200), (2, 16383), (1, 16384), (1500, 136),
         (1100, 1001), (1030, 2049), (1040, 4096)]


def _half(t):
    return 2.0 ** -8 if t == BF else U


def _make(rows, cols, dtype, pdtype, seed, offset=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g) * 2 + offset
    x[:, ::64] *= 20.0                                   # outlier channels
    w = 1 + 0.3 * torch.randn(cols, generator=g)
    b = 0.2 * torch.randn(cols, generator=g)
    dy = 0.1 * torch.randn((rows, cols), generator=g)
    return x.to(dtype), w.to(pdtype), b.to(pdtype), dy.to(dtype)


def _d(t):
    return t.double().cpu().numpy()


def _forward64(x, w, b, rms, eps=EPS):
    x = _d(x)
    mean = np.zeros(x.shape[0]) if rms else x.mean(1)
    c = x - mean[:, None]
    var = (c * c).mean(1)
    rstd = 1 / np.sqrt(var + eps)
    W = np.ones(x.shape[1]) if w is None else _d(w)
    B = np.zeros(x.shape[1]) if b is None else _d(b)
    y = c * rstd[:, None] * W + B
    d = 0 * mean if rms else S * np.abs(x).mean(1) + 2 * U * np.abs(mean)
    r_rel = (S + 8 * U) / 2 + 4 * U + d * d / (2 * (var + eps))
    ytol = (((d[:, None] + U * np.abs(c)) * rstd[:, None]
             + (r_rel[:, None] + 2 * U) * np.abs(c) * rstd[:, None]) * np.abs(W)
            + U * (np.abs(y) + np.abs(B)))
    return mean, rstd, y, d, r_rel * rstd, ytol


def _backward64(dy, x, w, mean, rstd, rms):
    x, dy, r = _d(x), _d(dy), _d(rstd)[:, None]
    m = 0 if rms else _d(mean)[:, None]
    W = np.ones(x.shape[1]) if w is None else _d(w)
    xh = (x - m) * r
    g = dy * W
    c1 = (g * xh).mean(1, keepdims=True)
    c2 = 0 * c1 if rms else g.mean(1, keepdims=True)
    dx = r * (g - c2 - xh * c1)
    s = S + 4 * U
    tol = r * (5 * U * (np.abs(g) + np.abs(c2) + np.abs(xh * c1))
               + (0 if rms else s * np.abs(g).mean(1, keepdims=True))
               + np.abs(xh) * s * np.abs(g * xh).mean(1, keepdims=True))
    n = (x.shape[0] / 256 + 53) * U
    return (dx, (dy * xh).sum(0), dy.sum(0), tol, n * np.abs(dy * xh).sum(0),
            n * np.abs(dy).sum(0))


def _within(got, want, tol, label):
    got = _d(got)
    assert np.all(np.isfinite(got)), label
    bad = np.abs(got - want) > tol
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError("%s: %d of %d outside; first %s: %r, want %r, tol %.3g" % (
            label, bad.sum(), bad.size, i, got[i], want[i], tol[i]))


@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
@pytest.mark.parametrize("dtype,pdtype", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)],
                         ids=["bf16", "bf16_f32params", "f32", "f32_bf16params"])
@pytest.mark.parametrize("shape", SIZES, ids=lambda s: "%dx%d" % s)
def test_forward_and_backward(shape, dtype, pdtype, rms):
    rows, cols = shape
    x, w, b, dy = _make(rows, cols, dtype, pdtype, rows * 31 + cols)
    G.say("layernorm", shape, dtype, pdtype, "rms", rms)
    xd, wd, bd, dyd = (t.to(G.DEV) for t in (x, w, b, dy))
    # the rows behind the last one stay as they are
    guard = torch.full((rows + 3, cols), 77.0, dtype=dtype, device=G.DEV)
    y, mean, rstd = ops.fp8_layernorm_fwd(xd, wd, bd, EPS, rms, y=guard[:rows])
    torch.cuda.synchronize()
    m64, r64, y64, dtol, rtol, ytol = _forward64(x, w, b, rms)
    assert torch.all(guard[rows:] == 77.0)
    if not rms:
        _within(mean, m64, dtol, "mean")
    _within(rstd, r64, rtol, "rstd")
    _within(y, y64, ytol + _half(dtype) * (np.abs(y64) + ytol), "y")
    G.say("layernorm bwd", shape, dtype, pdtype, "rms", rms)
    guard.fill_(77.0)
    dx, dw, db = ops.fp8_layernorm_bwd(dyd, xd, wd, mean, rstd, rms, dx=guard[:rows])
    torch.cuda.synchronize()
    dx64, dw64, db64, xt, wt, bt = _backward64(dy, x, w, mean, rstd, rms)
    assert torch.all(guard[rows:] == 77.0)
    _within(dx, dx64, xt + _half(dtype) * (np.abs(dx64) + xt), "dx")
    _within(dw, dw64, wt, "dweight")
    _within(db, db64, bt, "dbias")


@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
def test_gradients_against_differences(rms):
    """Directional derivatives of sum(y * dy) by central differences of the
    64-bit forward (step 1e-4: truncation about 1e-8 of the value, rounding
    1e-12), against the kernel's gradients along the same directions."""
    rows, cols = 6, 520
    x, w, b, dy = _make(rows, cols, F32, F32, 5)
    G.say("layernorm differences", "rms", rms)
    args = [t.to(G.DEV) for t in (x, w, b)]
    _, mean, rstd = ops.fp8_layernorm_fwd(*args, EPS, rms)
    grads = ops.fp8_layernorm_bwd(dy.to(G.DEV), args[0], args[1], mean, rstd, rms)
    torch.cuda.synchronize()
    _, _, _, xt, wt, bt = _backward64(dy, x, w, mean, rstd, rms)
    rng = np.random.default_rng(3)
    h = 1e-4
    for k, (p, gk, tol) in enumerate(zip((x, w, b), grads, (xt, wt, bt))):
        v = rng.standard_normal(tuple(p.shape))

        def loss(sign):
            q = [t.double() for t in (x, w, b)]
            q[k] = q[k] + sign * h * torch.from_numpy(v)
            return float((_forward64(*q, rms)[2] * _d(dy)).sum())

        diff = (loss(1) - loss(-1)) / (2 * h)
        got = float((_d(gk) * v).sum())
        # mean and rstd as the forward kernel left them are within 1e-5 of exact
        allowed = float((tol * np.abs(v)).sum()) + 1e-5 * float((np.abs(_d(gk) * v)).sum())
        assert abs(got - diff) <= allowed, (k, got, diff, allowed)


@pytest.mark.parametrize("offset", [0.0, 1000.0])
def test_offset_row(offset):
    """A common offset costs no digits of the variance (it is taken about
    the mean): 1000 with a deviation of 2, fp32."""
    x = (torch.randn((4, 3000), generator=torch.Generator().manual_seed(1)) * 2 + offset)
    y, mean, rstd = ops.fp8_layernorm_fwd(x.to(G.DEV), None, None, EPS)
    torch.cuda.synchronize()
    m64, r64, y64, dtol, rtol, ytol = _forward64(x, None, None, False)
    _within(mean, m64, dtol, "mean")
    _within(rstd, r64, rtol, "rstd")
    _within(y, y64, ytol + U * np.abs(y64), "y")


def test_constant_zero_and_nonfinite_rows():
    """A constant row normalizes to the bias, an infinity or a NaN stays in
    its own row."""
    cols = 1200
    x = torch.randn((6, cols), generator=torch.Generator().manual_seed(2))
    x[1] = 3.0
    x[2] = 0.0
    x[3, 7] = float("inf")
    x[4, 1199] = float("nan")
    w = torch.full((cols,), 2.0)
    b = torch.full((cols,), 0.5)
    G.say("layernorm special rows")
    for dtype in (F32, BF):
        y, mean, rstd = ops.fp8_layernorm_fwd(x.to(dtype).to(G.DEV), w.to(G.DEV), b.to(G.DEV),
                                              EPS)
        torch.cuda.synchronize()
        y = y.float().cpu()
        assert torch.all(y[1] == 0.5) and torch.all(y[2] == 0.5)
        assert torch.isnan(y[3, 7]) and torch.isnan(y[4]).all()
        want = _forward64(x.to(dtype), w, b, False)
        for r in (0, 5):
            tol = want[5][r] + _half(dtype) * (np.abs(want[2][r]) + want[5][r])
            assert np.all(np.abs(_d(y[r]) - want[2][r]) <= tol)


@pytest.mark.parametrize("cols", [7, 1200, 4098])
def test_sums_past_the_range(cols):
    """Squares that add up past fp32 give rstd = 0 (y is the bias), a sum of x
    past it NaN; squares below the range count as 0; the rows beside them are
    as ever."""
    x = torch.randn((6, cols), generator=torch.Generator().manual_seed(3))
    sign = torch.where(torch.arange(cols) % 2 == 0, 1.0, -1.0)
    x[0], x[1], x[2] = 1e20 * sign, 3e38, 1e-30 * sign
    w = torch.full((cols,), 2.0)
    b = torch.full((cols,), 0.5)
    G.say("layernorm range %d" % cols)
    for rms in (False, True):
        y, mean, rstd = ops.fp8_layernorm_fwd(x.to(G.DEV), w.to(G.DEV), b.to(G.DEV), EPS, rms)
        torch.cuda.synchronize()
        y, rstd = y.cpu(), rstd.cpu()
        assert rstd[0] == 0 and torch.all(y[0] == 0.5)
        assert torch.all(y[1] == 0.5) if rms else torch.isnan(y[1]).all()
        # 2 x / sqrt(EPS) is far below half a step of 0.5
        assert abs(float(rstd[2]) * EPS ** 0.5 - 1) < 2.0 ** -20 and torch.all(y[2] == 0.5)
        want = _forward64(x[3:], w, b, rms)
        assert np.all(np.abs(_d(y[3:]) - want[2]) <= want[5] + U * (np.abs(want[2]) + want[5]))


def _hq(qz):
    return tuple(G.host(t) for t in (qz.q, qz.qt, qz.scale, qz.scale_t, qz.amax))


Q_SIZES = [(16, 16), (272, 400), (48, 4112), (1040, 80), (528, 784), (32, 16384), (2064, 1024),
           (1088, 8208), (4096, 4096)]


@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
@pytest.mark.parametrize("rowwise", [False, True], ids=["tensorwise", "rowwise"])
@pytest.mark.parametrize("shape", Q_SIZES, ids=lambda s: "%dx%d" % s)
def test_quantize(shape, rowwise, rms):
    """With y stored: y is the forward's, and the codes are the oracle's
    quantize of that y, bit for bit.  Without: the same codes."""
    rows, cols = shape
    x, w, b, _ = _make(rows, cols, BF, BF if rows % 32 else F32, cols)
    G.say("layernorm quantize", shape, "rowwise", rowwise, "rms", rms)
    xd, wd, bd = (t.to(G.DEV) for t in (x, w, b))
    y = torch.empty_like(xd)
    ws = ops.alloc_layernorm_workspace(rows, cols, G.DEV, rowwise).fill_(0x7F)
    qz, mean, rstd = ops.fp8_layernorm_quantize(xd, wd, bd, EPS, rms, rowwise, y=y, workspace=ws)
    y0, mean0, rstd0 = ops.fp8_layernorm_fwd(xd, wd, bd, EPS, rms)
    q2, mean2, rstd2 = ops.fp8_layernorm_quantize(xd, wd, bd, EPS, rms, rowwise, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(y.view(torch.int16), y0.view(torch.int16))
    assert torch.equal(rstd, rstd0) and torch.equal(rstd, rstd2)
    if not rms:
        assert torch.equal(mean, mean0) and torch.equal(mean, mean2)
    ref = oracle.quantize(G.host(y), rowwise)
    G.assert_quantize_equal(_hq(qz), ref, "codes of y %s" % (shape,))
    G.assert_quantize_equal(_hq(q2), ref, "codes without y %s" % (shape,))


@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
@pytest.mark.parametrize("shape", [(1, 16), (1, 4096), (3, 16384), (17, 400), (50, 8192),
                                   (513, 1024), (1025, 2064)], ids=lambda s: "%dx%d" % s)
def test_quantize_rows(shape, rms):
    """The serving form: any number of rows, codes and scales of the rows
    alone, as the oracle's rowwise quantize gives them for this y."""
    rows, cols = shape
    x, w, b, _ = _make(rows, cols, BF, BF, cols + 1)
    G.say("layernorm quantize rows", shape, "rms", rms)
    xd, wd, bd = (t.to(G.DEV) for t in (x, w, b))
    y = torch.empty_like(xd)
    qz, mean, rstd = ops.fp8_layernorm_quantize(xd, wd, bd, EPS, rms, True, transposed=False, y=y)
    q2, _, _ = ops.fp8_layernorm_quantize(xd, wd, bd, EPS, rms, True, transposed=False,
                                          want_stats=False)
    y0, _, rstd0 = ops.fp8_layernorm_fwd(xd, wd, bd, EPS, rms)
    torch.cuda.synchronize()
    assert torch.equal(y.view(torch.int16), y0.view(torch.int16)) and torch.equal(rstd, rstd0)
    pad = np.zeros(((rows + 15) // 16 * 16, cols), np.uint16)
    pad[:rows] = G.host(y)
    ref = oracle.quantize(pad, True)
    for z in (qz, q2):
        assert np.array_equal(G.host(z.q), ref[0][:rows])
        assert np.array_equal(G.host(z.scale), ref[2][:rows])
        assert np.array_equal(G.host(z.amax), ref[4][:rows])


@pytest.mark.parametrize("rowwise", [False, True], ids=["tensorwise", "rowwise"])
def test_empty(rowwise):
    e = torch.empty((0, 64), dtype=BF, device=G.DEV)
    G.say("layernorm empty", rowwise)
    y, mean, rstd = ops.fp8_layernorm_fwd(e)
    qz, _, _ = ops.fp8_layernorm_quantize(e, rowwise=rowwise)
    dx, dw, db = ops.fp8_layernorm_bwd(e, e, None, mean, rstd)
    torch.cuda.synchronize()
    assert y.shape == (0, 64) and dx.shape == (0, 64)
    assert torch.all(dw == 0) and torch.all(db == 0)
    assert torch.all(qz.scale_t == float(oracle.scale_from_amax(0.0)))


def test_skipped_gradients_and_repeatability():
    rows, cols = 700, 1032
    x, w, b, dy = (t.to(G.DEV) for t in _make(rows, cols, BF, BF, 9))
    G.say("layernorm partial gradients")
    _, mean, rstd = ops.fp8_layernorm_fwd(x, w, b)
    full = ops.fp8_layernorm_bwd(dy, x, w, mean, rstd)
    again = ops.fp8_layernorm_bwd(dy, x, w, mean, rstd)
    dx, n1, n2 = ops.fp8_layernorm_bwd(dy, x, w, mean, rstd, want_w=False, want_b=False)
    n3, dw, n4 = ops.fp8_layernorm_bwd(dy, x, w, mean, rstd, want_x=False, want_b=False)
    n5, n6, db = ops.fp8_layernorm_bwd(dy, x, w, mean, rstd, want_x=False, want_w=False)
    torch.cuda.synchronize()
    assert n1 is n2 is n3 is n4 is n5 is n6 is None
    for a, p, q in zip(full, again, (dx, dw, db)):
        assert torch.equal(a, p) and torch.equal(a, q)


def test_side_stream_and_graph():
    """The same results on a stream of its own and from a captured graph,
    replayed three times with eager work between the replays."""
    rows, cols = 96, 1040
    x, w, b, dy = (t.to(G.DEV) for t in _make(rows, cols, BF, BF, 10))
    ws = ops.alloc_layernorm_workspace(rows, cols, G.DEV, True)
    out = ops.alloc_quantized(rows, cols, True, G.DEV)
    mean, rstd = (torch.empty(rows, device=G.DEV) for _ in range(2))
    dx, dw, db = torch.empty_like(x), torch.empty(cols, device=G.DEV), torch.empty(cols,
                                                                                  device=G.DEV)

    def step():
        ops.fp8_layernorm_quantize(x, w, b, EPS, False, True, mean=mean, rstd=rstd, out=out,
                                   workspace=ws)
        ops.fp8_layernorm_bwd(dy, x, w, mean, rstd, dx=dx, dweight=dw, dbias=db, workspace=ws)

    def results():
        torch.cuda.synchronize()
        return [t.clone() for t in (out.q, out.qt, out.scale, out.scale_t, mean, rstd, dx, dw,
                                    db)]

    G.say("layernorm stream and graph")
    step()
    want = results()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    for a, p in zip(want, results()):
        assert torch.equal(a, p)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        x.mul_(1.0 + k)                    # new input each replay
        graph.replay()
        got = results()
        step()
        for a, p in zip(results(), got):
            assert torch.equal(a, p)


def test_offsets_past_32_bits():
    """More than 2^32 elements: the last rows of y and dx are those of the
    formulas, the codes (both copies) those of the last rows of y."""
    rows, cols = 1 << 20, 4112                      # 8.6 GB of bf16
    bf = dict(dtype=BF, device=G.DEV)
    x = torch.zeros((rows, cols), **bf)
    tail = torch.randn((16, cols), generator=torch.Generator().manual_seed(4)).to(BF)
    x[-16:] = tail.to(G.DEV)
    w, b = _make(1, cols, BF, BF, 11)[1:3]
    wd, bd = w.to(G.DEV), b.to(G.DEV)
    G.say("layernorm past 32 bits", rows, cols)
    y, m, r = ops.fp8_layernorm_fwd(x, wd, bd)
    torch.cuda.synchronize()
    m64, r64, y64, dtol, rtol, ytol = _forward64(tail, w, b, False)
    _within(y[-16:], y64, ytol + _half(BF) * (np.abs(y64) + ytol), "y")
    _within(m[-16:], m64, dtol, "mean")
    assert torch.equal(y[5], bd)                    # a row of zeros gives the bias
    want = y[-16:].clone()
    del y
    dx, _, _ = ops.fp8_layernorm_bwd(x, x, wd, m, r, want_w=False, want_b=False)
    torch.cuda.synchronize()
    dx64, _, _, xt, _, _ = _backward64(tail, tail, w, m[-16:], r[-16:], False)
    _within(dx[-16:], dx64, xt + _half(BF) * (np.abs(dx64) + xt), "dx")
    assert not dx[:-16].any()
    del dx
    for rowwise in (False, True):
        G.say("layernorm quantize past 32 bits", rowwise)
        qz, _, _ = ops.fp8_layernorm_quantize(x, wd, bd, rowwise=rowwise)
        torch.cuda.synchronize()
        v = G.host(want)
        s = G.host(qz.scale)[-16:] if rowwise else G.host(qz.scale)
        st = G.host(qz.scale_t)
        f = oracle.bf16_to_f32(v)
        q = oracle.e4m3_encode((f * (s[:, None] if rowwise else s)).astype(np.float32).ravel())
        qt = oracle.e4m3_encode((f * st).astype(np.float32).ravel())
        assert np.array_equal(G.host(qz.q[-16:]).ravel(), q)
        assert np.array_equal(G.host(qz.qt[:, -16:].contiguous()).T.ravel(), qt)
        del qz


def test_given_stream_allocating():
    """A stream given to calls that allocate their outputs and workspaces."""
    x, w, b, dy = (t.to(G.DEV) for t in _make(64, 1040, BF, BF, 12))
    G.say("layernorm given stream")
    want = ops.fp8_layernorm_quantize(x, w, b)
    grads = ops.fp8_layernorm_bwd(dy, x, w, want[1], want[2])
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = ops.fp8_layernorm_quantize(x, w, b, stream=st)
    y, _, _ = ops.fp8_layernorm_fwd(x, w, b, stream=st)
    again = ops.fp8_layernorm_bwd(dy, x, w, got[1], got[2], stream=st)
    st.synchronize()
    assert torch.equal(got[0].q, want[0].q) and torch.equal(got[0].qt, want[0].qt)
    assert all(torch.equal(p, q) for p, q in zip(grads, again))
    assert torch.equal(ops.fp8_linear_quantize(y).q, want[0].q)
