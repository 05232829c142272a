"""GPU residual norm against the formulas in 64 bits.

Tolerances (u = 2^-24, one fp32 rounding; S = 86 u, the bound of a row sum
relative to its sum of magnitudes, and the bounds of a norm and of its
backward are derived in test_gpu_layernorm.py, whose functions are used here):

* s: the norm's bound with weight gate w and bias gate b, one more rounding
  for each of those products (u |xh gate w| + u |gate b|), the final
  alpha x + t within u |s| (fused), then the rounding to the stream's type.
* mean_pre, rstd_pre and y: the norm's bounds, from the s that was stored.
* dT: the norm's backward bound plus u |dT| for adding ds; call it D.  dx: D
  and one product, then the rounding to the stream's type.
* db: with h = dT gate w, |gate w| D + 2 u |h| enters the norm's backward, which
  is linear in h: e -> rstd (e + mean(e) + |xh| mean(|xh| e)).
* The sums over rows: (rows / 256 + 53) u of their sum of magnitudes, as for
  the layer norm (a thread's rows are at most rows / 256 and 16 row groups and
  32 partial rows follow), plus the sum of what D contributes.
"""
import numpy as np
import pytest
import torch

import oracle
from float8_mixed_precision_amd import ops
from tests import gpu_util as G
from tests.test_gpu_layernorm import BF, EPS, F32, S, U, _backward64, _d, _forward64, _half, _within

pytestmark = pytest.mark.gpu

SIZES = [(1, 1), (3, 5), (2, 7), (5, 8), (4, 9), (7, 100), (33, 513), (9, 1000), (3, 2050),
         (2, 4096), (3, 5001), (2, 8200), (2, 16383), (1, 16384), (1500, 136), (1100, 1001),
         (1040, 4096)]
NORMS = {"both": (True, True), "post": (True, False), "pre": (False, True)}


class Case:
    """Host inputs of one call and their device copies."""

    def __init__(self, rows, cols, dtype, pdtype, norms, seed, gate=True, ds=True):
        g = torch.Generator().manual_seed(seed)
        post, pre = NORMS[norms]
        rnd = lambda *shape: torch.randn(shape, generator=g)
        x = rnd(rows, cols) * 2 + 0.3
        x[:, ::64] *= 20.0                                   # outlier channels
        self.x, self.b = x.to(dtype), (rnd(rows, cols) * 1.5).to(BF)
        par = lambda base, dev: (base + dev * rnd(cols)).to(pdtype)
        self.post = (par(1, 0.3), par(0, 0.2)) if post else None
        self.pre = (par(1, 0.3), par(0, 0.2)) if pre else None
        self.gate = par(0.5, 0.3) if gate else None
        self.dy = (0.1 * rnd(rows, cols)).to(BF) if pre else None
        self.ds = (0.1 * rnd(rows, cols)).to(dtype) if ds or not pre else None
        dev = lambda t: None if t is None else tuple(map(dev, t)) if isinstance(t, tuple) else \
            t.to(G.DEV)
        self.dev = {n: dev(v) for n, v in vars(self).items()}

    def params(self):
        return {n: self.dev[n] for n in ("post", "pre", "gate")}


def _w(pair):
    return (None, None) if pair is None else pair


def _gated(c):
    """gate w and gate b of the post norm in 64 bits (b is None where it is 0)."""
    gate = np.ones(c.b.shape[1]) if c.gate is None else _d(c.gate)
    w, b = _w(c.post)
    return (gate if w is None else gate * _d(w)), (0 * gate if b is None else gate * _d(b))


def _stream64(c, alpha, rms, eps=EPS):
    """s in 64 bits and its tolerance before the rounding to the stream's type,
    with the post norm's (mean, rstd, tolerances)."""
    gw, gb = _gated(c)
    as_t = lambda a: torch.from_numpy(a)
    if c.post is None:
        t, ttol, stats = _d(c.b) * gw, U * np.abs(_d(c.b) * gw), None
    else:
        mean, rstd, t, dtol, rtol, ttol = _forward64(c.b, as_t(gw), as_t(gb), rms, eps)
        ttol = ttol + U * (np.abs(t - gb) + np.abs(gb))
        stats = (mean, rstd, dtol, rtol)
    s = alpha * _d(c.x) + t
    return s, ttol + U * np.abs(s), stats


def _grads64(c, s, stats, alpha, rms):
    """{name: (value, tolerance)} of the gradients, from the stored s and the
    statistics that the forward kernel left."""
    rows = c.b.shape[0]
    n = (rows / 256 + 53) * U
    r = {}
    dt = np.zeros(c.b.shape) if c.ds is None else _d(c.ds)
    D = 0 * dt
    if c.pre is not None:
        g, dw, db, D, wt, bt = _backward64(c.dy, s, c.pre[0], stats.mean_pre, stats.rstd_pre, rms)
        dt = dt + g
        D = D + U * np.abs(dt)
        r["dpre_weight"], r["dpre_bias"] = (dw, wt), (db, bt)
    r["dx"] = (alpha * dt, abs(alpha) * D + U * np.abs(alpha * dt))
    gate = np.ones(c.b.shape[1]) if c.gate is None else _d(c.gate)
    gw, _ = _gated(c)
    if c.post is None:
        b = _d(c.b)
        r["db"] = (dt * gw, np.abs(gw) * D + U * np.abs(dt * gw))
        r["dgate"] = ((dt * b).sum(0), n * np.abs(dt * b).sum(0) + (D * np.abs(b)).sum(0))
    else:
        db, _, _, tol, _, _ = _backward64(torch.from_numpy(dt), c.b, torch.from_numpy(gw),
                                          stats.mean_post, stats.rstd_post, rms)
        rs = _d(stats.rstd_post)[:, None]
        m = 0 if rms else _d(stats.mean_post)[:, None]
        xh = (_d(c.b) - m) * rs
        e = np.abs(gw) * D + 2 * U * np.abs(dt * gw)
        tol = tol + rs * (e + (0 if rms else e.mean(1, keepdims=True))
                          + np.abs(xh) * (np.abs(xh) * e).mean(1, keepdims=True))
        r["db"] = (db, tol)
        A, B = (dt * xh).sum(0), dt.sum(0)
        ea = n * np.abs(dt * xh).sum(0) + ((D + 3 * U * np.abs(dt)) * np.abs(xh)).sum(0)
        eb = n * np.abs(dt).sum(0) + D.sum(0)
        w, b = (np.ones_like(gate) if c.post[0] is None else _d(c.post[0]),
                0 * gate if c.post[1] is None else _d(c.post[1]))
        r["dpost_weight"] = (gate * A, np.abs(gate) * ea + U * np.abs(gate * A))
        r["dpost_bias"] = (gate * B, np.abs(gate) * eb + U * np.abs(gate * B))
        r["dgate"] = (w * A + b * B, np.abs(w) * ea + np.abs(b) * eb
                      + 3 * U * (np.abs(w * A) + np.abs(b * B)))
    if c.gate is None:
        r.pop("dgate", None)
    return r


def _check_grads(grads, want, dtype, label):
    for name, (v, tol) in want.items():
        got = getattr(grads, name)
        if name in ("dx", "db"):
            tol = tol + _half(got.dtype) * (np.abs(v) + tol)
        _within(got, v, tol, "%s %s" % (label, name))


def _run_forward(c, alpha, rms, dtype):
    rows, cols = c.b.shape
    guard = torch.full((rows + 3, cols), 77.0, dtype=dtype, device=G.DEV)
    guard_y = torch.full((rows + 3, cols), 77.0, dtype=BF, device=G.DEV)
    pre = c.pre is not None
    s, y, st = ops.fp8_resnorm_fwd(c.dev["b"], c.dev["x"], alpha=alpha, eps=EPS, rms=rms,
                                   s=guard[:rows], y=guard_y[:rows] if pre else None,
                                   **c.params())
    torch.cuda.synchronize()
    assert torch.all(guard[rows:] == 77.0) and torch.all(guard_y[rows:] == 77.0)
    return s, y, st


def _check_forward(c, s, y, st, alpha, rms, dtype):
    s64, stol, stats = _stream64(c, alpha, rms)
    _within(s, s64, stol + _half(dtype) * (np.abs(s64) + stol), "s")
    if stats is not None:
        if not rms:
            _within(st.mean_post, stats[0], stats[2], "mean_post")
        _within(st.rstd_post, stats[1], stats[3], "rstd_post")
    if c.pre is not None:
        m64, r64, y64, dtol, rtol, ytol = _forward64(s.cpu(), *c.pre, rms)
        if not rms:
            _within(st.mean_pre, m64, dtol, "mean_pre")
        _within(st.rstd_pre, r64, rtol, "rstd_pre")
        _within(y, y64, ytol + _half(BF) * (np.abs(y64) + ytol), "y")


@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
@pytest.mark.parametrize("dtype,pdtype", [(BF, BF), (F32, F32)], ids=["bf16", "f32"])
@pytest.mark.parametrize("norms", list(NORMS))
@pytest.mark.parametrize("shape", SIZES, ids=lambda s: "%dx%d" % s)
def test_forward_and_backward(shape, norms, dtype, pdtype, rms):
    rows, cols = shape
    if rows % 2:                                             # the mixed types too
        pdtype = F32 if pdtype == BF else BF
    c = Case(rows, cols, dtype, pdtype, norms, rows * 31 + cols, gate=cols % 3 != 0,
             ds=rows % 3 != 0)
    alpha = 1.0 if cols % 2 else -0.75
    G.say("resnorm", shape, norms, dtype, pdtype, "rms", rms)
    s, y, st = _run_forward(c, alpha, rms, dtype)
    _check_forward(c, s, y, st, alpha, rms, dtype)
    G.say("resnorm bwd", shape, norms, dtype, pdtype, "rms", rms)
    guard = torch.full((rows + 3, cols), 77.0, dtype=dtype, device=G.DEV)
    guard_b = torch.full((rows + 3, cols), 77.0, dtype=BF, device=G.DEV)
    new = lambda p: None if p is None else torch.full((cols,), float("nan"), device=G.DEV)
    grads = ops.ResNormGrads(guard[:rows], guard_b[:rows], new(c.gate), new(_w(c.post)[0]),
                             new(_w(c.post)[1]), new(_w(c.pre)[0]), new(_w(c.pre)[1]))
    ops.fp8_resnorm_bwd(c.dev["dy"], c.dev["ds"], c.dev["b"], s, st, alpha=alpha, rms=rms,
                        grads=grads, **c.params())
    torch.cuda.synchronize()
    assert torch.all(guard[rows:] == 77.0) and torch.all(guard_b[rows:] == 77.0)
    _check_grads(grads, _grads64(c, s.cpu(), st, alpha, rms), dtype, "%s" % (shape,))


@pytest.mark.parametrize("absent", ["weights", "biases", "all"])
def test_absent_parameters(absent):
    """A weight or gate that is not there is 1, a bias 0."""
    c = Case(37, 264, BF, BF, "both", 3, gate=absent != "all")
    for n in ("post", "pre"):
        w, b = getattr(c, n)
        pair = (None if absent != "biases" else w, None if absent != "weights" else b)
        setattr(c, n, pair)
        c.dev[n] = tuple(None if v is None else v.to(G.DEV) for v in pair)
    G.say("resnorm absent", absent)
    s, y, st = _run_forward(c, 0.5, False, BF)
    _check_forward(c, s, y, st, 0.5, False, BF)
    grads = ops.fp8_resnorm_bwd(c.dev["dy"], c.dev["ds"], c.dev["b"], s, st, alpha=0.5,
                                **c.params())
    torch.cuda.synchronize()
    want = _grads64(c, s.cpu(), st, 0.5, False)
    for n in ("post", "pre"):
        for p, v in zip(("weight", "bias"), getattr(c, n)):
            if v is None:
                assert getattr(grads, "d%s_%s" % (n, p)) is None
                del want["d%s_%s" % (n, p)]
    _check_grads(grads, want, BF, absent)


@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
@pytest.mark.parametrize("norms", list(NORMS))
def test_gradients_against_differences(norms, rms):
    """Directional derivatives of sum(y dy) + sum(s ds) by central differences of
    the 64-bit forward (step 1e-4: truncation about 1e-8 of the value), against
    the kernel's gradients along the same directions."""
    rows, cols = 6, 520
    c = Case(rows, cols, F32, F32, norms, 5)
    alpha = 0.75
    c.x = c.x / 4
    c.dev["x"] = c.x.to(G.DEV)
    G.say("resnorm differences", norms, "rms", rms)
    s, y, st = ops.fp8_resnorm_fwd(c.dev["b"], c.dev["x"], alpha=alpha, rms=rms, **c.params())
    grads = ops.fp8_resnorm_bwd(c.dev["dy"], c.dev["ds"], c.dev["b"], s, st, alpha=alpha, rms=rms,
                                **c.params())
    torch.cuda.synchronize()
    rng = np.random.default_rng(3)
    h = 1e-4
    names = {"dx": "x", "db": "b", "dgate": "gate", "dpost_weight": ("post", 0),
             "dpost_bias": ("post", 1), "dpre_weight": ("pre", 0), "dpre_bias": ("pre", 1)}
    tols = _grads64(c, s.cpu(), st, alpha, rms)

    class Moved:
        pass

    for name, where in names.items():
        gk = getattr(grads, name)
        if gk is None:
            continue
        v = rng.standard_normal(tuple(gk.shape))

        def loss(sign):
            m = Moved()
            step = sign * h * torch.from_numpy(v)
            for n in ("x", "b", "gate", "post", "pre"):
                t = getattr(c, n)
                if t is not None:
                    t = tuple(p.double() for p in t) if isinstance(t, tuple) else t.double()
                    if where == n:
                        t = t + step
                    elif isinstance(where, tuple) and where[0] == n:
                        t = tuple(p + step if k == where[1] else p for k, p in enumerate(t))
                setattr(m, n, t)
            s64 = _stream64(m, alpha, rms)[0]
            value = float((s64 * _d(c.ds)).sum())
            if c.pre is not None:
                value += float((_forward64(torch.from_numpy(s64), *m.pre, rms)[2]
                                * _d(c.dy)).sum())
            return value

        diff = (loss(1) - loss(-1)) / (2 * h)
        got = float((_d(gk) * v).sum())
        tol = tols[name][1] + (_half(gk.dtype) * np.abs(tols[name][0])
                               if name in ("dx", "db") else 0)
        # s and the statistics as the forward kernel left them are within 1e-5 of
        # exact
        allowed = float((tol * np.abs(v)).sum()) + 1e-5 * float((np.abs(_d(gk) * v)).sum())
        assert abs(got - diff) <= allowed, (name, got, diff, allowed)


def _hq(z):
    return tuple(G.host(t) for t in (z.q, z.qt, z.scale, z.scale_t, z.amax))


Q_SIZES = [(16, 16), (272, 400), (48, 4112), (1040, 80), (528, 784), (32, 16384), (1088, 8208),
           (4096, 4096)]


@pytest.mark.parametrize("norms", ["both", "pre"])
@pytest.mark.parametrize("rowwise", [False, True], ids=["tensorwise", "rowwise"])
@pytest.mark.parametrize("shape", Q_SIZES, ids=lambda s: "%dx%d" % s)
def test_quantize(shape, rowwise, norms):
    """s and the statistics are the forward's, the codes the oracle's quantize
    of its y, bit for bit, whether y is stored or not; of an fp32 stream too."""
    rows, cols = shape
    rms = rows % 32 == 0
    for dtype in (BF, F32):
        c = Case(rows, cols, dtype, BF, norms, cols + 1)
        G.say("resnorm quantize", shape, "rowwise", rowwise, norms, dtype)
        s0, y0, st0 = ops.fp8_resnorm_fwd(c.dev["b"], c.dev["x"], alpha=0.9, rms=rms,
                                          **c.params())
        ws = ops.alloc_resnorm_workspace(rows, cols, G.DEV, rowwise).fill_(0x7F)
        ref = None
        for y in (torch.empty_like(y0), None):
            if y is None and dtype == F32:
                continue
            s, z, st = ops.fp8_resnorm_quantize(c.dev["b"], c.dev["x"], alpha=0.9, rms=rms,
                                                rowwise=rowwise, y=y, workspace=ws, **c.params())
            torch.cuda.synchronize()
            assert torch.equal(s, s0)
            for n in ops.ResNormStats.__slots__:
                p, q = getattr(st, n), getattr(st0, n)
                assert (p is None and q is None) or torch.equal(p, q), n
            if y is not None:
                assert torch.equal(y.view(torch.int16), y0.view(torch.int16))
            ref = oracle.quantize(G.host(y0), rowwise) if ref is None else ref
            G.assert_quantize_equal(_hq(z), ref, "codes of y %s" % (shape,))


@pytest.mark.parametrize("norms", ["both", "pre"])
@pytest.mark.parametrize("shape", [(1, 16), (1, 4096), (3, 16384), (17, 400), (50, 8192),
                                   (1025, 2064)], ids=lambda s: "%dx%d" % s)
def test_quantize_rows(shape, norms):
    """The serving form: any number of rows, any stream."""
    rows, cols = shape
    for dtype in (BF, F32):
        c = Case(rows, cols, dtype, F32, norms, cols + 2)
        G.say("resnorm quantize rows", shape, norms, dtype)
        s0, y0, st0 = ops.fp8_resnorm_fwd(c.dev["b"], c.dev["x"], rms=True, **c.params())
        call = lambda **k: ops.fp8_resnorm_quantize(c.dev["b"], c.dev["x"], rms=True, rowwise=True,
                                                    transposed=False, **c.params(), **k)
        y = torch.empty_like(y0)
        s1, z1, st1 = call(y=y)
        s2, z2, st2 = call(want_stats=False)
        torch.cuda.synchronize()
        assert st2 is None and torch.equal(st1.rstd_pre, st0.rstd_pre)
        assert torch.equal(s1, s0) and torch.equal(s2, s0)
        assert torch.equal(y.view(torch.int16), y0.view(torch.int16))
        pad = np.zeros(((rows + 15) // 16 * 16, cols), np.uint16)
        pad[:rows] = G.host(y0)
        ref = oracle.quantize(pad, True)
        for z in (z1, z2):
            assert np.array_equal(G.host(z.q), ref[0][:rows])
            assert np.array_equal(G.host(z.scale), ref[2][:rows])
            assert np.array_equal(G.host(z.amax), ref[4][:rows])


@pytest.mark.parametrize("e5m2", [False, True], ids=["e4m3", "e5m2"])
@pytest.mark.parametrize("rowwise", [False, True], ids=["tensorwise", "rowwise"])
@pytest.mark.parametrize("shape", Q_SIZES, ids=lambda s: "%dx%d" % s)
def test_backward_quantize(shape, rowwise, e5m2):
    """With the codes of db: every gradient is the one without them, bit for
    bit, and the codes are the oracle's quantize of db."""
    rows, cols = shape
    norms = list(NORMS)[(rows // 16 + cols // 16) % 3]
    for dtype in (BF, F32):
        c = Case(rows, cols, dtype, BF, norms, cols + 3)
        G.say("resnorm bwd quantize", shape, "rowwise", rowwise, "e5m2", e5m2, norms, dtype)
        s, _, st = ops.fp8_resnorm_fwd(c.dev["b"], c.dev["x"], **c.params())
        args = (c.dev["dy"], c.dev["ds"], c.dev["b"], s, st)
        plain = ops.fp8_resnorm_bwd(*args, **c.params())
        ws = ops.alloc_resnorm_workspace(rows, cols, G.DEV, rowwise).fill_(0x7F)
        z = ops.alloc_quantized(rows, cols, rowwise, G.DEV)
        grads = ops.fp8_resnorm_bwd(*args, out=z, rowwise=rowwise, e5m2=e5m2, workspace=ws,
                                    **c.params())
        torch.cuda.synchronize()
        for n in ops.ResNormGrads.__slots__:
            p, q = getattr(plain, n), getattr(grads, n)
            assert (p is None and q is None) or torch.equal(p, q), n
        quantize = oracle.quantize_e5m2 if e5m2 else oracle.quantize
        ref = quantize(G.host(grads.db), rowwise)
        G.assert_quantize_equal(_hq(z), ref, "codes of db %s" % (shape,))


def test_constant_and_nonfinite_rows():
    """A block output of equal values normalizes to the bias; an infinity or a
    NaN in b or x stays in its own row."""
    cols = 1200
    c = Case(7, cols, F32, F32, "both", 2)
    c.b[1] = 3.0
    c.b[2, 7] = float("inf")
    c.b[3, 1199] = float("nan")
    c.x[4, 8] = float("-inf")
    c.x[5, 0] = float("nan")
    c.dev["b"], c.dev["x"] = c.b.to(G.DEV), c.x.to(G.DEV)
    G.say("resnorm special rows")
    s, y, st = ops.fp8_resnorm_fwd(c.dev["b"], c.dev["x"], **c.params())
    torch.cuda.synchronize()
    s, y = s.cpu(), y.cpu()
    assert torch.equal(s[1], c.x[1] + c.gate * c.post[1])
    assert torch.isnan(s[2, 7]) and torch.isnan(s[3]).all() and torch.isnan(y[2:6].float()).any(1).all()
    assert torch.isinf(s[4, 8]) and torch.isnan(s[5, 0]) and torch.isfinite(s[5, 1:]).all()
    s64, stol, _ = _stream64(c, 1.0, False)
    for r in (0, 6):
        assert np.all(np.abs(_d(s[r]) - s64[r]) <= stol[r] + U * (np.abs(s64[r]) + stol[r]))
        assert torch.isfinite(y[r].float()).all()


@pytest.mark.parametrize("rowwise", [False, True], ids=["tensorwise", "rowwise"])
def test_empty(rowwise):
    e = torch.empty((0, 64), dtype=BF, device=G.DEV)
    w = torch.ones(64, dtype=BF, device=G.DEV)
    G.say("resnorm empty", rowwise)
    s, y, st = ops.fp8_resnorm_fwd(e, e, (w, w), (w, w), w)
    _, z, _ = ops.fp8_resnorm_quantize(e, e, None, (w, w), rowwise=rowwise)
    zb = ops.alloc_quantized(0, 64, rowwise, G.DEV)
    g = ops.fp8_resnorm_bwd(e, None, e, s, st, (w, w), (w, w), w, out=zb, rowwise=rowwise)
    torch.cuda.synchronize()
    assert s.shape == y.shape == g.dx.shape == g.db.shape == (0, 64)
    for n in ops.ResNormGrads.__slots__[2:]:
        assert torch.all(getattr(g, n) == 0), n
    for q in (z, zb):
        assert torch.all(q.scale_t == float(oracle.scale_from_amax(0.0)))


def test_skipped_gradients_and_repeatability():
    rows, cols = 700, 1032
    c = Case(rows, cols, BF, BF, "both", 9)
    G.say("resnorm partial gradients")
    s, _, st = ops.fp8_resnorm_fwd(c.dev["b"], c.dev["x"], **c.params())
    args = (c.dev["dy"], c.dev["ds"], c.dev["b"], s, st)
    full = ops.fp8_resnorm_bwd(*args, **c.params())
    names = ops.ResNormGrads.__slots__
    for keep in (names, ("db",), ("db", "dx"), ("db", "dgate"), ("db", "dpost_bias"),
                 ("db", "dpre_weight"), ("db", "dpre_bias", "dpost_weight")):
        g = ops.ResNormGrads(**{n: torch.empty_like(getattr(full, n)) for n in keep})
        ops.fp8_resnorm_bwd(*args, grads=g, **c.params())
        torch.cuda.synchronize()
        for n in names:
            assert (getattr(g, n) is None) == (n not in keep)
            assert n not in keep or torch.equal(getattr(g, n), getattr(full, n)), (keep, n)


def test_side_stream_and_graph():
    """The same results on a stream of its own and from two captured graphs that
    share the workspace, replayed in turn with eager work between."""
    rows, cols = 96, 1040
    c = Case(rows, cols, BF, BF, "both", 10)
    ws = ops.alloc_resnorm_workspace(rows, cols, G.DEV, True)
    zy, zb = (ops.alloc_quantized(rows, cols, True, G.DEV) for _ in range(2))
    st = ops.alloc_resnorm_stats(rows, G.DEV)
    s = torch.empty((rows, cols), dtype=BF, device=G.DEV)
    new = lambda: torch.empty(cols, device=G.DEV)
    grads = ops.ResNormGrads(torch.empty_like(s), torch.empty_like(s), new(), new(), new(), new(),
                             new())

    def forward():
        ops.fp8_resnorm_quantize(c.dev["b"], c.dev["x"], rowwise=True, s=s, out=zy, stats=st,
                                 workspace=ws, **c.params())

    def backward():
        ops.fp8_resnorm_bwd(c.dev["dy"], c.dev["ds"], c.dev["b"], s, st, grads=grads, out=zb,
                            rowwise=True, e5m2=True, workspace=ws, **c.params())

    def results():
        torch.cuda.synchronize()
        return [t.clone() for z in (zy, zb) for t in (z.q, z.qt, z.scale, z.scale_t)] + [
            getattr(grads, n).clone() for n in ops.ResNormGrads.__slots__] + [s.clone()]

    forward(), backward()
    want = results()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        forward(), backward()
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(results(), want))
    graphs = []
    for f in (forward, backward):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            f()
    for k in range(3):
        c.dev["x"].add_(0.25 * k)
        forward(), backward()
        want = results()
        s.zero_()
        for g in graphs:
            g.replay()
        assert all(torch.equal(p, q) for p, q in zip(results(), want)), k


def test_offsets_past_32_bits():
    """A bf16 stream of more than 2^32 bytes: its last rows are those of a call
    on them alone."""
    cols = 4096
    rows = (1 << 31) // cols + 48
    c = Case(64, cols, BF, BF, "both", 12)
    G.say("resnorm past 2^32 bytes", rows)
    tile = lambda t: t.repeat(rows // 64 + 1, 1)[:rows]
    big = {n: tile(c.dev[n]) for n in ("b", "x", "dy", "ds")}
    for n in ("b", "x", "dy"):
        big[n][-16:] = big[n][:16].flip(1)
    s, y, st = ops.fp8_resnorm_fwd(big["b"], big["x"], rms=True, **c.params())
    g = ops.fp8_resnorm_bwd(big["dy"], big["ds"], big["b"], s, st, rms=True, **c.params())
    last = lambda t: t[-16:].clone()
    s1, y1, st1 = ops.fp8_resnorm_fwd(last(big["b"]), last(big["x"]), rms=True, **c.params())
    g1 = ops.fp8_resnorm_bwd(last(big["dy"]), last(big["ds"]), last(big["b"]), s1, st1, rms=True,
                             **c.params())
    torch.cuda.synchronize()
    for p, q in ((s, s1), (y, y1), (st.rstd_post, st1.rstd_post), (st.rstd_pre, st1.rstd_pre),
                 (g.dx, g1.dx), (g.db, g1.db)):
        assert torch.equal(p[-16:], q)
