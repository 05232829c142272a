"""Residual norm entry points: the calls that the library and the binding
refuse on the host, before anything is enqueued (fake device addresses, so
only where no GPU is visible), and the workspace sizes."""
import ctypes

import pytest
import torch

from float8_mixed_precision_amd import ops as E

A, BAD, BAD4 = 0x10000, 0x10008, 0x10002
P = lambda v: ctypes.c_void_p(v) if v else None
no_gpu = pytest.mark.skipif(torch.cuda.device_count() != 0,
                            reason="fake-pointer cases run without a GPU only")
OPERANDS = ("b", "x", "pw", "pb", "qw", "qb", "gate", "s", "y")
STATS = ("mp", "rp", "mq", "rq")
GRADS = ("dx", "db", "dgate", "dpw", "dpb", "dqw", "dqb")


def desc(d):
    z = lambda n: d[n] or 0
    return E._RESNORM.pack(d["rows"], d["cols"], d["kind"], d["norms"], d["dtype"], d["pdtype"],
                           d["alpha"], d["eps"], *(z(n) for n in OPERANDS + STATS))


def _d(k, **base):
    d = dict(rows=16, cols=32, kind=0, norms=3, dtype=0, pdtype=0, alpha=1.0, eps=1e-5,
             **{n: A for n in OPERANDS + STATS})
    d.update(base)
    d.update(k)
    return d


def fwd(**k):
    return E.lib().fp8_resnorm_fwd(desc(_d(k)), None)


def quant(**k):
    d = _d(k, y=k.get("y"))
    d = dict(dict(scaling=0, q=A, qt=A, sc=A, st=A, amax=None, ws=A, wsb=1 << 26), **d)
    return E.lib().fp8_resnorm_quantize(desc(d), d["scaling"], P(d["q"]), P(d["qt"]), P(d["sc"]),
                                        P(d["st"]), P(d["amax"]), P(d["ws"]), d["wsb"], None)


def bwd(**k):
    d = dict(dict(scaling=0, dy=A, ds=A, q=A, qt=A, sc=A, st=A, amax=None, ws=A, wsb=1 << 26,
                  **{n: A for n in GRADS}), **_d(k))
    g = E._RESNORM_GRADS.pack(*(d[n] or 0 for n in GRADS))
    return E.lib().fp8_resnorm_bwd(desc(d), P(d["dy"]), P(d["ds"]), g, d["scaling"], P(d["q"]),
                                   P(d["qt"]), P(d["sc"]), P(d["st"]), P(d["amax"]), P(d["ws"]),
                                   d["wsb"], None)


CALLS = pytest.mark.parametrize("call", [fwd, quant, bwd], ids=["fwd", "quantize", "bwd"])


@no_gpu
@CALLS
def test_shared_refusals(call):
    for k in (dict(kind=2), dict(kind=-1), dict(dtype=2), dict(pdtype=2), dict(norms=0),
              dict(norms=4), dict(norms=-1), dict(alpha=float("nan")), dict(alpha=float("inf")),
              dict(b=None), dict(s=None)):
        assert call(**k) == E.FP8L_EINVAL, k
    for k in (dict(rows=-16), dict(rows=1 << 31), dict(cols=0), dict(cols=16400)):
        assert call(**k) == E.FP8L_ESHAPE, k
    for n in ("b", "pw", "pb", "qw", "qb", "gate", "s"):
        assert call(**{n: BAD}) == E.FP8L_EALIGN, n
    for n in STATS:
        assert call(**{n: BAD4}) == E.FP8L_EALIGN, n
    L = E.lib()
    if call is fwd:
        assert L.fp8_resnorm_fwd(None, None) == E.FP8L_EINVAL


@no_gpu
def test_fwd_refusals():
    for eps in (-1e-5, float("nan"), float("inf")):
        assert fwd(eps=eps) == E.FP8L_EINVAL and quant(eps=eps) == E.FP8L_EINVAL
    assert fwd(x=None) == E.FP8L_EINVAL and fwd(y=None) == E.FP8L_EINVAL
    assert fwd(x=BAD) == E.FP8L_EALIGN and fwd(y=BAD) == E.FP8L_EALIGN
    none = dict.fromkeys(OPERANDS + STATS)
    assert fwd(rows=0, **none) == E.FP8L_OK                  # nothing to do


@no_gpu
def test_quantize_refusals():
    for scaling in (2, 3, -1):
        assert quant(scaling=scaling) == E.FP8L_EINVAL       # E4M3 only
    for scaling in (0, 1):
        c = lambda **k: quant(scaling=scaling, **k)
        assert c(norms=1) == E.FP8L_EINVAL                   # no y to quantize
        assert c(rows=17) == E.FP8L_ESHAPE and c(cols=24) == E.FP8L_ESHAPE
        for n in ("x", "q", "sc", "st", "rq", "mq", "ws"):
            assert c(**{n: None}) == E.FP8L_EINVAL, n
        assert c(dtype=1) == E.FP8L_EINVAL                   # an fp32 stream needs y
        need = E.lib().fp8_resnorm_workspace_bytes(16, 32, scaling)
        assert c(wsb=need - 1) == E.FP8L_EWORKSPACE
        for n in ("ws", "q", "qt", "y"):
            assert c(**{n: BAD}) == E.FP8L_EALIGN, n
        for n in ("sc", "st", "amax"):
            assert c(**{n: BAD4}) == E.FP8L_EALIGN, n
    assert quant(qt=None) == E.FP8L_EINVAL                   # tensorwise needs qt
    rows_only = dict(scaling=1, qt=None, st=None, ws=None, wsb=0, **dict.fromkeys(STATS))
    assert quant(rows=17, cols=24, **rows_only) == E.FP8L_ESHAPE
    assert quant(rows=17, sc=None, **rows_only) == E.FP8L_EINVAL
    assert quant(rows=0, b=None, x=None, s=None, q=None, sc=None, **rows_only) == E.FP8L_OK


@no_gpu
def test_bwd_refusals():
    for scaling in (4, 5, -1):
        assert bwd(scaling=scaling) == E.FP8L_EINVAL
    for scaling in (0, 1, 2, 3):
        c = lambda **k: bwd(scaling=scaling, **k)
        for n in ("db", "dy", "rp", "mp", "rq", "mq", "q", "qt", "sc", "st", "ws"):
            assert c(**{n: None}) == E.FP8L_EINVAL, n
        assert c(rows=17) == E.FP8L_ESHAPE and c(cols=24) == E.FP8L_ESHAPE
        need = E.lib().fp8_resnorm_workspace_bytes(16, 32, scaling)
        assert c(wsb=need - 1) == E.FP8L_EWORKSPACE
        for n in ("dy", "ds", "dx", "db", "q", "qt", "ws"):
            assert c(**{n: BAD}) == E.FP8L_EALIGN, n
        for n in ("sc", "st", "amax", "dgate", "dpw", "dpb", "dqw", "dqb"):
            assert c(**{n: BAD4}) == E.FP8L_EALIGN, n
    # what a norm that is not there would give is refused, as is a stream
    # without any gradient
    plain = dict(q=None, qt=None, sc=None, st=None)
    assert bwd(norms=1, dqw=None, dqb=None, **plain) == E.FP8L_EINVAL           # dy without pre
    assert bwd(norms=1, dy=None, dqw=None, dqb=None, ds=None, **plain) == E.FP8L_EINVAL
    assert bwd(norms=1, dy=None, dqb=None, **plain) == E.FP8L_EINVAL
    assert bwd(norms=2, dpw=None, **plain) == E.FP8L_EINVAL
    assert bwd(gate=None, **plain) == E.FP8L_EINVAL
    assert bwd(ws=None, **plain) == E.FP8L_EINVAL            # the parameters' gradients
    g = E._RESNORM_GRADS.pack(*([A] * 7))
    assert E.lib().fp8_resnorm_bwd(None, P(A), P(A), g, 0, None, None, None, None, None, None, 0,
                                   None) == E.FP8L_EINVAL
    assert E.lib().fp8_resnorm_bwd(desc(_d({})), P(A), P(A), None, 0, None, None, None, None, None,
                                   None, 0, None) == E.FP8L_EINVAL


def test_workspace_bytes():
    f = E.lib().fp8_resnorm_workspace_bytes
    assert f(8, 0, 0) == 0 and f(-1, 16, 0) == 0 and f(8, 16385, 0) == 0 and f(8, 16, 4) == 0
    for scaling in (0, 1, 2, 3):
        last = 0
        for rows in (0, 1, 16, 17, 400, 8192, 1 << 20):
            n = f(rows, 4096, scaling)
            # four sums of each of 256 workgroups, and the maxima
            need = 256 * 4 * 4096 * 4 + ((2 * rows + 256 * 2 * 4096) if scaling & 1 else 4 * 2048)
            assert n % 256 == 0 and n >= need and n >= last
            last = n


@no_gpu
def test_every_output_apart_from_every_buffer():
    """An output (or the workspace) that meets any other buffer of its call is
    refused.  (Fake addresses, 2^24 bytes apart.)"""
    def check(call, names, outs):
        apart = {n: A + (k << 24) for k, n in enumerate(names)}
        for one in outs:
            for other in apart:
                if other != one:
                    assert call(**dict(apart, **{one: apart[other]})) == E.FP8L_EINVAL, (one, other)
        if "ws" in apart:
            for other in apart:
                if other != "ws":
                    inside = dict(apart, **{other: apart["ws"] + 64})
                    assert call(**inside) == E.FP8L_EINVAL, (other, "in the workspace")

    check(fwd, OPERANDS + STATS, ("s", "y") + STATS)
    codes = ("q", "qt", "sc", "st", "amax")
    for scaling in (0, 1):
        check(lambda **k: quant(scaling=scaling, **k), OPERANDS + STATS + codes + ("ws",),
              ("s", "y") + STATS + codes + ("ws",))
    check(lambda **k: quant(scaling=1, qt=None, st=None, ws=None, wsb=0, **k),
          OPERANDS + STATS + ("q", "sc", "amax"), ("s", "y") + STATS + ("q", "sc", "amax"))
    read = tuple(n for n in OPERANDS if n not in ("x", "y")) + STATS + ("dy", "ds")
    for scaling in (0, 1, 2, 3):
        check(lambda **k: bwd(scaling=scaling, **k), read + GRADS + codes + ("ws",),
              GRADS + codes + ("ws",))


def test_binding_refusals():
    """The binding checks types, shapes, contiguity and which norms there are
    before the call."""
    bf, f32 = torch.bfloat16, torch.float32
    x = torch.zeros((16, 32), dtype=bf)
    w, r = torch.zeros(32, dtype=bf), torch.zeros(16)
    n = (w, w)
    st = E.ResNormStats(r, r, r, r)
    z = E.alloc_quantized(16, 32, False, "cpu")
    bad = [
        lambda: E.fp8_resnorm_fwd(x, x),                             # no norm at all
        lambda: E.fp8_resnorm_fwd(x.float(), x, n),
        lambda: E.fp8_resnorm_fwd(x, x.half(), n),
        lambda: E.fp8_resnorm_fwd(x, x[:8], n),
        lambda: E.fp8_resnorm_fwd(x.t(), x, n),
        lambda: E.fp8_resnorm_fwd(x, x, n, (w.float(), None)),       # mixed parameter types
        lambda: E.fp8_resnorm_fwd(x, x, n, gate=w[:16]),
        lambda: E.fp8_resnorm_fwd(x, x, n, s=x.float()),
        lambda: E.fp8_resnorm_fwd(x, x, n, y=x),                     # y without a pre norm
        lambda: E.fp8_resnorm_fwd(x, x, n, n, stats=E.ResNormStats(r[:8])),
        lambda: E.fp8_resnorm_quantize(x, x, n, None),
        lambda: E.fp8_resnorm_quantize(x, x, n, n, transposed=False),
        lambda: E.fp8_resnorm_quantize(x, x.float(), n, n),          # fp32 stream without y
        lambda: E.fp8_resnorm_quantize(x, x, n, n, out=E.alloc_quantized(16, 16, False, "cpu")),
        lambda: E.fp8_resnorm_quantize(x, x, n, n, out=E.Quantized(z.q, None, z.scale, z.scale_t,
                                                                  z.amax)),
        lambda: E.fp8_resnorm_bwd(x.float(), x, x, x, st, n, n),
        lambda: E.fp8_resnorm_bwd(x, x.float(), x, x, st, n, n),
        lambda: E.fp8_resnorm_bwd(x, x, x, x, E.ResNormStats(r, r.double()), n, n),
        lambda: E.fp8_resnorm_bwd(x, x, x, x, st, n, n, grads=E.ResNormGrads(x, x, dgate=w)),
        lambda: E.fp8_resnorm_bwd(x, x, x, x, st, n, n, out=E.Quantized(z.q, z.qt, None, z.scale_t,
                                                                        None)),
    ]
    good = [lambda: E.fp8_resnorm_fwd(x, x, n), lambda: E.fp8_resnorm_quantize(x, x, None, n),
            lambda: E.fp8_resnorm_bwd(x, None, x, x, st, n, n)]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError, match="must (be|have)|rowwise") as e:
            call()
        print(k, e.value)
    for call in good:                    # nothing wrong but the device
        with pytest.raises(ValueError, match="on a GPU"):
            call()
