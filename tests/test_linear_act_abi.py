"""Entry points of the linear with its epilogue: the calls that the library and
the binding refuse on the host, before anything is enqueued (fake device
addresses, so only where no GPU is visible), the workspace sizes, and the
stated errors of the activations."""
import ctypes
import itertools

import numpy as np
import pytest
import torch
from scipy.special import ndtr

from float8_mixed_precision_amd import ops as E

A, BAD, BAD4 = 0x10000, 0x10008, 0x10002
P = lambda v: ctypes.c_void_p(v) if v else None
no_gpu = pytest.mark.skipif(torch.cuda.device_count() != 0,
                            reason="fake-pointer cases run without a GPU only")


def fwd(x=A, sx=A, w=A, sw=A, M=16, N=32, K=48, scaling=0, bias=A, pdtype=0, act=2, res=None,
        z=A, y=A, q=A, qt=A, s=A, st=A, amax=None, ws=A, wsb=1 << 26):
    return E.lib().fp8_linear_act_fwd(P(x), P(sx), P(w), P(sw), M, N, K, scaling, P(bias), pdtype,
                                      act, P(res), P(z), P(y), P(q), P(qt), P(s), P(st), P(amax),
                                      P(ws), wsb, None)


def bwd(dy=A, sdy=A, w=A, sw=A, z=A, M=16, N=32, K=48, scaling=0, act=2, dz=A, q=A, qt=A, s=A,
        st=A, amax=None, db=A, pdtype=0, ws=A, wsb=1 << 26):
    return E.lib().fp8_linear_act_bwd(P(dy), P(sdy), P(w), P(sw), P(z), M, N, K, scaling, act,
                                      P(dz), P(q), P(qt), P(s), P(st), P(amax), P(db), pdtype,
                                      P(ws), wsb, None)


def ebwd(dy=A, z=A, M=16, N=32, scaling=0, act=2, dz=A, q=A, qt=A, s=A, st=A, amax=None, db=A,
         pdtype=0, ws=A, wsb=1 << 26):
    return E.lib().fp8_bias_act_bwd(P(dy), P(z), M, N, scaling, act, P(dz), P(q), P(qt), P(s),
                                    P(st), P(amax), P(db), pdtype, P(ws), wsb, None)


NONE = dict(q=None, qt=None, s=None, st=None)


@no_gpu
@pytest.mark.parametrize("call", [fwd, bwd, ebwd], ids=["fwd", "bwd", "bias_bwd"])
def test_shared_refusals(call):
    for scaling in (4, 5, -1) + ((2, 3) if call is fwd else ()):
        assert call(scaling=scaling) == E.FP8L_EINVAL
    for scaling in (0, 1) if call is fwd else (0, 1, 2, 3):
        c = lambda **k: call(scaling=scaling, **k)
        for act in (-1, 6):
            assert c(act=act) == E.FP8L_EINVAL
        assert c(pdtype=2) == E.FP8L_EINVAL
        assert c(N=24) == E.FP8L_ESHAPE and c(N=-16) == E.FP8L_ESHAPE
        assert c(M=17) == E.FP8L_ESHAPE and c(M=-16) == E.FP8L_ESHAPE
        for n in ("q", "qt", "s", "ws"):
            if not (call is fwd and scaling == 1 and n == "qt"):
                assert c(**{n: None}) == E.FP8L_EINVAL, n
        assert c(st=None) == E.FP8L_EINVAL
        need = E.lib().fp8_linear_act_workspace_bytes(16, 32, scaling)
        assert c(wsb=need - 1) == E.FP8L_EWORKSPACE
        for n in ("z", "q", "qt", "ws"):
            assert c(**{n: BAD}) == E.FP8L_EALIGN, n
        for n in ("s", "st", "amax"):
            assert c(**{n: BAD4}) == E.FP8L_EALIGN, n


@no_gpu
def test_fwd_refusals():
    for scaling in (0, 1):
        c = lambda **k: fwd(scaling=scaling, **k)
        assert c(K=24) == E.FP8L_ESHAPE and c(K=-16) == E.FP8L_ESHAPE
        assert c(M=1 << 20, K=1 << 12) == E.FP8L_ESHAPE      # 2^32 bytes of codes
        assert c(N=1 << 20, K=1 << 12) == E.FP8L_ESHAPE
        assert c(M=1 << 16, N=1 << 15) == E.FP8L_ESHAPE
        for n in ("x", "sx", "w", "sw"):
            assert c(**{n: None}) == E.FP8L_EINVAL, n
        for n in ("x", "w", "bias", "res", "y"):
            assert c(**{n: BAD}) == E.FP8L_EALIGN, n
        for n in ("sx", "sw"):
            assert c(**{n: BAD4}) == E.FP8L_EALIGN, n
        # y may be left out only where z and codes are written, and nothing is added
        assert c(y=None, z=None) == E.FP8L_EINVAL
        assert c(y=None, res=A + (1 << 20)) == E.FP8L_EINVAL
        assert c(y=None, **NONE) == E.FP8L_EINVAL
        # an amax alone is a quantize without its outputs
        assert c(amax=A, **NONE) == E.FP8L_EINVAL
        assert c(M=0, x=None, sx=None, y=None, z=None, **NONE) == E.FP8L_EINVAL  # scales of w
    # codes of the rows alone are rowwise, with neither qt nor scale_t
    assert fwd(qt=None, st=None) == E.FP8L_EINVAL
    rows = dict(scaling=1, qt=None, st=None, M=17)
    assert fwd(s=None, **rows) == E.FP8L_EINVAL and fwd(q=None, **rows) == E.FP8L_EINVAL
    assert fwd(q=BAD, **rows) == E.FP8L_EALIGN and fwd(s=BAD4, **rows) == E.FP8L_EALIGN
    assert fwd(scaling=1, qt=None) == E.FP8L_EINVAL          # scale_t without qt
    assert fwd(scaling=1, st=None) == E.FP8L_EINVAL          # qt without scale_t


@no_gpu
def test_bwd_refusals():
    for scaling in (0, 1, 2, 3):
        c = lambda **k: bwd(scaling=scaling, **k)
        assert c(K=24) == E.FP8L_ESHAPE and c(M=1 << 16, N=1 << 15) == E.FP8L_ESHAPE
        for n in ("dy", "sdy", "w", "sw", "z", "dz"):
            assert c(**{n: None}) == E.FP8L_EINVAL, n
        for n in ("dy", "w", "dz", "db"):
            assert c(**{n: BAD}) == E.FP8L_EALIGN, n
        for n in ("sdy", "sw"):
            assert c(**{n: BAD4}) == E.FP8L_EALIGN, n
        c = lambda **k: ebwd(scaling=scaling, **k)
        for n in ("dy", "z", "dz"):
            assert c(**{n: None}) == E.FP8L_EINVAL, n
        for n in ("dy", "dz", "db"):
            assert c(**{n: BAD}) == E.FP8L_EALIGN, n
        assert c(M=1 << 29, N=1 << 10) == E.FP8L_ESHAPE


@no_gpu
def test_every_output_apart_from_every_buffer():
    """An output (or the workspace) that meets any other buffer of its call is
    refused, but for the residual that is y.  (Fake addresses, 2^24 bytes apart.)"""
    def check(call, names, outs, allowed=()):
        names, outs = names.split(), outs.split()
        apart = {n: A + (k << 24) for k, n in enumerate(names)}
        for one in outs:
            for other in apart:
                if other != one and (one, other) not in allowed:
                    assert call(**dict(apart, **{one: apart[other]})) == E.FP8L_EINVAL, (one, other)
        for other in apart:
            if other != "ws":
                inside = dict(apart, **{other: apart["ws"] + 64})
                assert call(**inside) == E.FP8L_EINVAL, (other, "in the workspace")
        if "res" in names:                                   # y inside the residual
            assert call(**dict(apart, y=apart["res"] + 16)) == E.FP8L_EINVAL

    for scaling in (0, 1):
        check(lambda **k: fwd(scaling=scaling, **k),
              "x sx w sw bias res z y q qt s st amax ws", "z y q qt s st amax ws",
              (("y", "res"),))
    check(lambda **k: fwd(scaling=1, qt=None, st=None, **k),
          "x sx w sw bias res z y q s amax ws", "z y q s amax ws", (("y", "res"),))
    for scaling in (0, 1, 2, 3):
        check(lambda **k: bwd(scaling=scaling, **k),
              "dy sdy w sw z dz q qt s st amax db ws", "dz q qt s st amax db ws")
        check(lambda **k: ebwd(scaling=scaling, **k),
              "dy z dz q qt s st amax db ws", "dz q qt s st amax db ws")


def test_workspace_never_shrinks():
    """One workspace for the largest batch (or width) serves every smaller one, and
    holds the partial maxima of both tile sizes and the column sums behind them."""
    f = E.lib().fp8_linear_act_workspace_bytes
    assert f(-1, 16, 0) == 0 and f(16, 24, 0) == 0 and f(16, 16, 4) == 0 and f(16, -16, 0) == 0
    Ms = (list(range(0, 320, 16)) + [1, 17, 63, 65, 255, 257] + list(range(320, 4200, 48))
          + [8192, 16384, 65536])
    Ns = [0, 16, 64, 128, 144, 256, 400, 1024, 2048, 3968, 4096, 4112, 8192, 8208, 14336, 16400,
          20496, 28672, 65552, 131088]
    up = lambda n, d: -(-n // d)
    for scaling in (0, 1, 2, 3):
        for grid, at in (([sorted(Ms), Ns], lambda u, v: f(u, v, scaling)),
                         ([Ns, sorted(Ms)], lambda u, v: f(v, u, scaling))):
            for v in grid[1]:
                sizes = [at(u, v) for u in grid[0]]
                assert all(p <= q for p, q in zip(sizes, sizes[1:])), (scaling, v, sizes)
        for M in Ms:
            for N in Ns:
                few = up(M, 256) * up(N, 256) <= 80 or (M <= 64 and up(N, 128) <= 1024)
                tm, tn = (64, 128) if few else (256, 256)
                maxima = 2 * 2 * (up(N, tn) * M + up(M, tm) * N) if scaling & 1 else 4 * 1024
                n = f(M, N, scaling)
                assert n % 256 == 0 and n >= maxima + 4 * 2 * up(M, tm) * N
                assert n >= 4 * up(M, 64) * N + 4 * up(M, 64) * up(N, 256)


def test_binding_refusals():
    bf, u8 = torch.bfloat16, torch.uint8
    x, w = torch.zeros((16, 48), dtype=u8), torch.zeros((32, 48), dtype=u8)
    s, v = torch.ones(1), torch.zeros(32)
    m = torch.zeros((16, 32), dtype=bf)
    z = E.alloc_quantized(16, 32, False, "cpu")
    zr = E.alloc_quantized(16, 32, True, "cpu")
    bad = [
        lambda: E.fp8_linear_act_fwd(x.float(), s, w, s),
        lambda: E.fp8_linear_act_fwd(x, s, w[:, :32].contiguous(), s),
        lambda: E.fp8_linear_act_fwd(x, s, w, s, rowwise=True),       # rowwise needs vectors
        lambda: E.fp8_linear_act_fwd(x, s, w, s, v.half()),
        lambda: E.fp8_linear_act_fwd(x, s, w, s, v[:16]),
        lambda: E.fp8_linear_act_fwd(x, s, w, s, v, "swish"),
        lambda: E.fp8_linear_act_fwd(x, s, w, s, residual=m.float()),
        lambda: E.fp8_linear_act_fwd(x, s, w, s, residual=m[:8]),
        lambda: E.fp8_linear_act_fwd(x, s, w, s, y=m.t()),
        lambda: E.fp8_linear_act_fwd(x, s, w, s, z=m.float()),
        lambda: E.fp8_linear_act_fwd(x, s, w, s, out=E.alloc_quantized(32, 16, False, "cpu")),
        lambda: E.fp8_linear_act_fwd(x, s, w, s, out=E.Quantized(z.q, None, z.scale, None, None)),
        lambda: E.fp8_linear_act_fwd(x, s, w, s, out=z, transposed=False),
        lambda: E.fp8_linear_act_fwd(x, torch.ones(16), w, torch.ones(32), rowwise=True,
                                     transposed=False,
                                     out=E.Quantized(None, None, zr.scale, None, None)),
        lambda: E.fp8_linear_act_bwd(x, s, w, s, None, "gelu"),
        lambda: E.fp8_linear_act_bwd(x, s, w, s, m[:8], "gelu"),
        lambda: E.fp8_linear_act_bwd(x, s, w, s, m, "gelu", dbias=v.half()),
        lambda: E.fp8_linear_act_bwd(x, s, w, s, m, "gelu", dbias=v[:16]),
        lambda: E.fp8_linear_act_bwd(x, s, w, s, m, "gelu", out=zr),
        lambda: E.fp8_bias_act_bwd(m[0]),
        lambda: E.fp8_bias_act_bwd(m.float()),
        lambda: E.fp8_bias_act_bwd(m, None, "relu"),
        lambda: E.fp8_bias_act_bwd(m, m.t(), "relu"),
        lambda: E.fp8_bias_act_bwd(m, dbias=v[:8]),
        lambda: E.fp8_bias_act_bwd(m, out=E.alloc_quantized(16, 16, False, "cpu")),
    ]
    good = [lambda: E.fp8_linear_act_fwd(x, s, w, s, v, "gelu", m),
            lambda: E.fp8_linear_act_bwd(x, s, w, s, m, "gelu", bias_dtype=bf),
            lambda: E.fp8_bias_act_bwd(m, bias_dtype=bf)]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError, match="must (be|have)|rowwise") as e:
            call()
        assert "GPU" not in str(e.value), (k, e.value)
    for call in good:                    # nothing wrong but the device
        with pytest.raises(ValueError, match="on a GPU"):
            call()


@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "gelu"])
def test_stated_errors(act):
    """The header's error bounds against the kernels' sequence in 32 bits (hardware
    exponential and reciprocal taken as correctly rounded, and one unit off either
    way, results below the normal range flushed), for every finite bf16 z."""
    f32, f64, unit = np.float32, np.float64, 2.0 ** -23
    z = (np.arange(1 << 16, dtype=np.uint32) << 16).view(f32)
    z = z[np.isfinite(z)]
    Z = z.astype(f64)

    def fma(a, b, c):
        return (np.asarray(a, f64) * np.asarray(b, f64) + np.asarray(c, f64)).astype(f32)

    def flush(r):
        return np.where(np.abs(r) < 2.0 ** -126, f32(0), r)

    def kernel(de, dr):
        rcp = lambda x: flush((1 / x.astype(f64) * (1 + dr * unit)).astype(f32))
        ex2 = lambda x: flush((np.exp2(x.astype(f64)) * (1 + de * unit)).astype(f32))
        if act == "gelu":
            co = (-0.0845932811498642, 0.2405729740858078, -0.04864469915628433,
                  0.16476468741893768, 0.10670444369316101, 0.12127471715211868,
                  -7.979083602549508e-05)
            t = np.minimum(np.abs(z), f32(64))
            u = rcp(fma(t, f32(0.3), f32(1)))
            m = np.full_like(z, f32(co[0]))
            for c in co[1:]:
                m = fma(m, u, f32(c))
            e = ex2((t * f32(-0.72134752044448170)) * t)
            n = e * m
            cdf = np.where(z >= 0, f32(1) - n, n)
            return (fma(-t, n, np.maximum(z, f32(0))),
                    fma(np.copysign(t, z), e * f32(0.39894228040143268), cdf))
        log2e, k = f32(1.44269504088896341), f32(1.59576912160573071)
        c1, c3, d1, d3 = ((-log2e, f32(0), f32(1), f32(0)) if act == "silu" else
                          (-log2e * k, -log2e * k * f32(0.044715), k,
                           f32(3) * k * f32(0.044715)))
        x = np.maximum(z, f32(-128))
        b = np.minimum(x, f32(128))
        value = x * rcp(f32(1) + ex2(b * fma(c3, b * b, c1)))
        x = np.clip(z, f32(-128), f32(128))
        q = x * x
        e = ex2(np.minimum(x * fma(c3, q, c1), f32(126)))
        s = rcp(f32(1) + e)
        return value, fma(s, (x * fma(d3, q, d1)) * (e * s), s)

    with np.errstate(all="ignore"):
        if act == "gelu":
            v, phi = Z * Z / 2, np.exp(-Z * Z / 2) / np.sqrt(2 * np.pi)
            a, d = Z * ndtr(Z), ndtr(Z) + Z * phi
        else:
            k, c = (1.0, 0.0) if act == "silu" else (np.sqrt(8 / np.pi), 0.044715)
            v = k * (Z + c * Z ** 3)
            s, s1 = 1 / (1 + np.exp(-v)), 1 / (1 + np.exp(v))
            a = Z * s
            d = s + np.where((s > 0) & (s1 > 0), Z * k * (1 + 3 * c * Z * Z) * s * s1, 0)
        rel = (3 * np.abs(v) + 8) * 2.0 ** -24 + (2.0 ** -18 if act == "gelu" else 0)
        tol = np.where(np.abs(a) >= 2.0 ** -100, rel * np.abs(a), 2.0 ** -100)
        for de, dr in itertools.product((-1, 0, 1), (-1, 0, 1)):
            value, slope = kernel(de, dr)
            assert np.all(np.abs(value - a) <= tol)
            assert np.all(np.abs(slope - d) <= (2.0 ** -19 if act == "gelu" else 2.0 ** -21))
            # far below half a bf16 step wherever the value is in bf16's normal range
            ok = np.abs(a) >= 2.0 ** -100
            assert np.all((np.abs(value - a) < 2.0 ** -14 * np.abs(a))[ok])
