"""Layer norm entry points: the calls that the library and the binding refuse
on the host, before anything is enqueued (fake device addresses, so only
where no GPU is visible), and the workspace sizes."""
import ctypes

import pytest
import torch

from float8_mixed_precision_amd import ops as E

A, BAD, BAD4 = 0x10000, 0x10008, 0x10002
P = lambda v: ctypes.c_void_p(v) if v else None
no_gpu = pytest.mark.skipif(torch.cuda.device_count() != 0,
                            reason="fake-pointer cases run without a GPU only")


def fwd(x=A, rows=3, cols=5, kind=0, dtype=0, w=A, b=A, pdtype=0, eps=1e-5, y=A, mean=A, rstd=A):
    return E.lib().fp8_layernorm_fwd(P(x), rows, cols, kind, dtype, P(w), P(b), pdtype, eps, P(y),
                                     P(mean), P(rstd), None)


def quant(x=A, rows=16, cols=32, kind=0, w=A, b=A, pdtype=0, eps=1e-5, scaling=0, y=None, mean=A,
          rstd=A, q=A, qt=A, s=A, st=A, amax=None, ws=A, wsb=1 << 26):
    return E.lib().fp8_layernorm_quantize(P(x), rows, cols, kind, P(w), P(b), pdtype, eps, scaling,
                                          P(y), P(mean), P(rstd), P(q), P(qt), P(s), P(st),
                                          P(amax), P(ws), wsb, None)


def bwd(dy=A, x=A, w=A, mean=A, rstd=A, rows=3, cols=5, kind=0, dtype=0, pdtype=0, dx=A, dw=A,
        db=A, ws=A, wsb=1 << 26):
    return E.lib().fp8_layernorm_bwd(P(dy), P(x), P(w), P(mean), P(rstd), rows, cols, kind, dtype,
                                     pdtype, P(dx), P(dw), P(db), P(ws), wsb, None)


@no_gpu
@pytest.mark.parametrize("call", [fwd, quant, bwd], ids=["fwd", "quantize", "bwd"])
def test_shared_refusals(call):
    assert call(kind=2) == E.FP8L_EINVAL
    assert call(kind=-1) == E.FP8L_EINVAL
    assert call(pdtype=2) == E.FP8L_EINVAL
    assert call(rows=-16) == E.FP8L_ESHAPE
    assert call(rows=1 << 31) == E.FP8L_ESHAPE
    assert call(cols=0) == E.FP8L_ESHAPE
    assert call(cols=16400) == E.FP8L_ESHAPE
    assert call(x=None) == E.FP8L_EINVAL
    assert call(x=BAD) == E.FP8L_EALIGN
    assert call(w=BAD) == E.FP8L_EALIGN
    assert call(mean=BAD4) == E.FP8L_EALIGN
    assert call(rstd=BAD4) == E.FP8L_EALIGN


@no_gpu
def test_fwd_refusals():
    assert fwd(dtype=2) == E.FP8L_EINVAL
    assert fwd(y=None) == E.FP8L_EINVAL
    assert fwd(y=BAD) == E.FP8L_EALIGN
    assert fwd(b=BAD) == E.FP8L_EALIGN
    for eps in (-1e-5, float("nan"), float("inf")):
        assert fwd(eps=eps) == E.FP8L_EINVAL
        assert quant(eps=eps) == E.FP8L_EINVAL
    assert fwd(rows=0, x=None, y=None, mean=None, rstd=None) == E.FP8L_OK   # nothing to do


@no_gpu
def test_quantize_refusals():
    for scaling in (2, 3, -1):
        assert quant(scaling=scaling) == E.FP8L_EINVAL       # E4M3 only
    for scaling in (0, 1):
        assert quant(rows=17, scaling=scaling) == E.FP8L_ESHAPE
        assert quant(cols=24, scaling=scaling) == E.FP8L_ESHAPE
        assert quant(q=None, scaling=scaling) == E.FP8L_EINVAL
        assert quant(s=None, scaling=scaling) == E.FP8L_EINVAL
        assert quant(st=None, scaling=scaling) == E.FP8L_EINVAL
        assert quant(rstd=None, scaling=scaling) == E.FP8L_EINVAL     # y = NULL needs them
        assert quant(mean=None, scaling=scaling) == E.FP8L_EINVAL
        assert quant(ws=None, scaling=scaling) == E.FP8L_EINVAL
        need = E.lib().fp8_layernorm_workspace_bytes(16, 32, scaling)
        assert quant(wsb=need - 1, scaling=scaling) == E.FP8L_EWORKSPACE
        for name in ("ws", "q", "qt", "y", "b"):
            assert quant(**{name: BAD, "scaling": scaling}) == E.FP8L_EALIGN
        for name in ("s", "st", "amax"):
            assert quant(**{name: BAD4, "scaling": scaling}) == E.FP8L_EALIGN
    assert quant(qt=None) == E.FP8L_EINVAL                   # tensorwise needs qt
    rows_only = dict(scaling=1, qt=None, st=None, ws=None, wsb=0, mean=None, rstd=None)
    assert quant(rows=17, cols=24, **rows_only) == E.FP8L_ESHAPE
    assert quant(rows=17, s=None, **rows_only) == E.FP8L_EINVAL
    assert quant(rows=0, x=None, q=None, s=None, **rows_only) == E.FP8L_OK


@no_gpu
def test_bwd_refusals():
    assert bwd(dtype=2) == E.FP8L_EINVAL
    assert bwd(dx=None, dw=None, db=None) == E.FP8L_EINVAL
    assert bwd(dy=None) == E.FP8L_EINVAL
    assert bwd(rstd=None) == E.FP8L_EINVAL
    assert bwd(mean=None) == E.FP8L_EINVAL
    assert bwd(ws=None) == E.FP8L_EINVAL
    need = E.lib().fp8_layernorm_workspace_bytes(3, 5, 0)
    assert bwd(wsb=need - 1) == E.FP8L_EWORKSPACE
    for name in ("dy", "dx", "ws"):
        assert bwd(**{name: BAD}) == E.FP8L_EALIGN
    for name in ("dw", "db"):
        assert bwd(**{name: BAD4}) == E.FP8L_EALIGN


def test_workspace_bytes():
    f = E.lib().fp8_layernorm_workspace_bytes
    assert f(8, 0, 0) == 0 and f(-1, 16, 0) == 0 and f(8, 16385, 0) == 0 and f(8, 16, 4) == 0
    assert f(8192, 4096, 0) >= 256 * 2 * 4096 * 4
    assert f(8192, 4096, 0) % 256 == 0 and f(8192, 4096, 1) % 256 == 0
    assert E.fp8_layernorm_workspace_bytes(8192, 4096, True) == f(8192, 4096, 1)


def test_binding_refusals():
    """The binding checks types, shapes and contiguity before the call."""
    bf, f32 = torch.bfloat16, torch.float32
    x = torch.zeros((16, 32), dtype=bf)
    w = torch.zeros(32, dtype=bf)
    r = torch.zeros(16)
    bad = [
        lambda: E.fp8_layernorm_fwd(x.half()),
        lambda: E.fp8_layernorm_fwd(x[0]),
        lambda: E.fp8_layernorm_fwd(x.t()),
        lambda: E.fp8_layernorm_fwd(x[:, ::2]),
        lambda: E.fp8_layernorm_fwd(x, w[:16]),
        lambda: E.fp8_layernorm_fwd(x, w, w.float()),
        lambda: E.fp8_layernorm_fwd(x, w, y=torch.zeros((16, 32))),
        lambda: E.fp8_layernorm_fwd(x, w, mean=torch.zeros(15)),
        lambda: E.fp8_layernorm_quantize(x.float()),
        lambda: E.fp8_layernorm_quantize(x, transposed=False),
        lambda: E.fp8_layernorm_quantize(x, y=torch.zeros((16, 32), dtype=f32)),
        lambda: E.fp8_layernorm_quantize(x, out=E.alloc_quantized(16, 16, False, "cpu")),
        lambda: E.fp8_layernorm_bwd(x.float(), x, w, r, r),
        lambda: E.fp8_layernorm_bwd(x[:8], x, w, r, r),
        lambda: E.fp8_layernorm_bwd(x, x, w, r.double(), r),
        lambda: E.fp8_layernorm_bwd(x, x, w, r, r, dweight=torch.zeros(32, dtype=bf)),
    ]
    good = [lambda: E.fp8_layernorm_fwd(x, w, w), lambda: E.fp8_layernorm_quantize(x, w),
            lambda: E.fp8_layernorm_bwd(x, x, w, r, r)]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError, match="must be (a|both|dense)|rowwise|dense") as e:
            call()
        print(k, e.value)
    for call in good:                    # nothing wrong but the device
        with pytest.raises(ValueError, match="on a GPU"):
            call()


@no_gpu
def test_overlapping_buffers():
    n = 16 * 32
    at = lambda k: A + k * 4096                 # disjoint places for [16, 32]
    for y in (at(0), at(0) - 64, at(0) + 2 * n - 16):
        assert fwd(x=at(0), rows=16, cols=32, y=y, mean=at(2), rstd=at(3)) == E.FP8L_EINVAL
    assert fwd(x=at(0), rows=16, cols=32, y=at(1), mean=at(1), rstd=at(3)) == E.FP8L_EINVAL
    apart = dict(x=at(0), mean=at(1), rstd=at(2), q=at(3), qt=at(4), y=at(5))
    for one in ("mean", "rstd", "q", "qt", "y"):
        for other in apart:
            if other != one:
                assert quant(**dict(apart, **{one: apart[other]})) == E.FP8L_EINVAL
    apart = dict(rows=16, cols=32, dy=at(0), x=at(1), mean=at(2), rstd=at(3), dx=at(4), dw=at(5),
                 db=at(6))
    for one in ("dx", "dw", "db"):
        for other in ("dy", "x", "mean", "rstd", "dx", "dw", "db"):
            if other != one:
                assert bwd(**dict(apart, **{one: apart[other]})) == E.FP8L_EINVAL
