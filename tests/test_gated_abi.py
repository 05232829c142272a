"""Gated feed-forward entry points: what the library and the binding refuse
before anything is enqueued (fake device addresses, so only where no GPU is
visible), and the workspace sizes."""
import ctypes

import pytest
import torch

from float8_mixed_precision_amd import ops as E

A, BAD, BAD4 = 0x10000, 0x10008, 0x10002
P = lambda v: ctypes.c_void_p(v) if v else None
no_gpu = pytest.mark.skipif(torch.cuda.device_count() != 0,
                            reason="fake-pointer cases run without a GPU only")


def fwd(x=A, sx=A, w1=A, s1=A, w3=A, s3=A, M=16, H=32, K=48, scaling=0, a=None, b=None, h=A,
        hq=A, hqt=A, s=A, st=A, amax=None, ws=A, wsb=1 << 26):
    return E.lib().fp8_gated_fwd(P(x), P(sx), P(w1), P(s1), P(w3), P(s3), M, H, K, scaling, P(a),
                                 P(b), P(h), P(hq), P(hqt), P(s), P(st), P(amax), P(ws), wsb, None)


def bwd(dy=A, sdy=A, w=A, sw=A, a=A, b=A, M=16, H=32, D=48, scaling=0, da=A, db=A, daq=A, daqt=A,
        das=A, dast=A, daa=None, dbq=A, dbqt=A, dbs=A, dbst=A, dba=None, ws=A, wsb=1 << 26):
    return E.lib().fp8_gated_bwd(P(dy), P(sdy), P(w), P(sw), P(a), P(b), M, H, D, scaling, P(da),
                                 P(db), P(daq), P(daqt), P(das), P(dast), P(daa), P(dbq), P(dbqt),
                                 P(dbs), P(dbst), P(dba), P(ws), wsb, None)


@no_gpu
def test_fwd_refusals():
    for scaling in (2, 3, 4, -1):
        assert fwd(scaling=scaling) == E.FP8L_EINVAL
    for scaling in (0, 1):
        c = lambda **k: fwd(scaling=scaling, **k)
        for dim in ("H", "K"):
            assert c(**{dim: 24}) == E.FP8L_ESHAPE
            assert c(**{dim: -16}) == E.FP8L_ESHAPE
        assert c(M=17) == E.FP8L_ESHAPE                      # h is quantized
        assert c(M=-1) == E.FP8L_ESHAPE
        assert c(M=1 << 20, K=1 << 12) == E.FP8L_ESHAPE      # 2^32 bytes of codes
        assert c(H=1 << 20, K=1 << 12) == E.FP8L_ESHAPE
        assert c(M=1 << 16, H=1 << 15) == E.FP8L_ESHAPE
        for name in ("x", "sx", "w1", "s1", "w3", "s3", "h", "hq", "hqt", "s", "st", "ws"):
            assert c(**{name: None}) == E.FP8L_EINVAL
        assert c(a=A) == E.FP8L_EINVAL and c(b=A) == E.FP8L_EINVAL
        need = E.lib().fp8_gated_workspace_bytes(16, 32, scaling)
        assert c(wsb=need - 1) == E.FP8L_EWORKSPACE
        for name in ("x", "w1", "w3", "h", "hq", "hqt", "ws"):
            assert c(**{name: BAD}) == E.FP8L_EALIGN
        assert c(a=BAD, b=A) == E.FP8L_EALIGN and c(a=A, b=BAD) == E.FP8L_EALIGN
        for name in ("sx", "s1", "s3", "s", "st", "amax"):
            assert c(**{name: BAD4}) == E.FP8L_EALIGN
        none = dict(hq=None, hqt=None, s=None, st=None, ws=None, wsb=0)
        assert c(M=17, h=None, **none) == E.FP8L_EINVAL
        assert c(M=0, x=None, sx=None, h=None, **none) == E.FP8L_OK
        # an amax alone is a quantize without its outputs
        assert c(amax=A, **none) == E.FP8L_EINVAL


@no_gpu
def test_bwd_refusals():
    for scaling in (4, 5, -1):
        assert bwd(scaling=scaling) == E.FP8L_EINVAL
    for scaling in (0, 1, 2, 3):
        c = lambda **k: bwd(scaling=scaling, **k)
        for dim in ("M", "H", "D"):
            assert c(**{dim: 24}) == E.FP8L_ESHAPE
            assert c(**{dim: -16}) == E.FP8L_ESHAPE
        assert c(M=1 << 16, H=1 << 15) == E.FP8L_ESHAPE
        for name in ("dy", "sdy", "w", "sw", "a", "b", "da", "db", "daq", "daqt", "das", "dast",
                     "dbq", "dbqt", "dbs", "dbst", "ws"):
            assert c(**{name: None}) == E.FP8L_EINVAL
        need = E.lib().fp8_gated_workspace_bytes(16, 32, scaling)
        assert c(wsb=need - 1) == E.FP8L_EWORKSPACE
        for name in ("dy", "w", "a", "b", "da", "db", "daq", "daqt", "dbq", "dbqt", "ws"):
            assert c(**{name: BAD}) == E.FP8L_EALIGN
        for name in ("sdy", "sw", "das", "dast", "daa", "dbs", "dbst", "dba"):
            assert c(**{name: BAD4}) == E.FP8L_EALIGN


def test_workspace_bytes():
    f = E.lib().fp8_gated_workspace_bytes
    assert f(-1, 16, 0) == 0 and f(16, 24, 0) == 0 and f(16, 16, 4) == 0
    for scaling in (0, 1, 2, 3):
        n = f(8192, 14336, scaling)
        assert n % 256 == 0 and n >= E.fp8_swiglu_workspace_bytes(8192, 14336, bool(scaling & 1))
    # rowwise: the row and column partials of both outputs fit
    assert f(272, 400, 1) >= 2 * 2 * (8 * 272 + 4 * 400)


def test_binding_refusals():
    bf, u8 = torch.bfloat16, torch.uint8
    x, w = torch.zeros((16, 48), dtype=u8), torch.zeros((32, 48), dtype=u8)
    s = torch.ones(1)
    ab = torch.zeros((16, 32), dtype=bf)
    bad = [
        lambda: E.fp8_gated_fwd(x.float(), s, w, s, w, s),
        lambda: E.fp8_gated_fwd(x, s, w[:16], s, w, s),
        lambda: E.fp8_gated_fwd(x, s, w, s, w[:, :32].contiguous(), s),
        lambda: E.fp8_gated_fwd(x, s, w, s, w, s, True),          # rowwise needs vectors
        lambda: E.fp8_gated_fwd(x, s.double(), w, s, w, s),
        lambda: E.fp8_gated_fwd(x, s, w, s, w, s, a=ab.float(), b=ab),
        lambda: E.fp8_gated_fwd(x, s, w, s, w, s, h=ab.t()),
        lambda: E.fp8_gated_fwd(x, s, w, s, w, s, out=E.alloc_quantized(32, 16, False, "cpu")),
        lambda: E.fp8_gated_bwd(x, s, w, s, ab, ab[:8]),
        lambda: E.fp8_gated_bwd(x, s, w, s, ab, ab.float()),
        lambda: E.fp8_gated_bwd(x, s, w, s, ab, ab, qa=E.alloc_quantized(16, 32, True, "cpu")),
    ]
    good = [lambda: E.fp8_gated_fwd(x, s, w, s, w, s),
            lambda: E.fp8_gated_bwd(x, s, w, s, ab, ab)]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError, match="must be (a|both|dense)|rowwise|dense") as e:
            call()
        print(k, e.value)
    for call in good:                    # nothing wrong but the device
        with pytest.raises(ValueError, match="on a GPU"):
            call()


@no_gpu
def test_overlapping_buffers():
    at = lambda k: A + k * 4096                 # disjoint places
    apart = dict(x=at(0), w1=at(1), w3=at(2), a=at(3), b=at(4), h=at(5), hq=at(6), hqt=at(7))
    for one in ("a", "b", "h", "hq", "hqt"):
        for other in apart:
            if other != one:
                assert fwd(**dict(apart, **{one: apart[other]})) == E.FP8L_EINVAL
    apart = dict(dy=at(0), w=at(1), a=at(2), b=at(3), da=at(4), db=at(5), daq=at(6), daqt=at(7),
                 dbq=at(8), dbqt=at(9))
    for one in ("da", "db", "daq", "daqt", "dbq", "dbqt"):
        for other in apart:
            if other != one:
                assert bwd(**dict(apart, **{one: apart[other]})) == E.FP8L_EINVAL
