"""GPU linear with its epilogue, and the gradient through it.

* The product p before it is rounded comes from the plain GEMM's instructions
  in its order: for more than 16 tokens it equals fp8_linear_bwd_w_f32's output
  of the same operands bit for bit, so z = bf16(fl32(p + bias)) and, without an
  activation, y = bf16(fl32(fl32(p + bias) + residual)) are checked bit for bit.
  With fewer tokens (the contraction split over 8 waves) p is within the
  instruction's accumulation bound (tests/mfma_model.py) plus 7 fp32 additions.
* act and act' are checked in 64 bits from the written bf16 z, within the errors
  that the header states; one fp32 rounding (u = 2^-24) for the residual's sum or
  the product with dh, then the rounding to bf16, half a step (2^-8).
* dbias sums the unrounded dz: at most 64 rows in turn and log steps per slice,
  then 16 + 16 + rows / 1024 slices: (rows / 1024 + 128) u of the sum of
  magnitudes, plus what the slope's error contributes.
* The codes and scales are the oracle's quantize of the written bf16 values, bit
  for bit, whether those are stored or not."""
import numpy as np
import pytest
import torch
from scipy.special import ndtr

import oracle
from float8_mixed_precision_amd import ops
from float8_mixed_precision_amd import workloads as W
from tests import gpu_util as G
from tests import mfma_model as MM

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
RW = pytest.mark.parametrize("rowwise", [False, True], ids=["tensorwise", "rowwise"])
SIZE_ID = lambda s: "%dx%dx%d" % s
K2 = np.sqrt(8 / np.pi)


def _value(t):
    return t.double().cpu().numpy()


def act64(z, act):
    """act(z), its derivative and the stated error bounds of both, in 64 bits."""
    with np.errstate(all="ignore"):
        if act == "none":
            return z, np.ones_like(z), 0 * z, 0 * z
        p = np.where(np.isnan(z), z, np.maximum(z, 0))
        if act == "relu":
            return p, (z > 0) * 1.0, 0 * p, 0 * p
        if act == "relu2":
            return p * p, 2 * p, U * p * p, 0 * p
        if act == "gelu":
            v, cdf = z * z / 2, ndtr(z)
            phi = np.exp(-v) / np.sqrt(2 * np.pi)
            a, d, more, ds = z * cdf, cdf + z * phi, 2.0 ** -18, 2.0 ** -19
        else:
            k, c = (1.0, 0.0) if act == "silu" else (K2, 0.044715)
            v = k * (z + c * z ** 3)
            s, s1 = 1 / (1 + np.exp(-v)), 1 / (1 + np.exp(v))
            w = z * k * (1 + 3 * c * z * z) * s1
            a, d, more, ds = z * s, s * (1 + np.where(s > 0, w, 0)), 0.0, 2.0 ** -21
        rel = (3 * np.abs(v) + 8) * U + more
        err = np.where(np.abs(a) >= 2.0 ** -100, rel * np.abs(a), 2.0 ** -100)
        return a, d, err, np.full_like(z, ds)


def _pad16(m):
    return (m + 15) // 16 * 16


def _x(M, K, rowwise, seed):
    z = ops.fp8_linear_quantize(G.dev_bf16(W.random_bf16(seed, (_pad16(M), K), 1.0, 0)), rowwise)
    return z.q, z.scale


def _w(N, K, rowwise, seed):
    z = ops.fp8_linear_quantize(G.dev_bf16(W.random_bf16(seed, (N, K), max(K, 1) ** -0.5, 1)),
                                rowwise)
    return z.q, z.scale


def _product32(xq, sx, wq, sw, rowwise, e5m2=False):
    """The unrounded product of more than 16 rows."""
    (M, K), N = xq.shape, wq.shape[0]
    return ops.fp8_linear_bwd_w_f32(xq, sx, wq, sw, K, M, N, rowwise, e5m2=e5m2)


def _bias(N, dtype, seed):
    return (torch.randn(N, generator=torch.Generator().manual_seed(seed)) * 0.3).to(dtype).to(G.DEV)


def _residual(M, N, seed):
    return G.dev_bf16(W.random_bf16(seed, (M, N), 2.0, 2))


def _bits(t):
    return t.view(torch.int16)


def _hq(z):
    return tuple(G.host(t) for t in (z.q, z.qt, z.scale, z.scale_t, z.amax))


def check_y(y, z, act, residual, label):
    """y from the bf16 z (with an activation)."""
    a, _, err, _ = act64(_value(z), act)
    want = a if residual is None else a + _value(residual)
    tol = err + U * np.abs(want)
    tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    got = _value(y)
    assert np.all(np.isfinite(got)), label
    bad = np.abs(got - want) > tol
    assert not bad.any(), "%s: %d outside, first %s" % (label, bad.sum(), np.argwhere(bad)[0])


def check_dz(dz, dh, z, act, label):
    """dz from the fp32 dh; returns what dbias is checked with."""
    dh = _value(dh)
    d, ds = (np.ones_like(dh), 0 * dh) if act == "none" else act64(_value(z), act)[1::2]
    want = dh * d
    err = np.abs(dh) * ds + 2 * U * np.abs(want)
    tol = err + 2.0 ** -8 * (np.abs(want) + err)
    bad = ~(np.abs(_value(dz) - want) <= tol)
    assert not bad.any(), "%s: %d outside, first %s" % (label, bad.sum(), np.argwhere(bad)[0])
    return want, err


def check_dbias(dbias, want, err, label):
    n = (want.shape[0] / 1024 + 128) * U
    tol = n * np.abs(want).sum(0) + err.sum(0)
    v = want.sum(0)
    if dbias.dtype == BF:
        tol = tol + 2.0 ** -8 * (np.abs(v) + tol)
    bad = ~(np.abs(_value(dbias) - v) <= tol)
    assert not bad.any(), "%s: %d outside, first %s" % (label, bad.sum(), np.argwhere(bad)[0])


FWD = [(32, 144, 400), (80, 16, 16), (272, 400, 528), (256, 128, 128), (1040, 784, 304),
       (512, 2048, 256),
       # large tiles, several of them a workgroup
       (2064, 8208, 144), (4112, 4112, 384), (8192, 2048, 128)]


@RW
@pytest.mark.parametrize("mnk,act", [(s, a) for s in FWD for a in ops.ACTS
                                     if s[0] * s[1] < 1 << 22 or a in ("none", "gelu", "silu")])
def test_forward(mnk, act, rowwise):
    M, N, K = mnk
    xq, sx = _x(M, K, rowwise, 70)
    wq, sw = _w(N, K, rowwise, 71)
    bias = None if N % 3 == 0 else _bias(N, F32 if N % 32 else BF, N)
    res = _residual(M, N, 72)
    G.say("linear act fwd", mnk, act, "rowwise", rowwise)
    p = _product32(xq, sx, wq, sw, rowwise)
    z32 = p if bias is None else p + bias.float()
    ws = ops.alloc_linear_act_workspace(M, N, rowwise, G.DEV).fill_(0x7F)
    new = lambda: torch.empty((M, N), dtype=BF, device=G.DEV)
    call = lambda **k: ops.fp8_linear_act_fwd(xq, sx, wq, sw, bias, act, rowwise=rowwise,
                                              workspace=ws, **k)
    for r in (None, res):
        z, q1, q2, q3 = new(), *(ops.alloc_quantized(M, N, rowwise, G.DEV) for _ in range(3))
        y = call(residual=r, z=z, out=q1, y=new())
        y2 = call(residual=r)                                # nothing else
        y3 = call(residual=r, out=q2)                        # z not stored
        torch.cuda.synchronize()
        label = "%s %s %s" % (mnk, act, r is not None)
        assert torch.equal(_bits(z), _bits(z32.to(BF))), label
        if act == "none":
            want = z32.to(BF) if r is None else (z32 + r.float()).to(BF)
            assert torch.equal(_bits(y), _bits(want)), label
        else:
            check_y(y, z, act, r, label)
        assert torch.equal(_bits(y), _bits(y2)) and torch.equal(_bits(y), _bits(y3)), label
        ref = oracle.quantize(G.host(y), rowwise)
        G.assert_quantize_equal(_hq(q1), ref, "codes of y " + label)
        G.assert_quantize_equal(_hq(q2), ref, "codes of y, z not stored " + label)
        if r is None:
            z4 = new()
            assert call(z=z4, out=q3) is None                # y not stored
            torch.cuda.synchronize()
            assert torch.equal(_bits(z), _bits(z4)), label
            G.assert_quantize_equal(_hq(q3), ref, "codes of y, y not stored " + label)


@RW
@pytest.mark.parametrize("mnk", [(17, 272, 4112), (50, 1040, 784), (40, 28672, 32), (65, 400, 528),
                                 (131, 256, 128), (257, 144, 272), (769, 2048, 256),
                                 (2081, 8208, 144), (50, 4096, 2064), (33, 528, 14336)],
                         ids=SIZE_ID)
def test_any_number_of_tokens(mnk, rowwise):
    """M tokens give the first M rows of the padded call, in place of the
    residual too; the rows behind them stay as they were."""
    M, N, K = mnk
    P = _pad16(M)
    act = list(ops.ACTS)[(M + N // 16) % 6]
    xq, sx = _x(M, K, rowwise, 73)
    wq, sw = _w(N, K, rowwise, 74)
    bias, res = _bias(N, BF, 75), _residual(P, N, 76)
    G.say("linear act ragged", mnk, act, "rowwise", rowwise)
    zp = torch.empty((P, N), dtype=BF, device=G.DEV)
    want = ops.fp8_linear_act_fwd(xq, sx, wq, sw, bias, act, res, rowwise, z=zp)
    # (exact-size copies: no readable row behind the operands' last one)
    xs, ss = xq[:M].clone(), sx[:M].clone() if rowwise else sx
    y, z, acc = (torch.full((P + 16, N), 7.0, dtype=BF, device=G.DEV) for _ in range(3))
    acc[:M] = res[:M]
    ops.fp8_linear_act_fwd(xs, ss, wq, sw, bias, act, res[:M].clone(), rowwise, y=y[:M], z=z[:M])
    ops.fp8_linear_act_fwd(xs, ss, wq, sw, bias, act, acc[:M], rowwise, y=acc[:M])
    torch.cuda.synchronize()
    assert torch.equal(_bits(y[:M]), _bits(want[:M])) and torch.equal(_bits(z[:M]), _bits(zp[:M]))
    assert torch.equal(_bits(acc[:M]), _bits(want[:M]))
    for t in (y, z, acc):
        assert torch.all(t[M:] == 7.0)


@RW
@pytest.mark.parametrize("mnk", [(1, 16, 16), (1, 512, 4096), (2, 144, 1040), (15, 400, 528),
                                 (16, 256, 2048), (3, 14336, 144), (1, 4096, 14336),
                                 (16, 14336, 128), (17, 128, 1040), (50, 256, 14336),
                                 (100, 128, 8208)], ids=SIZE_ID)
def test_few_tokens(mnk, rowwise):
    M, N, K = mnk
    act = ("none", "gelu")[N % 32 == 0]
    xq, sx = _x(M, K, rowwise, 77)
    xs, ss = xq[:M].clone(), sx[:M].clone() if rowwise else sx
    wq, sw = _w(N, K, rowwise, 78)
    bias, res = _bias(N, F32, 79), _residual(_pad16(M), N, 80)[:M].clone()
    G.say("linear act few tokens", mnk, "rowwise", rowwise)
    y, z = (torch.full((M + 3, N), 7.0, dtype=BF, device=G.DEV) for _ in range(2))
    ops.fp8_linear_act_fwd(xs, ss, wq, sw, bias, act, res, rowwise, y=y[:M], z=z[:M])
    y2 = ops.fp8_linear_act_fwd(xs, ss, wq, sw, bias, act, res, rowwise)
    torch.cuda.synchronize()
    assert torch.equal(_bits(y[:M]), _bits(y2))
    assert torch.all(y[M:] == 7.0) and torch.all(z[M:] == 7.0)
    A, B = G.host(xs), G.host(wq)
    ii, jj = np.divmod(np.arange(M * N), N)
    val = np.nan_to_num(oracle.e4m3_values())
    sa = np.broadcast_to(1 / G.host(ss).astype(np.float64), (M,))[:, None]
    sb = np.broadcast_to(1 / G.host(sw).astype(np.float64), (N,))[None, :]
    want = (val[A] @ val[B].T) * sa * sb
    # the instruction against sequential fp32 sums, those against exact ones (K
    # additions; at most 16 more where the contraction is split), two scalings
    D = MM.sum_difference_bound(A, B, ii, jj).reshape(M, N)
    D = D + (K + 16) * U * (np.abs(val)[A] @ np.abs(val)[B].T)
    tol = D * sa * sb * (1 + 2.0 ** -20) + 3 * U * np.abs(want)
    want = want + _value(bias)
    tol = tol + U * np.abs(want)
    ztol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    assert np.all(np.abs(_value(z[:M]) - want) <= ztol), mnk
    if act == "none":
        v = want + _value(res)
        t = tol + U * np.abs(v)
        assert np.all(np.abs(_value(y[:M]) - v) <= t + 2.0 ** -8 * (np.abs(v) + t)), mnk
    else:
        check_y(y[:M], z[:M], act, res, "y %s" % (mnk,))
    if M % 16 == 0:
        q1, q2 = (ops.alloc_quantized(M, N, rowwise, G.DEV) for _ in range(2))
        y3 = ops.fp8_linear_act_fwd(xs, ss, wq, sw, bias, act, None, rowwise, out=q1)
        z2 = torch.empty_like(y3)
        ops.fp8_linear_act_fwd(xs, ss, wq, sw, bias, act, None, rowwise, z=z2, out=q2)
        torch.cuda.synchronize()
        assert torch.equal(_bits(z2), _bits(z[:M]))
        ref = oracle.quantize(G.host(y3), rowwise)
        G.assert_quantize_equal(_hq(q1), ref, "codes %s" % (mnk,))
        G.assert_quantize_equal(_hq(q2), ref, "codes, y not stored %s" % (mnk,))


@pytest.mark.parametrize("mnk", [(1, 16, 16), (1, 14336, 256), (5, 400, 528), (50, 4096, 1040),
                                 (300, 8208, 144), (33, 256, 14336), (2000, 8192, 128)],
                         ids=SIZE_ID)
def test_codes_of_rows(mnk):
    """The serving form: any number of tokens, codes and scales of the rows alone."""
    M, N, K = mnk
    act = list(ops.ACTS)[N // 16 % 6]
    xq, sx = _x(M, K, True, 81)
    xs, ss = xq[:M].clone(), sx[:M].clone()
    wq, sw = _w(N, K, True, 82)
    bias, res = _bias(N, BF, 83), _residual(_pad16(M), N, 84)[:M].clone()
    new = lambda: ops.Quantized(torch.full((M + 2, N), 5, dtype=torch.uint8, device=G.DEV), None,
                                torch.empty(M, device=G.DEV), None, torch.empty(M, device=G.DEV))
    G.say("linear act rows", mnk, act)
    for r in (None, res):
        want = ops.fp8_linear_act_fwd(xs, ss, wq, sw, bias, act, r, True)
        pad = np.zeros((_pad16(M), N), np.uint16)
        pad[:M] = G.host(want)
        ref = oracle.quantize(pad, True)
        for stored in (True, False)[:2 if r is None else 1]:
            z, q = torch.empty((M, N), dtype=BF, device=G.DEV), new()
            out = ops.Quantized(q.q[:M], None, q.scale, None, q.amax)
            y = ops.fp8_linear_act_fwd(xs, ss, wq, sw, bias, act, r, True, out=out,
                                       transposed=False, z=None if stored else z)
            torch.cuda.synchronize()
            assert torch.equal(_bits(y), _bits(want)) if stored else y is None
            assert np.array_equal(G.host(out.q), ref[0][:M])
            assert np.array_equal(G.host(out.scale), ref[2][:M])
            assert np.array_equal(G.host(out.amax), ref[4][:M])
            assert torch.all(q.q[M:] == 5)


BWD = [(32, 16, 16), (80, 144, 48), (272, 400, 528), (256, 256, 128), (1040, 784, 304),
       (528, 4112, 400), (64, 28672, 48), (2064, 8208, 128), (4112, 4112, 272)]


@pytest.mark.parametrize("e5m2", [False, True], ids=["e4m3", "e5m2"])
@RW
@pytest.mark.parametrize("mhd", BWD, ids=SIZE_ID)
def test_backward(mhd, rowwise, e5m2):
    M, H, D = mhd
    qdy = ops.fp8_linear_quantize(G.dev_bf16(W.random_bf16(76, (M, D), 1e-2, 0)), rowwise,
                                  e5m2=e5m2)
    qw = ops.fp8_linear_quantize(G.dev_bf16(W.random_bf16(76, (D, H), 0.02, 1)), rowwise)
    z = G.dev_bf16(W.random_bf16(77, (M, H), 1.5, 2))
    dh = _product32(qdy.q, qdy.scale, qw.qt, qw.scale_t, rowwise, e5m2)
    ws = ops.alloc_linear_act_workspace(M, H, rowwise, G.DEV).fill_(0x7F)
    quantize = oracle.quantize_e5m2 if e5m2 else oracle.quantize
    for k, act in enumerate(ops.ACTS):
        if k % 3 and M * H > 1 << 22:
            continue
        G.say("linear act bwd", mhd, act, "rowwise", rowwise, "e5m2", e5m2)
        pd = (BF, F32)[k % 2]
        dz, q, db = ops.fp8_linear_act_bwd(qdy.q, qdy.scale, qw.qt, qw.scale_t,
                                           None if act == "none" else z, act, rowwise, e5m2,
                                           bias_dtype=pd, workspace=ws)
        dz2, _, none = ops.fp8_linear_act_bwd(qdy.q, qdy.scale, qw.qt, qw.scale_t, z, act, rowwise,
                                              e5m2)
        torch.cuda.synchronize()
        label = "%s %s" % (mhd, act)
        assert none is None and db.dtype == pd and torch.equal(_bits(dz), _bits(dz2)), label
        want, err = check_dz(dz, dh, z, act, "dz " + label)
        check_dbias(db, want, err, "dbias " + label)
        if act == "none":
            assert torch.equal(_bits(dz), _bits(dh.to(BF)))
        G.assert_quantize_equal(_hq(q), quantize(G.host(dz), rowwise), "codes of dz " + label)


@pytest.mark.parametrize("e5m2", [False, True], ids=["e4m3", "e5m2"])
@RW
@pytest.mark.parametrize("shape", [(16, 16), (80, 144), (272, 400), (1040, 784), (64, 28672),
                                   (2064, 8208), (8192, 1040), (16400, 528)],
                         ids=lambda s: "%dx%d" % s)
def test_bias_act_backward(shape, rowwise, e5m2):
    M, N = shape
    dy = G.dev_bf16(W.random_bf16(85, (M, N), 1e-2, 0))
    z = G.dev_bf16(W.random_bf16(86, (M, N), 1.5, 1))
    ws = ops.alloc_linear_act_workspace(M, N, rowwise, G.DEV).fill_(0x7F)
    quantize = oracle.quantize_e5m2 if e5m2 else oracle.quantize
    for k, act in enumerate(ops.ACTS):
        if k not in (0, 2) and M * N > 1 << 22:
            continue
        G.say("bias act bwd", shape, act, "rowwise", rowwise, "e5m2", e5m2)
        pd = (F32, BF)[k % 2]
        dz, q, db = ops.fp8_bias_act_bwd(dy, z, act, rowwise, e5m2, bias_dtype=pd, workspace=ws)
        torch.cuda.synchronize()
        label = "%s %s" % (shape, act)
        assert (dz is None) == (act == "none")
        want, err = check_dz(dy if dz is None else dz, dy, z, act, "dz " + label)
        check_dbias(db, want, err, "dbias " + label)
        ref = quantize(G.host(dy if dz is None else dz), rowwise)
        G.assert_quantize_equal(_hq(q), ref, "codes of dz " + label)
        if act == "none":                                    # with a dz of its own
            dz = torch.empty_like(dy)
            ops.fp8_bias_act_bwd(dy, None, act, rowwise, e5m2, dz=dz, out=q, workspace=ws)
            torch.cuda.synchronize()
            assert torch.equal(_bits(dz), _bits(dy))
            G.assert_quantize_equal(_hq(q), ref, "codes of dz " + label)


@pytest.mark.parametrize("at", [(0, 0), (8207, 4111), (4100, 2000)], ids=str)
def test_maxima_of_many_tiles(at):
    """More tiles than maxima that the cast reads: they are reduced in between, and the
    largest value counts wherever it lies."""
    M, N = 8208, 4112
    dy = G.dev_bf16(W.random_bf16(87, (M, N), 1e-2, 0))
    dy[at] = -37.5
    _, q, _ = ops.fp8_bias_act_bwd(dy, None, "none")
    z = G.dev_bf16(W.random_bf16(88, (M, N), 1.0, 1)).clamp_(min=0.25)
    dz, q2, db = ops.fp8_bias_act_bwd(dy, z, "relu", bias_dtype=F32)
    ref = ops.fp8_linear_quantize(dy)
    torch.cuda.synchronize()
    assert torch.equal(_bits(dz), _bits(dy))
    for got in (q, q2):
        assert got.amax.item() == 37.5
        for a, b in zip(_hq(got), _hq(ref)):
            assert torch.equal(torch.as_tensor(a), torch.as_tensor(b))
    # fp32 sums of 8208 terms, 64 rows in a tile and its 8 row phases, then 129 tiles
    exact = dy.double().sum(0)
    err = (dy.double().abs().sum(0) * (64 + 129)) * 2.0 ** -24
    assert bool(((db.double() - exact).abs() <= err).all())


def _every_bf16():
    z = (torch.arange(1 << 16, dtype=torch.int32) << 16).view(torch.float32).to(BF)
    return z


@pytest.mark.parametrize("act", [a for a in ops.ACTS if a != "none"])
def test_every_pre_activation(act):
    """act and act' of every bf16 value, through each of the kernels that
    evaluate them (zero operands: z is the bias)."""
    z = _every_bf16()
    fin = torch.isfinite(z.float()).numpy()
    zv = z.double().numpy()
    N = z.numel()
    a, d, err, ds = act64(zv, act)
    a, d = (np.where(fin, v, np.nan) for v in (a, d))
    tol = err + 2.0 ** -8 * (np.abs(a) + err) + 2.0 ** -133
    big = a > 3.38e38                                        # rounds to infinity, or nearly
    f = lambda v: torch.tensor(v, device=G.DEV)
    for M, K in ((1, 16), (16, 0), (32, 16), (64, 16), (512, 16)):
        G.say("every pre-activation", act, M, K)
        zero = lambda n: torch.zeros((n, K), dtype=torch.uint8, device=G.DEV)
        y = ops.fp8_linear_act_fwd(zero(M), f([1.0]), zero(N), f([1.0]), z.to(G.DEV), act)
        torch.cuda.synchronize()
        got = y[M - 1].double().cpu().numpy()
        assert torch.equal(_bits(y[0]), _bits(y[M - 1]))
        with np.errstate(invalid="ignore"):
            ok = np.abs(got - a) <= tol
        assert np.all((ok | big)[fin]), (M, zv[fin & ~ok & ~big][:5])
        assert np.all(got[big & fin] > 3.3e38)
        neg = got[np.isneginf(zv)][0]
        assert got[np.isposinf(zv)][0] == np.inf and neg == 0
        assert np.all(np.isnan(got[np.isnan(zv)]))
    dy = torch.ones((16, N), dtype=BF, device=G.DEV)
    dz, _, _ = ops.fp8_bias_act_bwd(dy, z.to(G.DEV).repeat(16, 1), act)
    torch.cuda.synchronize()
    got = dz[3].double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        okd = np.abs(got - d) <= ds + U * np.abs(d) + 2.0 ** -8 * (np.abs(d) + ds)
    assert np.all((okd | (d > 3.38e38))[fin]), zv[fin & ~okd][:5]
    # (s + w e s with s at most 2^-126 there and |w| below 2^19)
    assert np.abs(got[np.isneginf(zv)][0]) < 2.0 ** -106
    assert got[np.isposinf(zv)][0] == (np.inf if act == "relu2" else 1)
    # the same through the product's epilogues: dh = 1 in every element
    one = torch.full((1, 16), 0x38, dtype=torch.uint8, device=G.DEV)       # E4M3 1.0
    e0 = one.clone()
    e0[0, 1:] = 0
    for M in (32, 512):
        zz = z.to(G.DEV).repeat(M, 1)
        dz2, _, _ = ops.fp8_linear_act_bwd(e0.repeat(M, 1), f([1.0]), one.repeat(N, 1), f([1.0]),
                                           zz, act)
        torch.cuda.synchronize()
        got2 = dz2[M - 1].double().cpu().numpy()
        assert np.array_equal(got2[fin], got[fin]) and torch.equal(_bits(dz2[0]), _bits(dz2[M - 1]))


def test_gradient_against_differences():
    """d sum(act(z) g) / dz by central differences in 64 bits (step 1e-5:
    truncation about 1e-9)."""
    M, N = 16, 1040
    z = G.dev_bf16(W.random_bf16(87, (M, N), 1.5, 1))
    g = G.dev_bf16(W.random_bf16(88, (M, N), 1.0, 2))
    zv, gv, h = _value(z), _value(g), 1e-5
    for act in ("gelu", "gelu_tanh", "silu"):
        G.say("act differences", act)
        dz, _, _ = ops.fp8_bias_act_bwd(g, z, act)
        torch.cuda.synchronize()
        diff = gv * (act64(zv + h, act)[0] - act64(zv - h, act)[0]) / (2 * h)
        tol = 2.0 ** -8 * np.abs(diff) + np.abs(gv) * 2.0 ** -18
        assert np.all(np.abs(_value(dz) - diff) <= tol), act


@RW
@pytest.mark.parametrize("mnk", [(0, 64, 32), (48, 0, 32), (48, 64, 0), (528, 4112, 0), (5, 64, 0),
                                 (0, 0, 0)], ids=SIZE_ID)
def test_empty(mnk, rowwise):
    """No tokens, no outputs, and an empty contraction (z is the bias, dz and
    dbias zero)."""
    M, N, K = mnk
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device=G.DEV)
    s = lambda n: torch.ones(n if rowwise else 1, device=G.DEV)
    bias, res = _bias(N, F32, 1), _residual(M, N, 2) if M * N else torch.empty(
        (M, N), dtype=BF, device=G.DEV)
    G.say("linear act empty", mnk, rowwise)
    for act in ("none", "gelu"):
        z, y0 = (torch.empty((M, N), dtype=BF, device=G.DEV) for _ in range(2))
        y = ops.fp8_linear_act_fwd(u8(M, K), s(M), u8(N, K), s(N), bias, act, res, rowwise, z=z)
        torch.cuda.synchronize()
        assert torch.equal(z, bias.to(BF).repeat(M, 1))
        if act == "none":
            assert torch.equal(y, (bias + res.float()).to(BF))
        elif M * N:
            check_y(y, z, act, res, "empty")
        if M % 16 == 0:
            q = ops.alloc_quantized(M, N, rowwise, G.DEV)
            ops.fp8_linear_act_fwd(u8(M, K), s(M), u8(N, K), s(N), bias, act, None, rowwise, z=z,
                                   y=y0, out=q)
            q2 = ops.alloc_quantized(M, N, rowwise, G.DEV)
            ops.fp8_linear_act_fwd(u8(M, K), s(M), u8(N, K), s(N), bias, act, None, rowwise, z=z,
                                   out=q2)
            torch.cuda.synchronize()
            ref = oracle.quantize(G.host(y0), rowwise)
            G.assert_quantize_equal(_hq(q), ref, "empty")
            G.assert_quantize_equal(_hq(q2), ref, "empty, y not stored")
            dz, q3, db = ops.fp8_linear_act_bwd(u8(M, K), s(M), u8(N, K), s(N), z, act, rowwise,
                                                bias_dtype=F32)
            dz4, q4, db4 = ops.fp8_bias_act_bwd(torch.zeros_like(z), z, act, rowwise, bias_dtype=BF)
            torch.cuda.synchronize()
            assert torch.all(dz[: M if K == 0 else 0] == 0) and torch.all(db == 0)
            assert torch.all(db4 == 0) and db.shape == db4.shape == (N,)
            zero = oracle.quantize(np.zeros((M, N), np.uint16), rowwise)
            # (0 times a negative slope is -0)
            ref4 = zero if dz4 is None else oracle.quantize(G.host(dz4), rowwise)
            G.assert_quantize_equal(_hq(q4), ref4, "empty backward")
            assert dz4 is None or torch.all(dz4 == 0)
            if M * N == 0 or K == 0:
                G.assert_quantize_equal(_hq(q3), zero, "empty backward")


def test_nonfinite():
    """A NaN or an infinity in the bias stays in its column and shows in the amax."""
    M, N, K = 48, 400, 272
    xq, sx = _x(M, K, False, 90)
    wq, sw = _w(N, K, False, 91)
    G.say("linear act nonfinite")
    for act in ops.ACTS:
        clean = ops.fp8_linear_act_fwd(xq, sx, wq, sw, torch.zeros(N, device=G.DEV), act)
        for v in (float("nan"), float("inf")):
            bias = torch.zeros(N, device=G.DEV)
            bias[37] = v
            z = torch.empty((M, N), dtype=BF, device=G.DEV)
            q, q2 = (ops.alloc_quantized(M, N, False, G.DEV) for _ in range(2))
            y = ops.fp8_linear_act_fwd(xq, sx, wq, sw, bias, act, out=q)
            ops.fp8_linear_act_fwd(xq, sx, wq, sw, bias, act, z=z, out=q2)
            torch.cuda.synchronize()
            rest = torch.arange(N, device=G.DEV) != 37
            assert torch.equal(_bits(y[:, rest]), _bits(clean[:, rest]))
            for a in (q.amax, q2.amax):
                assert torch.isnan(a).all() if v != v else torch.isinf(a).all(), (act, v)


@RW
def test_side_stream_and_graph(rowwise):
    """The same results on a stream of its own and from two captured graphs that
    share the workspace, replayed in turn with eager work between."""
    M, H, D = 96, 1040, 528
    xq, sx = _x(M, D, rowwise, 92)
    wq, sw = _w(H, D, rowwise, 93)
    qdy = ops.fp8_linear_quantize(G.dev_bf16(W.random_bf16(94, (M, D), 1e-2, 0)), rowwise)
    qw2 = ops.fp8_linear_quantize(G.dev_bf16(W.random_bf16(94, (D, H), 0.02, 1)), rowwise)
    bias = _bias(H, F32, 95)
    ws = ops.alloc_linear_act_workspace(M, H, rowwise, G.DEV)
    z, dz = (torch.empty((M, H), dtype=BF, device=G.DEV) for _ in range(2))
    qy, qz = (ops.alloc_quantized(M, H, rowwise, G.DEV) for _ in range(2))
    db = torch.empty(H, device=G.DEV)

    def forward():
        ops.fp8_linear_act_fwd(xq, sx, wq, sw, bias, "gelu", rowwise=rowwise, z=z, out=qy,
                               workspace=ws)

    def backward():
        ops.fp8_linear_act_bwd(qdy.q, qdy.scale, qw2.qt, qw2.scale_t, z, "gelu", rowwise, dz=dz,
                               out=qz, dbias=db, workspace=ws)

    def results():
        torch.cuda.synchronize()
        return [t.clone() for q in (qy, qz) for t in (q.q, q.qt, q.scale, q.scale_t, q.amax)] + [
            z.clone(), dz.clone(), db.clone()]

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
        bias.add_(0.25)
        forward(), backward()
        want = results()
        z.zero_()
        for g in graphs:
            g.replay()
        assert all(torch.equal(p, q) for p, q in zip(results(), want)), k


def test_largest_outputs():
    """Outputs of almost 2^31 bytes: the last rows are those of a call on them."""
    M, N, K = 32752, 32768, 16
    xq, sx = _x(M, K, True, 96)
    wq, sw = _w(N, K, True, 97)
    bias = _bias(N, BF, 98)
    G.say("linear act largest outputs")
    z = torch.empty((M, N), dtype=BF, device=G.DEV)
    q = ops.alloc_quantized(M, N, True, G.DEV)
    res = torch.ones((1, N), dtype=BF, device=G.DEV).repeat(M, 1)
    y = ops.fp8_linear_act_fwd(xq, sx, wq, sw, bias, "silu", res, True, z=z, out=q)
    last = slice(M - 272, M)
    z1 = torch.empty((272, N), dtype=BF, device=G.DEV)
    y1 = ops.fp8_linear_act_fwd(xq[last].clone(), sx[last].clone(), wq, sw, bias, "silu",
                                res[last].clone(), True, z=z1)
    dz, qz, db = ops.fp8_linear_act_bwd(xq, sx, wq, sw, z, "silu", True, bias_dtype=F32)
    dz1, _, _ = ops.fp8_linear_act_bwd(xq[last].clone(), sx[last].clone(), wq, sw, z1, "silu", True)
    torch.cuda.synchronize()
    assert torch.equal(_bits(y[last]), _bits(y1)) and torch.equal(_bits(z[last]), _bits(z1))
    assert torch.equal(_bits(dz[last]), _bits(dz1))
    rows = [0, 1, 16383, M - 1]
    ref = oracle.quantize(np.concatenate([G.host(y[rows]), np.zeros((12, N), np.uint16)]), True)
    assert np.array_equal(G.host(q.q[rows]), ref[0][:4])
    assert torch.equal(q.amax[M:], y.abs().amax(0).float())
    assert torch.equal(qz.amax[M:], dz.abs().amax(0).float())
    # (bf16 dz summed in fp64 against the sum of the unrounded ones: half a bf16 step
    # of each)
    s = dz.double()
    assert torch.all((db.double() - s.sum(0)).abs() <= 2.0 ** -8 * s.abs().sum(0) * 1.01 + 1e-30)
