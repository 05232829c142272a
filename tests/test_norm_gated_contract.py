"""What the norm's and the gated feed-forward's entry points promise beyond
their argument checks: host side, no GPU needed."""
import numpy as np
import pytest
import torch

from float8_mixed_precision_amd import ops as E
from tests import test_gated_abi as gated_abi
from tests import test_layernorm_abi as norm_abi

A = 0x10000
no_gpu = pytest.mark.skipif(torch.cuda.device_count() != 0,
                            reason="fake-pointer cases run without a GPU only")


@pytest.mark.parametrize("rowwise", [False, True], ids=["tensorwise", "rowwise"])
def test_transposed_outputs_must_be_there(rowwise):
    """A training call whose outputs lack the transposed copy is refused (the
    library's serving form would leave scale_t and the columns' amax as they
    were); the serving form itself has no use for either."""
    x = torch.zeros((16, 32), dtype=torch.bfloat16)
    for name in ("qt", "scale_t"):
        z = E.alloc_quantized(16, 32, rowwise, "cpu")
        setattr(z, name, None)
        with pytest.raises(ValueError, match="must have qt and scale_t"):
            E.fp8_layernorm_quantize(x, rowwise=rowwise, out=z)
    z = E.Quantized(torch.empty((16, 32), dtype=torch.uint8), None, torch.empty(16), None,
                    torch.empty(16))
    with pytest.raises(ValueError, match="on a GPU"):       # nothing wrong but the device
        E.fp8_layernorm_quantize(x, rowwise=True, transposed=False, out=z)


@pytest.mark.parametrize("rowwise", [False, True], ids=["tensorwise", "rowwise"])
def test_codes_of_h_must_be_there(rowwise):
    """An `out` that holds no codes is refused, not taken for a call without one."""
    x, w = (torch.zeros((n, 48), dtype=torch.uint8) for n in (16, 32))
    sx, sw = (torch.ones(n if rowwise else 1) for n in (16, 32))
    z = E.alloc_quantized(16, 32, rowwise, "cpu")
    for out in (E.Quantized(None, None, None, None, None),
                E.Quantized(None, z.qt, z.scale, z.scale_t, z.amax),
                E.Quantized(z.q, None, z.scale, z.scale_t, z.amax),
                E.Quantized(z.q, z.qt, None, z.scale_t, z.amax),
                E.Quantized(z.q, z.qt, z.scale, None, z.amax)):
        with pytest.raises(ValueError, match="out must have q, qt, scale and scale_t"):
            E.fp8_gated_fwd(x, sx, w, sw, w, sw, rowwise, out=out)
    z.amax = None                                            # optional
    with pytest.raises(ValueError, match="on a GPU"):
        E.fp8_gated_fwd(x, sx, w, sw, w, sw, rowwise, out=z)


def test_workspace_never_shrinks():
    """A workspace sized for the largest batch (or width) serves every
    smaller one, and it holds the partial maxima of both tile sizes: the rows' per
    wave column, the columns' per wave row, of small tiles (64 rows x half a
    large tile's columns) wherever those may be in use."""
    f = E.lib().fp8_gated_workspace_bytes
    Ms = (list(range(0, 320, 16)) + [1, 17, 63, 65, 255, 257] + list(range(320, 4200, 48))
          + [8192, 16384, 65536])
    Hs = [16, 64, 128, 144, 256, 400, 1024, 2048, 3968, 4096, 4112, 8192, 8208, 12272, 14336,
          16384, 16400, 20480, 20496, 28672, 65536, 65552, 131072, 131088]
    for scaling in (0, 1, 2, 3):
        for grid, at in (([sorted(Ms), Hs], lambda u, v: f(u, v, scaling)),
                         ([Hs, sorted(Ms)], lambda u, v: f(v, u, scaling))):
            for v in grid[1]:
                sizes = [at(u, v) for u in grid[0]]
                assert all(p <= q for p, q in zip(sizes, sizes[1:])), (scaling, v, sizes)
    up = lambda n, d: -(-n // d)
    for M in Ms:
        for H in Hs:
            for bn in (128, 256):                # h; da and db
                n = up(M, 256) * up(H, bn)
                few = n <= (128 if bn == 128 else 80) or (M <= 64 and up(H, bn // 2) <= 1024)
                tm, tn = (64, bn // 2) if few else (256, bn)
                need = 2 * 2 * (up(H, tn) * M + up(M, tm) * H)
                assert f(M, H, 1) >= need * (1 if bn == 128 else 2), (M, H, bn)


@no_gpu
def test_every_output_apart_from_every_buffer():
    """An output (or the workspace) that meets any other buffer of its call is
    refused: parameters, scale vectors and amax as well as the matrices, and a
    buffer inside the workspace.  (Fake addresses, 2^24 bytes apart.)"""
    at = lambda names: {n: A + (k << 24) for k, n in enumerate(names.split())}

    def check(call, names, outs):
        apart = at(names)
        for one in outs.split():
            for other in apart:
                if other != one:
                    assert call(**dict(apart, **{one: apart[other]})) == E.FP8L_EINVAL, (one, other)
        if "ws" in apart:
            for other in apart:
                if other != "ws":
                    inside = dict(apart, **{other: apart["ws"] + 64})
                    assert call(**inside) == E.FP8L_EINVAL, (other, "in the workspace")

    n = dict(rows=16, cols=32)
    check(lambda **k: norm_abi.fwd(**n, **k), "x w b y mean rstd", "y mean rstd")
    for scaling in (0, 1):
        check(lambda **k: norm_abi.quant(scaling=scaling, **n, **k),
              "x w b y mean rstd q qt s st amax ws", "y mean rstd q qt s st amax ws")
    check(lambda **k: norm_abi.quant(scaling=1, qt=None, st=None, ws=None, wsb=0, **n, **k),
          "x w b y mean rstd q s amax", "y mean rstd q s amax")
    check(lambda **k: norm_abi.bwd(**n, **k), "dy x w mean rstd dx dw db ws", "dx dw db ws")
    for scaling in (0, 1):
        check(lambda **k: gated_abi.fwd(scaling=scaling, **k),
              "x sx w1 s1 w3 s3 a b h hq hqt s st amax ws", "a b h hq hqt s st amax ws")
    for scaling in (0, 1, 2, 3):
        check(lambda **k: gated_abi.bwd(scaling=scaling, **k),
              "dy sdy w sw a b da db daq daqt das dast daa dbq dbqt dbs dbst dba ws",
              "da db daq daqt das dast daa dbq dbqt dbs dbst dba ws")


def test_stated_errors_of_silu():
    """The header's error bounds against the kernels' sequence in 32 bits
    (hardware exponential and reciprocal taken as correctly rounded, and one unit
    off either way), for every finite bf16 gate: silu relative, silu' absolute.  A
    relative bound of the same size does not hold for silu' near its zero."""
    f32, f64 = np.float32, np.float64
    x = (np.arange(1 << 16, dtype=np.uint32) << 16).view(f32)
    x = x[np.isfinite(x) & (np.abs(x) < 2.0 ** 100)]
    a = x.astype(f64)
    unit = 2.0 ** -23
    with np.errstate(all="ignore"):
        s = 1 / (1 + np.exp(-a))
        u = a * s
        d = s + u * (1 - s)
        r = (np.abs(a) + 4) * unit
        worst = 0.0
        for de in (-1, 0, 1):
            for dr in (-1, 0, 1):
                e = np.exp2((x * f32(-1.44269504088896341)).astype(f64))
                e = (e * (1 + de * unit)).astype(f32)
                sk = (1 / (f32(1) + e).astype(f64) * (1 + dr * unit)).astype(f32)
                uk = x * sk
                dk = (uk.astype(f64) * (f32(1) - sk).astype(f64) + sk).astype(f32)   # one rounding
                assert np.all(np.abs(uk - u) <= r * np.abs(u) + 2.0 ** -119)
                err = np.abs(dk - d)
                assert np.all(err <= r * (s + 2 * np.abs(u)) + 2.0 ** -22 * (s + np.abs(u))
                              + 2.0 ** -118)
                # (no bf16 gate lies so near the zero that da is off by more than a
                # rounding border's width)
                assert np.all((err < 2.0 ** -10 * np.abs(d))[np.abs(a) < 80])
                near = np.abs(a + 1.278) < 0.01
                worst = max(worst, np.max((err / np.abs(d) / r)[near]))
    assert worst > 10
