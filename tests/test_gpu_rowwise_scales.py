"""Rowwise quantize on both sides of where the cast takes its scales from the
partial maxima itself (up to 96 partials of a row or a column, and few tiles):
codes, scales and amax bit for bit the oracle's, on a workspace that holds
garbage, with specials in the first and last rows and columns.  (Where a row or
column holds a NaN or an infinity its amax says so and its codes are
unspecified.)"""
import numpy as np
import pytest
import torch

import oracle
from float8_mixed_precision_amd import ops
from tests import gpu_util as G

pytestmark = pytest.mark.gpu

# partials: one per 256 columns of a row, one per 64 rows of a column
SIZES = [(16, 16), (144, 272), (6144, 16), (6160, 16), (16, 24576), (16, 24592), (2048, 4096),
         (2064, 5136), (4096, 3088)]


def _bits(rows, cols):
    rng = np.random.default_rng(rows * 31 + cols)
    x = rng.standard_normal((rows, cols)).astype(np.float32)
    x *= np.exp2(rng.integers(-6, 7, (rows, 1))).astype(np.float32)
    b = (x.view(np.uint32) >> 16).astype(np.uint16)
    b[0, -1] = 0x7F80                                  # +inf
    b[-1, 0] = 0xFFC1                                  # NaN
    b[1] = 0                                           # an empty row
    b[:, 3] = 0x8000                                   # a column of -0
    return b


def _check(got, ref, rows, label):
    q, qt, scale, scale_t, amax = got
    am = ref[4]
    if amax is not None:
        assert np.array_equal(np.isnan(amax), np.isnan(am)), label
        assert np.array_equal(amax[~np.isnan(am)], am[~np.isnan(am)]), label
    for name, codes, want, s, ws, fin in (
            ("q", q, ref[0], scale, ref[2], np.isfinite(am[:rows])),
            ("qt", qt, ref[1], scale_t, ref[3], np.isfinite(am[rows:]))):
        assert fin.sum() >= len(fin) - 2
        assert np.array_equal(s[fin].view(np.uint32), ws[fin].view(np.uint32)), (label, name)
        assert np.array_equal(codes[fin], want[fin]), (label, name)


@pytest.mark.parametrize("e5m2", [False, True], ids=["e4m3", "e5m2"])
@pytest.mark.parametrize("shape", SIZES, ids=lambda s: "%dx%d" % s)
def test_quantize(shape, e5m2):
    rows, cols = shape
    bits = _bits(rows, cols)
    G.say("rowwise scales", shape, "e5m2", e5m2)
    ws = torch.full((ops.fp8_linear_workspace_bytes(rows, cols, True) or 256,), 0x7F,
                    dtype=torch.uint8, device=G.DEV)
    q = ops.fp8_linear_quantize(G.dev_bf16(bits), True, None, ws, e5m2=e5m2)
    torch.cuda.synchronize()
    ref = oracle.quantize_e5m2(bits, True) if e5m2 else oracle.quantize(bits, True)
    _check(tuple(G.host(t) for t in (q.q, q.qt, q.scale, q.scale_t, q.amax)), ref, rows,
           "%s" % (shape,))


def test_without_amax_and_unaligned_scales():
    """No amax vector, scale vectors at 4-byte addresses, and the floats
    around them left as they were."""
    rows, cols = 144, 272
    bits = _bits(rows, cols)
    G.say("rowwise scales unaligned")
    x = G.dev_bf16(bits)
    u8 = lambda *s: torch.empty(s, dtype=torch.uint8, device=G.DEV)
    q, qt, ws = u8(rows, cols), u8(cols, rows), u8(ops.fp8_linear_workspace_bytes(rows, cols, True))
    s = torch.full((rows + 2,), -7.0, device=G.DEV)
    st = torch.full((cols + 2,), -7.0, device=G.DEV)
    rc = ops.lib().fp8_linear_quantize(x.data_ptr(), rows, cols, 1, q.data_ptr(), qt.data_ptr(),
                                       s[1:].data_ptr(), st[1:].data_ptr(), None, ws.data_ptr(),
                                       ws.numel(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0
    ref = oracle.quantize(bits, True)
    s, st = G.host(s), G.host(st)
    _check((G.host(q), G.host(qt), s[1:-1], st[1:-1], None), ref, rows, "unaligned")
    assert s[0] == s[-1] == st[0] == st[-1] == -7.0
