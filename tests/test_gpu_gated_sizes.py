"""GPU gated feed-forward at the borders between its kernels: batches that
shrink under one workspace, token counts and widths on both sides of each
choice of kernel.  Outputs are compared with the plain GEMM's and with calls of
their own workspace, codes with the oracle's quantize."""
import numpy as np
import pytest
import torch

import oracle
from float8_mixed_precision_amd import ops
from float8_mixed_precision_amd import workloads as W
from tests import gpu_util as G
from tests import test_gpu_gated
from tests.test_gpu_gated import RW, RW_IDS, _hq, _pad16, _weights, _x, check_dab, check_h

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rowwise", RW, ids=RW_IDS)
def test_one_workspace_for_shrinking_batches(rowwise):
    """The workspace of the largest batch serves the smaller ones (small tiles
    take more partial maxima than large ones), and nothing is written behind it."""
    H, K = 4096, 144
    size = ops.fp8_gated_workspace_bytes(1296, H, rowwise)
    buf = torch.full((size + 4096,), 0x5A, dtype=torch.uint8, device=G.DEV)
    (w1, s1), (w3, s3) = _weights(H, K, rowwise, 90)
    w2 = ops.fp8_linear_quantize(G.dev_bf16(W.random_bf16(90, (K, H), 0.02, 3)), rowwise)
    for M in (1296, 1280, 272, 16):
        G.say("gated workspace", M, "rowwise", rowwise)
        xq, sx = _x(M, K, rowwise, 91)
        out = []
        for ws in (buf[:size], ops.alloc_gated_workspace(M, H, rowwise, G.DEV)):
            a, b = (torch.empty((M, H), dtype=torch.bfloat16, device=G.DEV) for _ in range(2))
            z = ops.alloc_quantized(M, H, rowwise, G.DEV)
            h = ops.fp8_gated_fwd(xq, sx, w1, s1, w3, s3, rowwise, a=a, b=b, out=z, workspace=ws)
            da, db, qa, qb = ops.fp8_gated_bwd(xq, sx, w2.qt, w2.scale_t, a, b, rowwise,
                                               workspace=ws)
            torch.cuda.synchronize()
            out.append([G.host(t) for t in (h, da, db)] + [t for q in (z, qa, qb) for t in _hq(q)])
        for p, q in zip(*out):
            assert np.array_equal(p, q), M
        assert torch.all(buf[size:] == 0x5A)


# Large tiles with fewer rows than a wave's 128 (and than the 120 rows that its
# row offsets reach): one row of tiles, more than 128 (forward) or 80 (backward)
# of them; up to 64 rows where even the small tiles would be more than 1024.
@pytest.mark.parametrize("rowwise", RW, ids=RW_IDS)
@pytest.mark.parametrize("mh", [(80, 16400), (112, 16512), (67, 16400), (48, 65552)],
                         ids=lambda s: "%dx%d" % s)
def test_forward_one_row_of_large_tiles(mh, rowwise):
    M, H = mh
    K = 144
    P = _pad16(M)
    xq, sx = _x(M, K, rowwise, 92)
    (w1, s1), (w3, s3) = _weights(H, K, rowwise, 92)
    G.say("gated fwd, one row of large tiles", mh, "rowwise", rowwise)
    pa, pb = (ops.fp8_linear_fwd(xq, sx, w, s, rowwise) for w, s in ((w1, s1), (w3, s3)))
    xs, ss = xq[:M].clone(), sx[:M].clone() if rowwise else sx
    z = ops.alloc_quantized(M, H, rowwise, G.DEV) if M == P else None
    bufs = [torch.full((P + 1, H), 7.0, dtype=torch.bfloat16, device=G.DEV) for _ in range(3)]
    h = ops.fp8_gated_fwd(xs, ss, w1, s1, w3, s3, rowwise, h=bufs[0][:M], a=bufs[1][:M],
                          b=bufs[2][:M], out=z)
    h2 = ops.fp8_gated_fwd(xs, ss, w1, s1, w3, s3, rowwise)
    torch.cuda.synchronize()
    assert torch.equal(bufs[1][:M], pa[:M]) and torch.equal(bufs[2][:M], pb[:M])
    assert torch.equal(h, h2)
    for t in bufs:
        assert torch.all(t[M:] == 7.0)
    check_h(G.host(h), G.host(pa[:M]), G.host(pb[:M]), "h %s" % (mh,))
    if z is not None:
        G.assert_quantize_equal(_hq(z), oracle.quantize(G.host(h), rowwise), "codes %s" % (mh,))


@pytest.mark.parametrize("rowwise", RW, ids=RW_IDS)
@pytest.mark.parametrize("mh", [(80, 20496), (112, 20736), (16, 131088)],
                         ids=lambda s: "%dx%d" % s)
def test_backward_one_row_of_large_tiles(mh, rowwise):
    M, H = mh
    D = 80
    qdy = ops.fp8_linear_quantize(G.dev_bf16(W.random_bf16(93, (M, D), 1e-2, 0)), rowwise)
    qw = ops.fp8_linear_quantize(G.dev_bf16(W.random_bf16(93, (D, H), 0.02, 1)), rowwise)
    a, b = W.random_bf16(94, (M, H), 3.0, 0), W.random_bf16(94, (M, H), 1.0, 1)
    G.say("gated bwd, one row of large tiles", mh, "rowwise", rowwise)
    da, db, qa, qb = ops.fp8_gated_bwd(qdy.q, qdy.scale, qw.qt, qw.scale_t, G.dev_bf16(a),
                                       G.dev_bf16(b), rowwise)
    dh, _ = ops.fp8_linear_bwd(qdy.q, qdy.scale, None, None, qw.qt, qw.scale_t, None, None, M, D,
                               H, rowwise, want_w=False)
    torch.cuda.synchronize()
    check_dab(G.host(da), G.host(db), G.host(dh), a, b, "bwd %s" % (mh,))
    for z, t in ((qa, da), (qb, db)):
        G.assert_quantize_equal(_hq(z), oracle.quantize(G.host(t), rowwise), "codes %s" % (mh,))


# 5 to 16 tokens on both sides of where the few-token kernel hands over to the
# small tiles (192 of 64 columns), and 4 tokens, which it keeps at any width.
@pytest.mark.parametrize("rowwise", RW, ids=RW_IDS)
@pytest.mark.parametrize("mh", [(4, 14336), (5, 12272), (16, 12272), (5, 12288), (8, 14336),
                                (13, 14336), (16, 12288), (16, 14336)],
                         ids=lambda s: "%dx%d" % s)
def test_decode_batches_of_wide_blocks(mh, rowwise):
    """a, b within the instruction's bound of the oracle's, h from them, the
    codes of h at 16 tokens (test_few_tokens' checks); the small tiles' a and b
    are the plain GEMM's bits, at any number of tokens the padded call's."""
    M, H = mh
    K = 272
    test_gpu_gated.test_few_tokens((M, H, K), rowwise)
    if M > 4 and H >= 12288:
        xq, sx = _x(M, K, rowwise, 95)
        (w1, s1), (w3, s3) = _weights(H, K, rowwise, 95)
        G.say("gated decode batch", mh, "rowwise", rowwise)
        pa, pb = (ops.fp8_linear_fwd(xq, sx, w, s, rowwise) for w, s in ((w1, s1), (w3, s3)))
        xs, ss = xq[:M].clone(), sx[:M].clone() if rowwise else sx
        a, b = (torch.empty((M, H), dtype=torch.bfloat16, device=G.DEV) for _ in range(2))
        ops.fp8_gated_fwd(xs, ss, w1, s1, w3, s3, rowwise, a=a, b=b)
        torch.cuda.synchronize()
        assert torch.equal(a, pa[:M]) and torch.equal(b, pb[:M])


@pytest.mark.parametrize("rowwise", RW, ids=RW_IDS)
def test_outputs_of_almost_2_31_bytes(rowwise):
    """[M, H] bf16 matrices just below 2^31 bytes, the largest that are taken: a
    and b are the plain GEMM's, h, da and db follow from them in sampled rows (first,
    last, random), the amax is that of the stored matrix and a sampled row's
    rowwise codes are the oracle's; nothing is written behind an output."""
    M, H, K = 65520, 16384, 32
    xq, sx = _x(M, K, rowwise, 96)
    (w1, s1), (w3, s3) = _weights(H, K, rowwise, 96)
    w2 = ops.fp8_linear_quantize(G.dev_bf16(W.random_bf16(97, (K, H), 0.02, 3)), rowwise)
    G.say("gated 2^31 bytes", "rowwise", rowwise)
    bufs = [torch.full((M * H + 4096,), 7.0, dtype=torch.bfloat16, device=G.DEV)
            for _ in range(5)]
    h, a, b, da, db = (t[:M * H].view(M, H) for t in bufs)
    z = ops.alloc_quantized(M, H, rowwise, G.DEV)
    ws = ops.alloc_gated_workspace(M, H, rowwise, G.DEV)
    ops.fp8_gated_fwd(xq, sx, w1, s1, w3, s3, rowwise, h=h, a=a, b=b, out=z, workspace=ws)
    for t, w, s in ((a, w1, s1), (b, w3, s3)):
        assert torch.equal(t, ops.fp8_linear_fwd(xq, sx, w, s, rowwise))
    _, _, qa, qb = ops.fp8_gated_bwd(xq, sx, w2.qt, w2.scale_t, a, b, rowwise, da=da, db=db,
                                     workspace=ws)
    dh, _ = ops.fp8_linear_bwd(xq, sx, None, None, w2.qt, w2.scale_t, None, None, M, K, H, rowwise,
                               want_w=False)
    torch.cuda.synchronize()
    for t in bufs:
        assert torch.all(t[M * H:] == 7.0)
    rows = torch.tensor(sorted({0, 1, M - 1, M - 2, 65279, 65280}
                               | set(np.random.default_rng(5).integers(0, M, 26).tolist())),
                        device=G.DEV)
    some = lambda t: G.host(t[rows])
    check_h(some(h), some(a), some(b), "h")
    check_dab(some(da), some(db), some(dh), some(a), some(b), "da db")
    for q, t in ((z, h), (qa, da), (qb, db)):
        if rowwise:
            assert torch.equal(q.amax[:M], t.abs().amax(1).float())
            assert torch.equal(q.amax[M:], t.abs().amax(0).float())
            sample = some(t)
            for k, r in enumerate(rows.tolist()):
                ref = oracle.quantize(np.repeat(sample[k:k + 1], 16, 0), True)
                assert np.array_equal(G.host(q.q[r]), ref[0][0]), r
        else:
            assert q.amax.item() == t.abs().amax().item()
