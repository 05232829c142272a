"""The linear with its epilogue at the ends of its ranges: calls that enqueue nothing
or that the library refuses on the host (fake device addresses, so only where no
GPU is visible)."""
import ctypes

import pytest
import torch

from float8_mixed_precision_amd import ops as E

A = 0x10000
P = lambda v: ctypes.c_void_p(v) if v else None
no_gpu = pytest.mark.skipif(torch.cuda.device_count() != 0,
                            reason="fake-pointer cases run without a GPU only")


@no_gpu
@pytest.mark.parametrize("act", [E.FP8L_ACT_NONE, E.FP8L_ACT_GELU])
@pytest.mark.parametrize("q,scale,amax", [(A, A, A), (A, None, None), (None, A, None),
                                          (None, None, A)])
@pytest.mark.parametrize("y,z", [(A, A), (A, None), (None, A), (None, None)])
def test_codes_of_no_rows(y, z, q, scale, amax, act):
    """M = 0 tokens with the outputs of the serving form in hand (qt and scale_t absent):
    there is nothing to write and nothing is enqueued."""
    for N, K in ((32, 48), (0, 48), (32, 0), (8208, 4112)):
        at = iter(range(A, 1 << 40, 1 << 28))
        new = lambda v: P(next(at)) if v else None
        ok = E.lib().fp8_linear_act_fwd(
            new(A), new(A), new(A), new(A), 0, N, K, E.FP8L_ROWWISE, new(A), E.FP8L_BF16, act,
            None, new(z), new(y), new(q), None, new(scale), None, new(amax), new(A), 1 << 27, None)
        assert ok == E.FP8L_OK, (N, K)


# Sizes whose launches would reach 2^32 threads, the most that HIP takes, and ones that
# stay just below: a cast of 512 threads for each tile of 128 x 128 (and for every 64
# columns whose sums are finished beside it), a rowwise quantize's scales at 8 threads
# a row and a column.
TILES, ROWS = 1 << 30, 1 << 29
TOO_MANY = [(0, TILES, 16), (0, TILES - 112, 16), (0, 1 << 29, 144), (2, TILES, 128),
            (1, ROWS, 16), (3, ROWS - 64, 16), (1, 16, ROWS)]
FIT = [(0, TILES - 512, 16), (2, (1 << 29) - 512, 144), (1, ROWS - 128, 16), (3, 16, 1 << 27)]


def _apart():
    at = iter(range(A, 1 << 62, 1 << 44))
    return lambda: P(next(at))


def _bias_act(scaling, M, N, dbias=True):
    new = _apart()
    return E.lib().fp8_bias_act_bwd(new(), new(), M, N, scaling, E.FP8L_ACT_GELU, new(), new(), new(),
                                    new(), new(), new(), new() if dbias else None, E.FP8L_BF16,
                                    new(), 1 << 43, None)


def _quantize(scaling, M, N):
    new = _apart()
    return E.lib().fp8_linear_quantize(new(), M, N, scaling, new(), new(), new(), new(), new(),
                                       new(), 1 << 43, None)


def _swiglu(scaling, M, N):
    new = _apart()
    return E.lib().fp8_swiglu_fwd(new(), new(), M, N, scaling & 1, *(new() for _ in range(7)),
                                  1 << 43, None)


def _norm(scaling, M, N):
    new = _apart()
    return E.lib().fp8_layernorm_quantize(
        new(), M, N, E.FP8L_RMSNORM, new(), new(), E.FP8L_BF16, 1e-5, scaling & 1, new(), new(),
        new(), new(), new(), new(), new(), new(), new(), 1 << 43, None)


def _resnorm(scaling, M, N, grads=None):
    new = _apart()
    z = lambda: new().value
    r = E._RESNORM.pack(M, N, E.FP8L_RMSNORM, E.FP8L_POST_NORM | E.FP8L_PRE_NORM, E.FP8L_BF16,
                        E.FP8L_BF16, 1.0, 1e-5, *(z() for _ in range(13)))
    if grads is None:
        return E.lib().fp8_resnorm_quantize(r, scaling & 1, new(), new(), new(), new(), new(),
                                            new(), 1 << 43, None)
    g = E._RESNORM_GRADS.pack(z(), z(), *((z() if grads else 0) for _ in range(5)))
    return E.lib().fp8_resnorm_bwd(r, new(), new(), g, scaling, new(), new(), new(), new(), new(),
                                   new(), 1 << 43, None)


@no_gpu
@pytest.mark.parametrize("call", [
    _bias_act, lambda *a: _bias_act(*a, dbias=False), _quantize, _swiglu, _norm, _resnorm,
    lambda *a: _resnorm(*a, True), lambda *a: _resnorm(*a, False)],
    ids=["bias_act", "bias_act_no_sums", "quantize", "swiglu", "layernorm", "resnorm",
         "resnorm_bwd", "resnorm_bwd_no_sums"])
def test_sizes_past_a_launch(call):
    wide = call in (_bias_act, _quantize, _swiglu)
    for scaling, M, N in TOO_MANY:
        if N <= E.FP8L_NORM_MAX_COLS or wide:
            assert call(scaling, M, N) == E.FP8L_ESHAPE, (scaling, M, N)
    for scaling, M, N in FIT:
        # (without a device the launch itself fails)
        if N <= E.FP8L_NORM_MAX_COLS or wide:
            assert call(scaling, M, N) == E.FP8L_EHIP, (scaling, M, N)


@no_gpu
def test_sums_beside_the_cast_count():
    """The workgroups that finish sums of columns belong to the cast's launch."""
    M = TILES - 128                                    # 2^23 - 1 tiles
    assert _quantize(0, M, 16) == _bias_act(0, M, 16, dbias=False) == E.FP8L_EHIP
    assert _bias_act(0, M, 16) == E.FP8L_ESHAPE
    assert _resnorm(0, M, 16, False) == E.FP8L_EHIP
    assert _resnorm(0, M, 16, True) == E.FP8L_ESHAPE
    assert _resnorm(0, M - 128, 16, True) == E.FP8L_ESHAPE
    assert _resnorm(0, M - 256, 16, True) == E.FP8L_EHIP


@no_gpu
def test_casts_past_a_launch():
    """The cast with a given scale, whatever scaling its scale came from."""
    def call(M, N):
        new = _apart()
        return E.lib().fp8_linear_quantize_scaled(new(), M, N, new(), new(), new(), None)

    for scaling, M, N in TOO_MANY:
        if scaling in (0, 2):
            assert call(M, N) == E.FP8L_ESHAPE, (M, N)
    for _, M, N in FIT:
        assert call(M, N) == E.FP8L_EHIP, (M, N)
    assert call(TILES, 0) == E.FP8L_OK
