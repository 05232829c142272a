"""The inverse deviation alone, where its argument is exact in 32 bits: rows of
one nonzero element c with 12 significant bits, in 2^k columns without eps,
whose mean square c^2 / 2^k is an fp32 number.  rstd = 2^(k/2) / |c| may then
be off by its own rounding, half a unit in its last place, and by what the
kernel's Newton step leaves: with an estimate off by d <= 2^-23 relatively, 3/2
d^2, and 2^-24 2 d for the residual's rounding, below 2^-44 in all or 2^-20
units."""
import numpy as np
import pytest
import torch

from float8_mixed_precision_amd import ops
from tests import gpu_util as G

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("cols", [4, 64, 1024, 4096, 16384])
def test_rounded_once(cols, dtype):
    bits = 8 if dtype is torch.bfloat16 else 12
    rows = 1 << 11
    c = (1 << bits - 1) + np.arange(rows) % (1 << bits - 1)          # bits significant bits
    c = c * 2.0 ** (np.arange(rows) // 64 % 31 - 15.0 - bits)
    x = torch.zeros((rows, cols), dtype=dtype)
    x[torch.arange(rows), torch.arange(rows) * 7 % cols] = torch.from_numpy(c).to(dtype)
    assert torch.equal(x.double().sum(1), torch.from_numpy(c))       # c is exact in this type
    G.say("rstd", cols, dtype)
    _, _, rstd = ops.fp8_layernorm_fwd(x.to(G.DEV), eps=0.0, rms=True)
    torch.cuda.synchronize()
    got = G.host(rstd).astype(np.float64)
    want = np.sqrt(float(cols)) / c
    unit = 2.0 ** (np.floor(np.log2(want)) - 23)
    off = np.abs(got - want) / unit
    assert off.max() <= 0.5 + 2.0 ** -20, (off.max(), int(off.argmax()))


def test_ends_of_the_range():
    """No deviation and no eps: infinity.  Squares past the range: 0.  Squares
    whose mean lies below the normal range: still the root's value."""
    x = torch.zeros((4, 64))
    x[1, 3] = 2.0 ** 64
    x[2, 5] = 2.0 ** -70                         # mean square 2^-146, exact
    x[3, :] = float("nan")
    G.say("rstd ends")
    _, _, rstd = ops.fp8_layernorm_fwd(x.to(G.DEV), eps=0.0, rms=True)
    torch.cuda.synchronize()
    r = rstd.cpu().numpy()
    assert np.isposinf(r[0]) and r[1] == 0 and r[2] == 2.0 ** 73 and np.isnan(r[3])
