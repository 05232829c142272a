"""What the norm's and the gated feed-forward's entry points promise beyond
their argument checks: host side, no GPU needed."""
import pytest
import torch

from float8_mixed_precision_amd import ops as E


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
