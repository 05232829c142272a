"""MLPStep.flops against the products that a step runs (no GPU: the entry points are
replaced by ones that count)."""
import pytest
import torch

from float8_mixed_precision_amd import ops


@pytest.mark.parametrize("bias", [True, False], ids=["bias", "no_bias"])
def test_flops_are_those_of_the_products(monkeypatch, bias):
    M, D, H = 48, 32, 80
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    one = torch.ones(D, dtype=torch.bfloat16)
    step = ops.MLPStep(ops.alloc_quantized(M, D, False, "cpu"), bf(M, D), bf(H, D),
                       bf(H) if bias else None, bf(D, H), bf(D) if bias else None, bf(M, D),
                       bf(M, D), pre=(one, one))
    done = []

    def product(a, b):
        (m, k), n = a.shape, b.shape[0]
        assert b.shape[1] == k
        done.append(2 * m * n * k)

    monkeypatch.setattr(ops, "fp8_linear_act_fwd", lambda xq, sx, wq, sw, *a, **k: product(xq, wq))
    monkeypatch.setattr(ops, "fp8_linear_act_bwd", lambda dyq, sdy, wtq, *a, **k: product(dyq, wtq))
    monkeypatch.setattr(ops, "fp8_linear_gemm_grouped",
                        lambda problems, *a, **k: [product(p[0], p[2]) for p in problems])
    for name in ("fp8_linear_quantize", "fp8_resnorm_quantize", "fp8_resnorm_bwd",
                 "fp8_bias_act_bwd"):
        monkeypatch.setattr(ops, name, lambda *a, **k: None)
    step.run()
    assert len(done) == 6 and step.flops == sum(done)
