"""GPU test of the balance loss's gradient written over its own logits, at every row width."""

import pytest
import torch

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("fp8_quantized_moe_gb300")


@pytest.mark.parametrize("E", [1, 7, 32, 33, 64, 90, 96, 128, 130, 192, 256, 384, 511, 512, 700, 768, 1000, 1024])
@pytest.mark.parametrize("T,seqs,padded", [(5, 1, False), (1203, 3, True), (20000, 4, False)])
def test_gradient_over_the_logits(T, seqs, padded, E):
    g = torch.Generator(device="cuda").manual_seed(T + E)
    T = T // seqs * seqs
    logits = 3 * torch.randn(T, E, generator=g, device="cuda")
    ids = torch.randint(0, E, (T, min(E, 3)), generator=g, device="cuda", dtype=torch.int32)
    valid = torch.rand(T, generator=g, device="cuda") < 0.7 if padded else None
    b = moe.router_balance_loss(logits, ids, 0.5, seqs=seqs, valid=valid)
    want = moe.router_balance_loss_backward(logits, b)
    for _ in range(3):
        x = logits.clone()
        got = moe.router_balance_loss_backward(x, b, out=x)
        assert got.data_ptr() == x.data_ptr() and torch.equal(x, want)
    assert moe.device_error() == 0 and (E == 1 or want.any())
