"""The dK/dV kernel of D = 256 gives the same bits every time: its dV CTA once could take a query tile's slot for
loaded while an earlier dO load of that slot was still in flight."""
import pytest
import torch

from helpers import cuda_or_skip


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [False, True])
def test_wide_dkdv_repeats(causal):
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = torch.Generator(device="cuda")
    g.manual_seed(21)
    q, k, v, dO = (torch.randn(2, 12, 1500, 256, generator=g, device="cuda").bfloat16() for _ in range(4))
    o, lse = fa.fa_forward(q, k, v, causal=causal)
    dq, delta = fa.fa_backward_dq(q, k, v, o, dO, lse, causal=causal)
    dk, dv = fa.fa_backward_dkdv(q, k, v, dO, lse, delta, causal=causal)
    busy = torch.empty(64 << 20, device="cuda")
    for i in range(60):
        if i % 3 == 0:
            busy.fill_(i)  # evicts the operands from L2, so loads come back out of order
        again = fa.fa_backward_dkdv(q, k, v, dO, lse, delta, causal=causal)
        assert torch.equal(again[0], dk) and torch.equal(again[1], dv), i
    assert fa.fa_device_status() == 0
