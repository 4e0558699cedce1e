"""The Muon step with a factor, its first iterations on e4m3 operands."""
import pytest
import torch

import newton_schulz_03_amd as nsa

BF16 = torch.bfloat16


@pytest.mark.gpu
@pytest.mark.parametrize("nesterov", [False, True])
def test_e4m3_steps_with_a_power_of_two_factor(nesterov):
    """s = 1/4 multiplies exactly, so the step on g equals the plain step on g / 4."""
    gen = torch.Generator().manual_seed(61)
    ws, gs, ms = ([(torch.randn(s, generator=gen) * 1e-2).to(BF16).cuda()
                   for s in ((300, 700), (700, 300), (257, 771))] for _ in range(3))
    ws2, ms2 = [w.clone() for w in ws], [m.clone() for m in ms]
    nsa.step_batched(ws, gs, ms, nesterov=nesterov, fp8_steps=2,
                     grad_scale=torch.full((1,), 0.25, device="cuda"))
    nsa.step_batched(ws2, [g * 0.25 for g in gs], ms2, nesterov=nesterov, fp8_steps=2)
    assert all(torch.equal(a, b) for a, b in zip(ws + ms, ws2 + ms2))
