"""Counts of more than 32 bits are refused, and do not pass as what their low bits say."""
import pytest

import newton_schulz_03_amd as nsa

WIDE = [(1 << 31), (1 << 32) + 8, (1 << 62) + 8, (1 << 64) + 8, -(1 << 32) + 8, -(1 << 64) + 8]


@pytest.mark.parametrize("n", WIDE)
def test_refused(n):
    for call in (lambda: nsa.moe_workspace_bytes(1, 1, n), lambda: nsa.moe_workspace_bytes(1, n, 8),
                 lambda: nsa.moe_workspace_bytes(n, 1, 8), lambda: nsa.f4_workspace_bytes(n)):
        with pytest.raises(nsa.MuonError):
            call()


@pytest.mark.gpu
@pytest.mark.parametrize("n", WIDE)
def test_sort_refuses(n):
    import torch

    ids = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    with pytest.raises(nsa.MuonError):
        nsa.moe_sort(ids, n)
