"""The workspace of the token sort serves every shorter list too, on both sides of the
sizes at which the sort cuts a list differently."""
import pytest
import torch

import expert_plain as plain
import newton_schulz_03_amd as nsa

SIZES = [1, 1024, 4096, 4097, 5000, 65535, 65536, 65537, 131072, 1310720, 1310721, 2621440, 2621441,
         nsa.MOE_MAX_SLOTS]


@pytest.mark.parametrize("experts", [1, 2, 7, 384, 1023, 1024])
def test_never_less_for_more_slots(experts):
    sizes = sorted({n for s in SIZES for n in (s - 1, s, s + 1) if n <= nsa.MOE_MAX_SLOTS}
                   | set(range(4000, 70000, 333)) | set(range(70000, nsa.MOE_MAX_SLOTS, 33333)))
    got = [nsa.moe_workspace_bytes(n, 1, experts) for n in sizes]
    assert got == sorted(got)
    # by the slots alone, however many a token has
    assert nsa.moe_workspace_bytes(65536, 1, experts) == nsa.moe_workspace_bytes(8192, 8, experts)


def test_never_less_for_more_experts():
    for n in SIZES:
        got = [nsa.moe_workspace_bytes(n, 1, e) for e in range(1, nsa.MOE_MAX_EXPERTS + 1)]
        assert got == sorted(got)


@pytest.mark.gpu
def test_one_workspace_for_every_size():
    room = torch.empty(nsa.moe_workspace_bytes(1310721, 1, 384), dtype=torch.uint8, device="cuda")
    gen = torch.Generator().manual_seed(1)
    for n in (1310721, 1310720, 131072, 65537, 65536, 5000, 4097, 4096, 1):
        ids = torch.randint(-1, 385, (n, 1), generator=gen, dtype=torch.int32)
        got = nsa.moe_sort(ids.cuda(), 384, workspace=room)
        for name, g, w in zip(got._fields, got, plain.plan(ids.numpy(), 384)):
            assert (g.cpu().numpy() == w).all(), (n, name)
