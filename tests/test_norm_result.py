"""The result of a gradient norm or clip: eight bytes that a caller keeps from step
to step (a log of norms), and nothing else with them."""
import io

import pytest
import torch

import newton_schulz_03_amd as nsa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("count", [1, 5, 300])
def test_a_kept_result_keeps_nothing_else(count):
    gs = [torch.randn(100 + i, device="cuda") for i in range(count)]
    for r in (nsa.grad_norm_batched(gs), nsa.grad_norm_batched(gs, max_norm=1.0),
              nsa.grad_clip_batched(gs, 1.0)):
        assert r.shape == (2,) and r.dtype == torch.float32 and r.is_contiguous()
        assert r.untyped_storage().nbytes() == 8 and r.storage_offset() == 0
        file = io.BytesIO()
        torch.save(r, file)
        assert file.tell() < 4096


def test_memory_of_kept_results():
    gs = [torch.randn(1000, device="cuda")]
    nsa.grad_norm_batched(gs)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    kept = [nsa.grad_norm_batched(gs, max_norm=1.0) for _ in range(100)]
    # an allocation takes 512 bytes
    assert torch.cuda.memory_allocated() - before <= 512 * len(kept)
