"""Workspaces that the step, the orthogonalization and AdamW refuse before anything is
enqueued: in host memory, or with gaps."""
import pytest
import torch

import newton_schulz_03_amd as nsa

pytestmark = pytest.mark.gpu


def calls():
    """(name, bytes of workspace, call with a workspace, its tensors)."""
    shape = (64, 100)
    w, g, m = (torch.randn(shape, device="cuda").bfloat16() for _ in range(3))
    p, d, a, b = (torch.rand(1000, device="cuda") for _ in range(4))
    size = nsa.workspace_bytes([shape], torch.bfloat16)
    out = torch.empty_like(g)
    return [("step", size, lambda ws: nsa.step_batched([w], [g], [m], workspace=ws), (w, m)),
            ("orthogonalization", size, lambda ws: nsa.ns_batched([g], out=[out], workspace=ws), (out,)),
            ("adamw", nsa.adamw_workspace_bytes([1000]),
             lambda ws: nsa.adamw_batched([p], [d], [a], [b], workspace=ws), (p, a, b))]


def test_refused():
    for name, size, call, tensors in calls():
        before = [t.clone() for t in tensors]
        for ws in (torch.empty(2 * size + 256, dtype=torch.uint8),
                   torch.empty(2 * size + 256, dtype=torch.uint8, pin_memory=True),
                   torch.empty(2 * size + 512, dtype=torch.uint8, device="cuda")[::2]):
            with pytest.raises(ValueError, match="workspace"):
                call(ws)
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(tensors, before)), name


def test_taken():
    for name, size, call, _ in calls():
        room = torch.empty(size + 512, dtype=torch.uint8, device="cuda")
        call(room[(-room.data_ptr()) % 256:])
    torch.cuda.synchronize()
