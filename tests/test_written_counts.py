"""Tensors that the expert layers' operators write count the write, so that autograd
refuses to go back through what it saved of their old values."""
import pytest
import torch

import newton_schulz_03_amd as nsa
from newton_schulz_03_amd._binding import _lists


def test_the_count():
    a, b = torch.zeros(3), torch.zeros(4)
    view = a[:2]
    _lists().wrote(a, b, None)
    _lists().wrote(b)
    assert (a._version, view._version, b._version) == (1, 1, 2)
    with torch.inference_mode():
        c = torch.zeros(3)
    _lists().wrote(c)  # has no counter
    _lists().wrote()
    for bad in ([a], 3):
        with pytest.raises(TypeError):
            _lists().wrote(a, bad)
    assert a._version == 1


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(7, 16), (300, 1024)])
def test_dropout_of_a_saved_tensor_is_noticed(shape):
    x = torch.randn(shape, device="cuda", requires_grad=True)
    y = x.exp()  # its gradient reads y
    nsa.dropout_batched([y], 0.5, seed=1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    y = x.exp()
    out = nsa.dropout_batched([y], 0.5, seed=1, out=[torch.empty_like(y)])[0]
    assert (y._version, out._version) == (0, 1)
    y.sum().backward()
    assert torch.equal(x.grad, y.detach())


@pytest.mark.gpu
def test_given_outputs():
    ids = torch.tensor([[0, 1], [2, 0], [1, 2]], dtype=torch.int32, device="cuda")
    x = torch.randn((3, 40), device="cuda").bfloat16()
    w = torch.rand((3, 2), device="cuda")
    plan = nsa.moe_empty_plan(3, 2, 3, "cuda")
    nsa.moe_sort(ids, 3, plan=plan)
    assert all(t._version > 0 for t in plan)
    ys, out, dw = torch.zeros((6, 40), device="cuda").bfloat16(), torch.zeros_like(x), torch.zeros_like(w)
    dys = torch.zeros_like(ys)
    before = [t._version for t in (ys, out, dys, dw)]
    nsa.moe_dispatch(x, plan, out=ys)
    nsa.moe_combine(ys, plan, weights=w, out=out)
    nsa.moe_combine_backward(x, ys, plan, w, dys=dys, dweights=dw)
    assert [t._version for t in (ys, out, dys, dw)] == [v + 1 for v in before]
    op = nsa.f4_empty(3, 24, 40, "cuda")
    nsa.f4_quantize([torch.randn((24, 40), device="cuda") for _ in range(3)], out=op)
    y = torch.zeros((6, 24), device="cuda")
    nsa.f4_matmul(x, op, plan=plan, gather=True, out=y)
    assert (op.q._version, op.scales._version, y._version) == (1, 1, 1)
    # a call that is refused has written nothing
    with pytest.raises(ValueError):
        nsa.moe_combine(ys, plan, weights=w[:2], out=out)
    with pytest.raises(nsa.MuonError):
        nsa.dropout_batched([out], 2.0)
    assert out._version == before[1] + 1
    # read, not written
    assert x._version == w._version == ids._version == 0
    with torch.inference_mode():
        nsa.dropout_batched([torch.ones(5, device="cuda")], 0.5)
        kept = torch.zeros(5, device="cuda")
    nsa.dropout_batched([kept], 0.5)
