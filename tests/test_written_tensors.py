"""Tensors that share their data copy-on-write (torch._lazy_clone): a call that
writes one leaves the others as they were, and one that is only read keeps sharing."""
import math
from array import array

import pytest
import torch

import newton_schulz_03_amd as nsa
from newton_schulz_03_amd._binding import F8_BLOCK, _lists


def shares(a, b):
    """Whether two tensors have one address, without giving either its own memory."""
    one, other = (array("q", _lists().scan([t], False)[4])[0] for t in (a, b))
    return one == other


def test_addresses_of_read_and_written_tensors():
    x = torch.arange(6.0)
    y = torch._lazy_clone(x)
    assert shares(x, y)
    (at,) = array("q", _lists().scan([y], True)[4])
    assert not shares(x, y) and at == y.data_ptr()
    y.fill_(7)
    assert torch.equal(x, torch.arange(6.0))


@pytest.mark.gpu
def test_addresses_of_read_and_written_operands():
    op = nsa.f8_empty(3, 200, "cuda")
    for t in op:
        t.view(torch.uint8).fill_(1)
    twin = tuple(torch._lazy_clone(t) for t in op)
    _lists().scan_f8([twin], F8_BLOCK, False)
    assert all(shares(a, b) for a, b in zip(op, twin))
    got = _lists().scan_f8([twin], F8_BLOCK, True)
    assert not any(shares(a, b) for a, b in zip(op, twin))
    assert [array("q", got[k])[0] for k in (5, 6)] == [t.data_ptr() for t in twin]


def test_both_of_two_written_tensors_get_their_own():
    x = torch.zeros(8)
    y = torch._lazy_clone(x)
    one, other = array("q", _lists().scan([x, y], True)[4])
    assert one != other


def state(n=4099, dtype=torch.float32):
    g = torch.Generator().manual_seed(3)
    return [torch.randn(n, generator=g).to(dtype).cuda() for _ in range(2)] + \
        [torch.randn(n, generator=g).square().cuda() for _ in range(2)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_adamw_leaves_the_others(dtype):
    p, g, m, v = state(dtype=dtype)
    want = [t.clone() for t in (p, m, v)]
    nsa.adamw_batched([want[0]], [g], [want[1]], [want[2]])
    kept = [t.clone() for t in (p, g, m, v)]
    twins = [torch._lazy_clone(t) for t in (p, g, m, v)]
    nsa.adamw_batched(*([t] for t in twins))
    assert shares(twins[1], g)  # the gradient is read only
    assert all(torch.equal(a, b) for a, b in zip((p, g, m, v), kept))
    assert all(torch.equal(a, b) for a, b in zip((twins[0], *twins[2:]), want))


@pytest.mark.gpu
def test_adamw_takes_moments_that_share_their_data():
    p, g, m, _ = state()
    m.zero_()
    want = [t.clone() for t in (p, m, m)]
    nsa.adamw_batched([want[0]], [g], [want[1]], [want[2]])
    v = torch._lazy_clone(m)
    nsa.adamw_batched([p], [g], [m], [v])
    assert all(torch.equal(a, b) for a, b in zip((p, m, v), want))


@pytest.mark.gpu
def test_scale_and_clip_in_place_leave_the_others():
    g = state()[0]
    kept = g.clone()
    half = torch.full((1,), 0.5, device="cuda")
    a = torch._lazy_clone(g)
    nsa.grad_scale_batched([a], half)
    assert torch.equal(g, kept) and torch.equal(a, kept * 0.5)
    b = torch._lazy_clone(g)
    r = nsa.grad_clip_batched([b], 1e-2)
    assert torch.equal(g, kept) and torch.equal(b, kept * r[1])
    c = torch._lazy_clone(g)
    nsa.grad_norm_batched([c])
    assert shares(c, g)


@pytest.mark.gpu
def test_outputs_that_share_data_with_their_gradients():
    g = state()[0]
    kept, twin = g.clone(), torch._lazy_clone(g)
    r = nsa.grad_clip_batched([g], 1e-2, out=[twin])
    assert torch.equal(g, kept) and torch.equal(twin, kept * r[1])
    # gradients and outputs in one storage that shares its data as a whole
    whole = torch.cat([kept[:4096], kept[:4096]])
    other = torch._lazy_clone(whole)
    before = whole.clone()
    r = nsa.grad_clip_batched([other[:4096]], 1e-2, out=[other[4096:]])
    assert torch.equal(whole, before)
    assert torch.equal(other[:4096], kept[:4096]) and torch.equal(other[4096:], kept[:4096] * r[1])


@pytest.mark.gpu
def test_product_and_quantization_leave_the_others():
    g = torch.Generator().manual_seed(5)
    x = torch.randn((70, 300), generator=g).cuda()
    a = nsa.f8_quantize_batched([x])
    (want,) = nsa.f8_matmul_batched(a, a, out_dtype=torch.float32)
    old = torch.ones((70, 70), device="cuda")
    for accumulate in (False, True):
        out = torch._lazy_clone(old)
        nsa.f8_matmul_batched(a, a, out=[out], accumulate=accumulate)
        assert bool((old == 1).all()) and not shares(out, old)
        assert torch.equal(out, want + 1 if accumulate else want)
    room = nsa.f8_empty(70, 300, "cuda")
    room_t = nsa.f8_empty(300, 70, "cuda")
    for t in (*room, *room_t):
        t.view(torch.uint8).fill_(0x55)
    twins = [tuple(torch._lazy_clone(t) for t in o) for o in (room, room_t)]
    nsa.f8_quantize_batched([x], transpose=True, out=[twins[0]], out_t=[twins[1]])
    assert all(bool((t.view(torch.uint8) == 0x55).all()) for t in (*room, *room_t))
    assert torch.equal(twins[0][0].view(torch.uint8), a[0].q.view(torch.uint8))
    assert torch.equal(twins[0][1], a[0].scales)
    # operands that are only read keep sharing
    twin = tuple(torch._lazy_clone(t) for t in a[0])
    nsa.f8_matmul_batched([twin], a)
    assert all(shares(p, q) for p, q in zip(twin, a[0]))


@pytest.mark.gpu
def test_norm_result_that_shares_its_data():
    g = state()[0]
    old = torch.full((2,), 3.0, device="cuda")
    r = torch._lazy_clone(old)
    nsa.grad_norm_batched([g], max_norm=1.0, norm_type=math.inf, result=r)
    assert bool((old == 3).all()) and float(r[0]) == float(g.abs().max())
