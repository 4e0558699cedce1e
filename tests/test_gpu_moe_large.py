"""Dispatch, combine and its gradient where the sorted rows hold just over 256 MB, from
where rows of whole 16-byte pieces, and others of 2000 bytes and more, are read and
written with the nontemporal hint: a block, a wave or 16 lanes a token, both kinds of
length.  Copies and rows of the gradient bit for bit, sums with the bounds of
test_gpu_moe.py, all on the device."""
import pytest
import torch

import newton_schulz_03_amd as nsa

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, FP32: 2.0 ** -24}
U32 = 2.0 ** -24


@pytest.fixture(autouse=True)
def _announce(request):
    print(f"\n[gpu-test] {request.node.name}", flush=True)
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("cols,dtype,top_k", [
    (6144, BF16, 8), (2501, BF16, 8), (2501, FP32, 3), (1536, FP32, 8),     # a block a token
    (1001, FP32, 8), (501, BF16, 3), (1000, BF16, 8),                       # a wave
    (100, BF16, 8), (96, BF16, 8), (63, FP32, 9), (64, FP32, 2)])           # 16 lanes
def test_past_the_caches(cols, dtype, top_k):
    row = cols * dtype.itemsize
    tokens = (256 << 20) // (row * top_k) + 2
    assert tokens >= 2000 and tokens * top_k * row > 256 << 20
    gen = torch.Generator(device="cuda").manual_seed(cols)

    def normal(*shape, dt=dtype):
        return torch.randn(shape, generator=gen, device="cuda").to(dt)

    ids = torch.randint(-1, 40, (tokens, top_k), generator=gen, device="cuda", dtype=torch.int32)
    plan = nsa.moe_sort(ids, 40)
    n = int(plan.offsets[-1])
    assert torch.equal(plan.rows < 0, ids < 0) and 0 < n < tokens * top_k
    slots = plan.slots[:n].long()
    raw = torch.int16 if dtype == BF16 else torch.int32

    x = normal(tokens, cols)
    xs = torch.full((tokens * top_k, cols), 7.0, dtype=dtype, device="cuda")
    nsa.moe_dispatch(x, plan, out=xs)
    assert torch.equal(xs[:n].view(raw), x[slots // top_k].view(raw)) and bool((xs[n:] == 7).all())
    del xs

    ys, w = normal(tokens * top_k, cols), normal(tokens, top_k, dt=FP32)
    ys[n:] = float("nan")
    w[ids < 0] = float("nan")
    for weights in (w, None):
        got = nsa.moe_combine(ys, plan, weights=weights)
        for a in range(0, tokens, 4096):
            rows = plan.rows[a:a + 4096]
            on = (rows >= 0)[:, :, None]
            y = ys[rows.clamp(min=0).long()].double().masked_fill_(~on, 0.0)
            if weights is not None:
                y *= w[a:a + 4096, :, None].double().masked_fill(~on, 0.0)
            want, tol = y.sum(1), top_k * U32 * y.abs().sum(1)
            off = (got[a:a + 4096].double() - want).abs()
            assert bool((off <= tol + HALF[dtype] * (want.abs() + tol)).all())

    dout = normal(tokens, cols)
    dys = torch.full_like(ys, 7.0)
    dw = torch.full_like(w, 7.0)
    nsa.moe_combine_backward(dout, ys, plan, w, dys=dys, dweights=dw)
    assert bool((dys[n:] == 7).all())
    for a in range(0, n, 1 << 17):
        s = slots[a:a + (1 << 17)]
        part = (w.flatten()[s][:, None] * dout[s // top_k].float()).to(dtype)
        assert torch.equal(dys[a:a + (1 << 17)][:len(s)], part)
    for a in range(0, tokens, 4096):
        rows = plan.rows[a:a + 4096]
        on = rows >= 0
        terms = ys[rows.clamp(min=0).long()].double() * dout[a:a + 4096, None].double()
        terms.masked_fill_(~on[:, :, None], 0.0)
        off = (dw[a:a + 4096].double() - terms.sum(2)).abs()
        assert bool((off <= cols * U32 * terms.abs().sum(2)).all())
