"""Tokens to the experts and back, against plain 64-bit forms.

The plan is whole numbers: equal.  Dispatched rows are copies: equal bits.  A row
of dys is one fp32 product, rounded once more for bf16: equal to that arithmetic
on the CPU.  combine adds top_k products in fp32, each fused multiply-add off by
half a step of a partial sum: top_k 2^-24 of the sum of magnitudes, then one
rounding of half a step of the type (bf16 2^-8, fp32 2^-24, of the value as summed).
dweights sums cols products in fp32 in some order: cols 2^-24 of the sum of
magnitudes.
"""
import numpy as np
import pytest
import torch

import expert_plain as plain
import newton_schulz_03_amd as nsa
from parity_util import host_f64
from test_captured_calls import replays

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, FP32: 2.0 ** -24}
U32 = 2.0 ** -24


@pytest.fixture(autouse=True)
def _announce(request):
    print(f"\n[gpu-test] {request.node.name}", flush=True)
    yield
    torch.cuda.synchronize()


def route(tokens, top_k, experts, drop, seed, dtype=torch.int32):
    """Ids with repeats in a token, some dropped by ids on both sides of the range."""
    rng = np.random.default_rng(seed)
    ids = (rng.random((tokens, top_k)) ** 2 * experts).astype(np.int64)
    lost = rng.random((tokens, top_k)) < drop
    wide = dtype == torch.int64
    out = rng.choice([-1, experts, -2 ** 31, 2 ** 31 - 1] + ([1 << 32, -(1 << 40)] if wide else []),
                     (tokens, top_k))
    return torch.from_numpy(np.where(lost, out, ids)).to(dtype).cuda()


def check_plan(got, ids, experts):
    want = plain.plan(ids.cpu().numpy(), experts)
    for name, g, w in zip(got._fields, got, want):
        assert g.dtype == torch.int32 and np.array_equal(g.cpu().numpy(), w), name


def values(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).cuda()


@pytest.mark.parametrize("tokens,top_k,experts", [
    (0, 2, 5), (1, 1, 1), (1, 8, 384), (2, 64, 3), (63, 1, 7), (64, 1, 8), (65, 1, 9), (16, 8, 700), (127, 1, 3), (128, 1, 1024), (4, 8, 384), (33, 1, 511), (16, 1, 512), (17, 1, 512), (10, 1, 1024),
    (11, 1, 1023), (128, 8, 60), (512, 8, 384), (513, 8, 384), (8192, 8, 100), (8193, 8, 100), (129, 1, 600), (129, 8, 384),
    (1000, 3, 1024), (1024, 8, 1023), (1025, 8, 33), (4096, 8, 384), (3001, 7, 2), (9000, 6, 511)])
@pytest.mark.parametrize("drop", [0.0, 0.3])
def test_sort(tokens, top_k, experts, drop):
    for dtype in (torch.int32, torch.int64):
        ids = route(tokens, top_k, experts, drop, tokens + experts, dtype)
        check_plan(nsa.moe_sort(ids, experts), ids, experts)


@pytest.mark.parametrize("tokens,top_k,experts", [(40000, 8, 384), (150001, 7, 100), (2500000, 1, 16)])
def test_sort_long(tokens, top_k, experts):
    ids = route(tokens, top_k, experts, 0.05, 1)
    check_plan(nsa.moe_sort(ids, experts), ids, experts)


@pytest.mark.parametrize("tokens", [5, 3000, 30000])
def test_sort_one_expert_or_none(tokens):
    for e in (0, 6, 7, -1):
        ids = torch.full((tokens, 4), e, dtype=torch.int32, device="cuda")
        check_plan(nsa.moe_sort(ids, 7), ids, 7)


def test_sort_into_a_plan():
    plan = nsa.moe_empty_plan(3000, 8, 50, "cuda")
    for seed in range(3):
        ids = route(3000, 8, 50, 0.2, seed)
        assert nsa.moe_sort(ids, 50, plan=plan) is plan
        check_plan(plan, ids, 50)
    with pytest.raises(ValueError):
        nsa.moe_sort(ids[:5].contiguous(), 50, plan=plan)
    with pytest.raises(ValueError):
        nsa.moe_sort(ids, 51, plan=plan)


COLS = [1, 2, 3, 4, 7, 8, 20, 100, 511, 512, 513, 1000, 1001, 2048, 6144, 8200, 9001]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("cols", COLS)
def test_dispatch(cols, dtype):
    for tokens, top_k, drop in ((1, 1, 0.0), (37, 3, 0.4), (130, 8, 0.1)):
        ids = route(tokens, top_k, 9, drop, cols)
        plan = nsa.moe_sort(ids, 9)
        x = values((tokens, cols), dtype, cols)
        x[0, 0] = float("nan")
        out = torch.full((tokens * top_k, cols), 7.0, dtype=dtype, device="cuda")
        want = out.clone()
        _, _, rows, _ = plain.plan(ids.cpu().numpy(), 9)
        t, k = np.nonzero(rows >= 0)
        want[torch.from_numpy(rows[t, k]).cuda()] = x[torch.from_numpy(t).cuda()]
        assert nsa.moe_dispatch(x, plan, out=out) is out
        raw = torch.int16 if dtype == BF16 else torch.int32
        assert torch.equal(out.view(raw), want.view(raw))
        n = int(plan.offsets[-1])
        assert torch.equal(nsa.moe_dispatch(x, plan)[:n].view(raw), want[:n].view(raw))
        # as many rows as are wanted: the others are skipped
        few = torch.full((n // 2 + 1, cols), 7.0, dtype=dtype, device="cuda")
        some = nsa.moe_dispatch(x, plan, out=few[:n // 2])
        assert torch.equal(some.view(raw), want[:n // 2].view(raw)) and bool((few[n // 2] == 7).all())


def want_combine(ys, rows, w):
    """(sum, sum of magnitudes) in float64; dropped slots and rows past ys add nothing."""
    y = host_f64(ys)
    on = (rows >= 0) & (rows < len(y))
    w = np.where(on, 1.0 if w is None else host_f64(w), 0.0)
    terms = np.zeros(rows.shape + (y.shape[1],))
    terms[on] = y[rows[on]]
    terms = terms * w[:, :, None]
    return terms.sum(1), np.abs(terms).sum(1)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("cols", COLS)
def test_combine_and_its_gradient(cols, dtype):
    for tokens, top_k, drop in ((1, 1, 0.0), (3, 2, 1.0), (37, 3, 0.4), (130, 8, 0.1), (5, 64, 0.2)):
        ids = route(tokens, top_k, 9, drop, cols)
        plan = nsa.moe_sort(ids, 9)
        rows = plain.plan(ids.cpu().numpy(), 9)[2]
        n = int((rows >= 0).sum())
        ys = values((tokens * top_k, cols), dtype, cols + 1)
        w = values((tokens, top_k), FP32, cols + 2)
        # what no kept slot names is never read into a result
        ys[n:] = float("nan")
        w[torch.from_numpy(rows < 0).cuda()] = float("nan")
        for weights in (w, None):
            got = nsa.moe_combine(ys, plan, weights=weights)
            want, mag = want_combine(ys, rows, weights)
            tol = top_k * U32 * mag
            assert got.dtype == dtype
            assert np.all(np.abs(host_f64(got) - want) <= tol + HALF[dtype] * (np.abs(want) + tol))
        dout = values((tokens, cols), dtype, cols + 3)
        dys = torch.full_like(ys, 7.0)
        dw = torch.full_like(w, 7.0)
        got = nsa.moe_combine_backward(dout, ys, plan, w, dys=dys, dweights=dw)
        assert got[0] is dys and got[1] is dw
        d, wc = dout.cpu().float(), w.cpu()
        t, k = np.nonzero(rows >= 0)
        want = torch.full(dys.shape, 7.0).to(dtype)
        want[torch.from_numpy(rows[t, k])] = (wc[t, k][:, None] * d[t]).to(dtype)
        assert torch.equal(dys.cpu(), want)
        terms = np.zeros((tokens, top_k, cols))
        terms[t, k] = host_f64(ys)[rows[t, k]] * host_f64(dout)[t]
        assert np.all(np.abs(host_f64(dw) - terms.sum(2)) <= cols * U32 * np.abs(terms).sum(2))
        new = nsa.moe_combine_backward(dout, ys, plan, w)
        assert torch.equal(new[0][:n], dys[:n]) and torch.equal(new[1], dw)


def test_fewer_sorted_rows():
    """Rows past the last of ys (as a program has them that split ys by the sizes)."""
    ids = route(50, 4, 6, 0.2, 3)
    plan = nsa.moe_sort(ids, 6)
    rows = plain.plan(ids.cpu().numpy(), 6)[2]
    n = int(plan.offsets[-1])
    assert sum(plan.sizes()) == n
    ys, w, dout = values((n, 72), FP32, 1), values((50, 4), FP32, 2), values((50, 72), FP32, 3)
    full = torch.cat([ys, torch.full((200 - n, 72), float("nan"), device="cuda")])
    assert torch.equal(nsa.moe_combine(ys, plan, weights=w), nsa.moe_combine(full, plan, weights=w))
    a, b = nsa.moe_combine_backward(dout, ys, plan, w), nsa.moe_combine_backward(dout, full, plan, w)
    assert torch.equal(a[0], b[0][:n]) and torch.equal(a[1], b[1])
    cut = n // 3
    got = nsa.moe_combine(ys[:cut], plan, weights=w)
    want, mag = want_combine(ys[:cut], rows, w)
    assert np.all(np.abs(host_f64(got) - want) <= 5 * U32 * mag + U32 * np.abs(want))
    dys, dw = nsa.moe_combine_backward(dout, ys[:cut], plan, w)
    assert torch.equal(dys, a[0][:cut])
    assert torch.equal(dw, torch.where(torch.from_numpy(rows < cut).cuda(), a[1], torch.zeros_like(dw)))


def test_infinities_and_nans():
    ids = torch.tensor([[0, 1], [1, 0], [1, -1]], dtype=torch.int32, device="cuda")
    plan = nsa.moe_sort(ids, 2)
    ys = torch.ones((6, 9), device="cuda")
    ys[plan.rows[0, 0], 2] = float("inf")
    ys[plan.rows[1, 1], 3] = float("nan")
    w = torch.ones((3, 2), device="cuda")
    out = nsa.moe_combine(ys, plan, weights=w).cpu()
    want = torch.tensor([2.0, 2.0, 1.0])[:, None].repeat(1, 9)
    want[0, 2] = float("inf")
    want[1, 3] = float("nan")
    assert torch.equal(out.nan_to_num(5.0), want.nan_to_num(5.0))


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_gradients_against_differences(dtype):
    """Small whole numbers, so that every sum is exact: the differences of <dout,
    combine> along each weight and row are the gradients, and dispatch and combine
    are adjoint."""
    rng = np.random.default_rng(5)
    ids = route(11, 3, 4, 0.2, 8)
    plan = nsa.moe_sort(ids, 4)

    def whole(shape, most, dt=dtype):
        return torch.from_numpy(rng.integers(-most, most + 1, shape)).to(dt).cuda()

    ys, w, dout = whole((33, 6), 3), whole((11, 3), 2, FP32), whole((11, 6), 2)

    def loss(ys, w):
        return float((host_f64(nsa.moe_combine(ys, plan, weights=w)) * host_f64(dout)).sum())

    n = int(plan.offsets[-1])
    dys, dw = nsa.moe_combine_backward(dout, ys, plan, w)
    base = loss(ys, w)
    for t in range(11):
        for k in range(3):
            w2 = w.clone()
            w2[t, k] += 1
            assert loss(ys, w2) - base == float(dw[t, k])
    for p in range(0, n, 4):
        for c in (0, 5):
            y2 = ys.clone()
            y2[p, c] += 1
            assert loss(y2, w) - base == float(dys[p, c])
    x, z = whole((11, 6), 3), whole((33, 6), 3)
    xs = host_f64(nsa.moe_dispatch(x, plan))[:n]
    assert (xs * host_f64(z)[:n]).sum() == (host_f64(nsa.moe_combine(z, plan)) * host_f64(x)).sum()


def test_equal_calls_give_equal_bits():
    ids = route(3000, 8, 60, 0.1, 2)
    plan = nsa.moe_sort(ids, 60)
    ys, w, dout = values((24000, 520), BF16, 1), values((3000, 8), FP32, 2), values((3000, 520), BF16, 3)
    n = int(plan.offsets[-1])
    one = nsa.moe_combine(ys, plan, weights=w), *nsa.moe_combine_backward(dout, ys, plan, w)
    for _ in range(3):
        two = nsa.moe_combine(ys, plan, weights=w), *nsa.moe_combine_backward(dout, ys, plan, w)
        assert torch.equal(one[0], two[0]) and torch.equal(one[1][:n], two[1][:n]) and torch.equal(one[2], two[2])


def test_rows_past_32_bits():
    """Sorted rows whose bytes lie past 2^32: 2.5 M rows of 1000 bf16."""
    tokens, cols = 2_500_000, 1000
    ids = torch.zeros((tokens, 1), dtype=torch.int32, device="cuda")
    ids[1::2] = 1
    plan = nsa.moe_sort(ids, 2)
    x = torch.arange(tokens, device="cuda").remainder_(251).to(BF16)[:, None].expand(tokens, cols).contiguous()
    xs = nsa.moe_dispatch(x, plan)
    for p in (0, tokens // 2 - 1, tokens // 2, 2_147_484, 2_147_485, tokens - 1):
        t = int(plan.slots[p])
        assert t == (2 * p if p < tokens // 2 else 2 * (p - tokens // 2) + 1)
        assert torch.equal(xs[p], x[t])
    assert torch.equal(nsa.moe_combine(xs, plan), x)
    w = torch.full((tokens, 1), 2.0, device="cuda")
    dys, dw = nsa.moe_combine_backward(x, xs, plan, w)
    assert torch.equal(dys[-1], 2 * x[-1]) and torch.equal(dys[2_147_485], 2 * xs[2_147_485])
    # 1000 squares of a whole number below 251: exact
    assert torch.equal(dw[:, 0], 1000 * x[:, 0].float() ** 2)


@pytest.mark.parametrize("tokens", [40, 5000])
def test_captured(tokens):
    ids = route(tokens, 8, 40, 0.1, 4)
    x, w = values((tokens, 264), BF16, 1), values((tokens, 8), FP32, 2)

    def step():
        plan = nsa.moe_sort(ids, 40)
        xs = nsa.moe_dispatch(x, plan, out=torch.zeros((tokens * 8, 264), dtype=BF16, device="cuda"))
        y = nsa.moe_combine(xs, plan, weights=w)
        dys = torch.zeros_like(xs)
        return [*plan, xs, y, *nsa.moe_combine_backward(x, xs, plan, w, dys=dys)]

    got, want = [], []

    def change(k):
        ids.add_(1).remainder_(45)
        x.mul_(-1.25)
        w.add_(0.125)

    def run():
        got[:] = step()

    def eager():
        want[:] = step()

    replays(run, eager, lambda: zip(got, want), change)


def test_on_another_stream():
    ids = route(2000, 8, 40, 0.1, 4)
    x, w = values((2000, 264), BF16, 1), values((2000, 8), FP32, 2)
    plan = nsa.moe_sort(ids, 40)
    want = nsa.moe_combine(nsa.moe_dispatch(x, plan), plan, weights=w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        late = torch.empty_like(x)
        for _ in range(50):
            late.copy_(x)
        p2 = nsa.moe_sort(ids, 40)
        got = nsa.moe_combine(nsa.moe_dispatch(late, p2), p2, weights=w)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(plan, p2)) and torch.equal(got, want)


def test_a_given_workspace():
    ids = route(5000, 8, 40, 0.1, 4)
    nbytes = nsa.moe_workspace_bytes(5000, 8, 40)
    room = torch.full((nbytes + 512,), 0xEE, dtype=torch.uint8, device="cuda")
    at = (-room.data_ptr()) % 256
    check_plan(nsa.moe_sort(ids, 40, workspace=room[at:at + nbytes]), ids, 40)
    assert bool((room[at + nbytes:] == 0xEE).all()) and bool((room[:at] == 0xEE).all())
    for bad in (room[at:at + nbytes - 1], room[at + 1:]):
        with pytest.raises(nsa.MuonError):
            nsa.moe_sort(ids, 40, workspace=bad)
    for bad in (torch.empty(nbytes, dtype=torch.uint8), room[::2], room.view(torch.int32)):
        with pytest.raises(ValueError):
            nsa.moe_sort(ids, 40, workspace=bad)


def test_calls_on_two_streams_at_once():
    work = []
    for seed in (1, 2):
        ids = route(6000, 8, 64, 0.1, seed)
        x, w = values((6000, 520), BF16, seed), values((6000, 8), FP32, seed)
        plan = nsa.moe_sort(ids, 64)
        work.append((ids, x, w, plan, nsa.moe_combine(nsa.moe_dispatch(x, plan), plan, weights=w)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    got = [[], []]
    for _ in range(10):
        for s, (ids, x, w, _, _), g in zip(streams, work, got):
            with torch.cuda.stream(s):
                plan = nsa.moe_sort(ids, 64)
                g.append((plan, nsa.moe_combine(nsa.moe_dispatch(x, plan), plan, weights=w)))
    torch.cuda.synchronize()
    for (_, _, _, plan, out), g in zip(work, got):
        for p, o in g:
            assert all(torch.equal(a, b) for a, b in zip(p, plan)) and torch.equal(o, out)


def test_binding_refusals():
    ids = route(10, 2, 4, 0.0, 1)
    plan = nsa.moe_sort(ids, 4)
    x, ys = values((10, 16), BF16, 1), values((20, 16), BF16, 2)
    w = torch.ones((10, 2), device="cuda")
    for call in (lambda: nsa.moe_sort(ids.float(), 4), lambda: nsa.moe_dispatch(x.half(), plan),
                 lambda: nsa.moe_combine(ys, plan, weights=w.bfloat16()),
                 lambda: nsa.moe_combine_backward(x, ys.float(), plan, w)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: nsa.moe_sort(ids.t(), 4), lambda: nsa.moe_sort(ids[0], 4),
                 lambda: nsa.moe_dispatch(x[:9], plan), lambda: nsa.moe_dispatch(x[:, ::2], plan),
                 lambda: nsa.moe_dispatch(x, plan, out=ys[:, :8].contiguous()),
                 lambda: nsa.moe_combine(ys, plan, weights=w[:9]),
                 lambda: nsa.moe_combine(ys, plan, weights=w.cpu()),
                 lambda: nsa.moe_combine(ys, plan, out=ys[:9]),
                 lambda: nsa.moe_combine_backward(x, ys, plan, w, dys=ys[:19]),
                 lambda: nsa.moe_combine_backward(x, ys[:, :8].contiguous(), plan, w)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: nsa.moe_sort(ids, 0), lambda: nsa.moe_sort(ids, 1025),
                 lambda: nsa.moe_combine_backward(x, ys, plan, w, dys=ys)):
        with pytest.raises(nsa.MuonError):
            call()


def test_shared_tensors_are_left():
    """Written tensors that share their data copy-on-write get memory of their own."""
    ids = route(10, 2, 4, 0.0, 1)
    plan = nsa.moe_sort(ids, 4)
    x = values((10, 16), BF16, 1)
    for make in (lambda o: nsa.moe_dispatch(x, plan, out=o), lambda o: nsa.moe_combine(nsa.moe_dispatch(x, plan), plan, out=o)):
        base = torch.zeros((20 if make(None).shape[0] == 20 else 10, 16), dtype=BF16, device="cuda")
        twin = torch._lazy_clone(base)
        make(twin)
        assert not bool(base.any()) and bool(twin.any())
