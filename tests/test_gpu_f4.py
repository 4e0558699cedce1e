"""4-bit weights with group scales and their products, against 64-bit forms.

Quantization is exact arithmetic up to the one rounding to a code: operands are
compared byte by byte with a numpy implementation in float64.

Products: a weight's value and a bf16 element have an exact product in fp32; the
sum of K of them is formed in fp32, each of at most K additions off by at most one
unit in the last place of a partial sum, 2^-23 of the sum of magnitudes (whether
it rounds or cuts off); then one rounding of half a step of the type (bf16 2^-8,
fp32 2^-24, of the value as summed).
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


@pytest.fixture(autouse=True)
def _announce(request):
    print(f"\n[gpu-test] {request.node.name}", flush=True)
    yield
    torch.cuda.synchronize()


def values(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).cuda()


def check_operand(op, ws):
    for i, w in enumerate(ws):
        q, s = plain.f4_layout(*plain.f4(host_f64(w)))
        assert np.array_equal(op.scales[i].cpu().numpy(), s)
        assert np.array_equal(op.q[i].cpu().numpy(), q)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (16, 31), (15, 32), (17, 33), (40, 127), (33, 129),
                                       (16, 512), (64, 513), (100, 700), (7, 1030), (256, 2048), (130, 6144)])
def test_quantize(rows, cols, dtype):
    ws = [values((rows, cols), dtype, i, 0.02 * 3.0 ** i) for i in range(3)]
    op = nsa.f4_quantize(ws)
    assert (op.rows, op.cols) == (rows, cols)
    check_operand(op, ws)
    kept = nsa.f4_empty(3, cols, rows, "cuda")
    for t in (kept.q, kept.scales):
        t.fill_(0xEE)
    assert nsa.f4_quantize(ws, transpose=True, out=kept) is kept
    check_operand(kept, [w.t() for w in ws])


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_quantize_ends_of_the_range(dtype):
    """Ties, zeros of both signs, subnormal numbers, the largest ones, infinities and
    NaN, a kind to a group."""
    rng = np.random.default_rng(2)
    w = torch.zeros((18, 256))
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    for r in range(16):
        for g, scale in enumerate((1.0, 2.0 ** -120, 2.0 ** 120, 2.0 ** -127, 2.0 ** 125)):
            v = torch.cat([ties, -ties, torch.from_numpy(rng.uniform(-6, 6, 16)).float()])
            w[r, 32 * g:32 * g + 32] = v[torch.from_numpy(rng.permutation(32))] * scale
    w[0, 160:192] = 2.0 ** -149 if dtype == FP32 else 2.0 ** -133
    w[1, 160:192] = torch.finfo(dtype).max
    w[2, 165] = float("inf")
    w[3, 170] = float("nan")
    w[4, 191] = -float("inf")
    w[5, 192:224] = -0.0
    w[6, 192] = -1e-3
    w = w.to(dtype).cuda()
    check_operand(nsa.f4_quantize([w]), [w])
    check_operand(nsa.f4_quantize([w.t().contiguous()], transpose=True), [w])


@pytest.mark.parametrize("count", [1, 479, 480, 481, 600, 1024])
def test_quantize_many(count):
    # pointers of up to 480 matrices travel as kernel arguments
    whole = values((count, 5, 40), BF16, count)
    op = nsa.f4_quantize(list(whole))
    for i in {0, count // 3, count // 2, count - 1}:
        q, s = plain.f4_layout(*plain.f4(host_f64(whole[i])))
        assert np.array_equal(op.q[i].cpu().numpy(), q) and np.array_equal(op.scales[i].cpu().numpy(), s)


def operand(count, rows, cols, seed, std=0.02):
    """An operand and the float64 values of its matrices."""
    ws = [values((rows, cols), BF16, seed + i, std) for i in range(count)]
    op = nsa.f4_quantize(ws)
    return op, [plain.f4_values(*plain.f4(host_f64(w)), cols) for w in ws]


def check(y, x, w, dtype):
    """y (rows x R) = x w^T for float64 x and w."""
    got, want, mag = host_f64(y), x @ w.T, np.abs(x) @ np.abs(w).T
    tol = x.shape[1] * 2.0 ** -23 * mag
    assert np.all(np.abs(got - want) <= tol + HALF[dtype] * (np.abs(want) + tol))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (5, 7), (16, 8), (17, 31), (31, 32), (64, 100), (48, 127), (130, 128),
                                       (33, 129), (40, 500), (16, 512), (96, 520), (257, 1000), (300, 1024),
                                       (2048, 2048), (256, 6144), (100, 8193), (64, 896), (40, 1408), (33, 2560)])
def test_one_matrix(rows, cols, dtype):
    op, (w,) = operand(1, rows, cols, rows + cols)
    for m in (1, 2, 3, 4, 5, 8, 15, 16, 17, 31, 33, 48, 64, 65, 130):
        x = values((m, cols), BF16, m)
        room = torch.full((m + 1, rows), 7.0, dtype=dtype, device="cuda")
        y = nsa.f4_matmul(x, op, out=room[:m])
        check(y, host_f64(x), w, dtype)
        assert bool((room[m] == 7).all())
        assert torch.equal(nsa.f4_matmul(x, op, out_dtype=dtype), y)


def route(tokens, top_k, experts, drop, seed):
    rng = np.random.default_rng(seed)
    ids = (rng.random((tokens, top_k)) ** 2 * experts).astype(np.int32)
    ids[rng.random((tokens, top_k)) < drop] = -1
    return torch.from_numpy(ids).cuda()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("tokens,top_k,experts", [(1, 1, 1), (1, 8, 24), (3, 4, 9), (40, 2, 5), (200, 3, 4), (70, 6, 24),
                                                  (20, 2, 70)])
@pytest.mark.parametrize("rows,cols", [(48, 200), (70, 515), (256, 1024)])
def test_experts(tokens, top_k, experts, rows, cols, dtype):
    op, ws = operand(experts, rows, cols, experts)
    for drop in (0.0, 0.3, 1.0):
        ids = route(tokens, top_k, experts, drop, tokens)
        plan = nsa.moe_sort(ids, experts)
        offsets, _, _, slots = plain.plan(ids.cpu().numpy(), experts)
        x = values((tokens, cols), BF16, tokens + 1)
        xs = nsa.moe_dispatch(x, plan)
        n = offsets[-1]
        xs[n:] = float("nan")
        y = torch.full((tokens * top_k, rows), 7.0, dtype=dtype, device="cuda")
        y2 = y.clone()
        assert nsa.f4_matmul(xs, op, plan=plan, out=y) is y
        nsa.f4_matmul(x, op, plan=plan, gather=True, out=y2)
        assert torch.equal(y, y2) and bool((y[n:] == 7).all())
        def check_rows(y, n):
            for e in range(experts):
                a, b = offsets[e], min(offsets[e + 1], n)
                if a < b:
                    check(y[a:b], host_f64(x)[slots[a:b] // top_k], ws[e], dtype)

        check_rows(y, n)
        # fewer rows: those of xs, and of a smaller out (the order of the sums may be another)
        if n > 1:
            check_rows(nsa.f4_matmul(xs[:n - 1].contiguous(), op, plan=plan, out_dtype=dtype), n - 1)
            few = torch.full((n, rows), 7.0, dtype=dtype, device="cuda")
            nsa.f4_matmul(x, op, plan=plan, gather=True, out=few[:n - 1])
            check_rows(few, n - 1)
            assert bool((few[n - 1] == 7).all())


def test_every_code_scale_and_place():
    """One column of x at a time: the product is the weight itself, exact in fp32."""
    rng = np.random.default_rng(1)
    rows, cols = 40, 640
    codes = rng.integers(0, 16, (rows, cols))
    scales = rng.integers(2, 253, (rows, cols // 32))
    q, s = plain.f4_layout(codes, scales)
    op = nsa.F4Operand(torch.from_numpy(q)[None].cuda(), torch.from_numpy(s)[None].cuda(), rows, cols)
    x = torch.eye(cols, dtype=BF16, device="cuda")
    y = host_f64(nsa.f4_matmul(x, op, out_dtype=FP32))
    assert np.array_equal(y.T, plain.f4_values(codes, scales, cols))


def test_nan_groups_and_rows():
    op, (w,) = operand(1, 33, 300, 4)
    x = values((5, 300), BF16, 1)
    base = nsa.f4_matmul(x, op, out_dtype=FP32)
    # a NaN or an infinity in a row of x is that row's alone
    bad = x.clone()
    bad[2, 7] = float("nan")
    bad[4, 299] = float("inf")
    y = nsa.f4_matmul(bad, op, out_dtype=FP32)
    assert torch.equal(y[[0, 1, 3]], base[[0, 1, 3]]) and bool(y[2].isnan().all())
    assert not bool(torch.isfinite(y[4]).any())
    # a NaN group is its weight row's alone
    m = values((33, 300), BF16, 4, 0.02)
    m[9, 290] = float("inf")
    y = nsa.f4_matmul(x, nsa.f4_quantize([m]), out_dtype=FP32)
    assert bool(y[:, 9].isnan().all())
    y[:, 9] = base[:, 9]
    assert torch.equal(y, base)
    # also where x is zero there
    x[:, 288:300] = 0
    assert bool(nsa.f4_matmul(x, nsa.f4_quantize([m]), out_dtype=FP32)[:, 9].isnan().all())


def test_nothing_to_sum():
    op = nsa.f4_quantize([torch.zeros((20, 0), dtype=BF16, device="cuda")])
    x = torch.zeros((3, 0), dtype=BF16, device="cuda")
    y = torch.full((3, 20), 7.0, device="cuda")
    assert not bool(nsa.f4_matmul(x, op, out=y).any())
    op, _ = operand(1, 20, 40, 1)
    assert nsa.f4_matmul(torch.zeros((0, 40), dtype=BF16, device="cuda"), op).shape == (0, 20)
    assert nsa.f4_matmul(x.new_zeros((3, 40)), nsa.f4_empty(1, 0, 40, "cuda")).shape == (3, 0)


def test_a_plan_without_tokens():
    op, _ = operand(3, 20, 40, 1)
    plan = nsa.moe_sort(torch.zeros((0, 2), dtype=torch.int64, device="cuda"), 3)
    x = torch.zeros((0, 40), dtype=BF16, device="cuda")
    assert nsa.f4_matmul(x, op, plan=plan, gather=True).shape == (0, 20)
    assert nsa.f4_matmul(x, op, plan=plan).shape == (0, 20)


def test_more_rows_than_the_products_are_for():
    # passes of 64 rows: over the grid, and again within a block
    op, (w,) = operand(1, 40, 136, 3)
    x = values((1111, 136), BF16, 1)
    check(nsa.f4_matmul(x, op, out_dtype=FP32), host_f64(x), w, FP32)
    op, ws = operand(9, 40, 136, 3)
    ids = torch.zeros((1500, 1), dtype=torch.int32, device="cuda")
    ids[:8, 0] = torch.arange(1, 9, device="cuda")
    plan = nsa.moe_sort(ids, 9)
    x = values((1500, 136), BF16, 2)
    y = nsa.f4_matmul(x, op, plan=plan, gather=True, out_dtype=FP32)
    check(y[:1492], host_f64(x)[8:], ws[0], FP32)
    for e in range(1, 9):
        check(y[1491 + e:1492 + e], host_f64(x)[e - 1:e], ws[e], FP32)


def test_weights_past_4_gb():
    """The last expert's matrix lies past 2^32 bytes of codes."""
    experts, rows, cols = 700, 2048, 6144
    op = nsa.f4_empty(experts, rows, cols, "cuda")
    op.q.zero_()
    op.scales.fill_(127)
    w = values((rows, cols), BF16, 1)
    one = nsa.f4_quantize([w])
    op.q[-1], op.scales[-1] = one.q[0], one.scales[0]
    ids = torch.tensor([[experts - 1, 0]], dtype=torch.int32, device="cuda")
    x = values((1, cols), BF16, 2)
    y = nsa.f4_matmul(x, op, plan=nsa.moe_sort(ids, experts), gather=True, out_dtype=FP32)
    assert not bool(y[0].any())
    check(y[1:], host_f64(x), plain.f4_values(*plain.f4(host_f64(w)), cols), FP32)


def test_equal_calls_give_equal_bits():
    op, _ = operand(5, 300, 2048, 1)
    plan = nsa.moe_sort(route(60, 2, 5, 0.1, 1), 5)
    x = values((60, 2048), BF16, 1)
    y = nsa.f4_matmul(x, op, plan=plan, gather=True, out_dtype=FP32)
    n = int(plan.offsets[-1])
    for _ in range(3):
        assert torch.equal(nsa.f4_matmul(x, op, plan=plan, gather=True, out_dtype=FP32)[:n], y[:n])


def test_a_decode_step_captured():
    """Sort, two gathered products, one more and the combine, replayed on other
    tokens and ids: nothing of the plan is read on the host."""
    experts, hidden, ffn = 12, 200, 136
    up, down = operand(experts, ffn, hidden, 1)[0], operand(experts, hidden, ffn, 90)[0]
    ids = route(9, 3, experts, 0.1, 2)
    x, w = values((9, hidden), BF16, 3), values((9, 3), FP32, 4)
    got, want = [], []

    def step():
        plan = nsa.moe_sort(ids, experts)
        h = torch.zeros((27, ffn), dtype=BF16, device="cuda")
        nsa.f4_matmul(x, up, plan=plan, gather=True, out=h)
        y = nsa.f4_matmul(torch.relu(h), down, plan=plan)
        return [nsa.moe_combine(y, plan, weights=w)]

    def run():
        got[:] = step()

    def eager():
        want[:] = step()

    def change(k):
        ids.add_(1).remainder_(experts + 2)
        x.mul_(-1.25)

    replays(run, eager, lambda: zip(got, want), change)


def test_on_another_stream():
    op, (w,) = operand(1, 300, 2048, 1)
    x = values((3, 2048), BF16, 1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        late = torch.empty_like(x)
        for _ in range(200):
            late.copy_(x)
        y = nsa.f4_matmul(late, op, out_dtype=FP32)
    s.synchronize()
    check(y, host_f64(x), w, FP32)


def test_binding_refusals():
    op, _ = operand(2, 20, 40, 1)
    one, _ = operand(1, 20, 40, 1)
    plan = nsa.moe_sort(route(3, 2, 2, 0.0, 1), 2)
    x = values((3, 40), BF16, 1)
    for call in (lambda: nsa.f4_matmul(x, op), lambda: nsa.f4_matmul(x, one, gather=True),
                 lambda: nsa.f4_matmul(x, one, plan=plan), lambda: nsa.f4_matmul(x[:, :39].contiguous(), one),
                 lambda: nsa.f4_matmul(x[:2], op, plan=plan, gather=True),
                 lambda: nsa.f4_matmul(values((7, 40), BF16, 1), op, plan=plan),
                 lambda: nsa.f4_matmul(x, one, out=torch.zeros((2, 20), device="cuda")),
                 lambda: nsa.f4_matmul(x, one, out=torch.zeros((3, 21), device="cuda")),
                 lambda: nsa.f4_matmul(x, one, out=torch.zeros((3, 20), device="cuda"), out_dtype=BF16),
                 lambda: nsa.f4_matmul(x, one._replace(q=one.q[:, :1])),
                 lambda: nsa.f4_matmul(x, one._replace(scales=one.scales.cpu())),
                 lambda: nsa.f4_quantize([x], out=op), lambda: nsa.f4_quantize([x[0]]),
                 lambda: nsa.f4_quantize([x[:, ::2]])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: nsa.f4_matmul(x.float(), one), lambda: nsa.f4_quantize([x.half()]),
                 lambda: nsa.f4_matmul(x, one, out_dtype=torch.float16)):
        with pytest.raises(TypeError):
            call()
