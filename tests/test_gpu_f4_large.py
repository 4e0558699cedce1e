"""4-bit products of many strips of 16 weight rows: the kernels of two and four strips a
wave, with one or more shares of the columns, and the one of many rows with two strips
a wave, whose sizes the other tests do not reach.  Every output, against 64 bits on the
device; the bound is that of test_gpu_f4.py: K additions off by at most 2^-23 of the
sum of magnitudes, then one rounding."""
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


def operand(count, rows, cols, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return nsa.f4_quantize([torch.randn((rows, cols), generator=gen, device="cuda").mul_(0.02).bfloat16()
                            for _ in range(count)])


def weights(op, i):
    """The float64 values of matrix i, on the device: byte 4 a + b of chunk 16 c + r of a
    tile holds columns 32 a + 8 c + 2 b and the next one of row r."""
    q, s = op.q[i], op.scales[i]
    rt, kt = q.shape[:2]
    b = q.view(rt, kt, 4, 16, 4, 4)
    codes = torch.stack([b & 15, b >> 4], dim=-1).permute(0, 3, 1, 4, 2, 5, 6).reshape(16 * rt, 128 * kt).long()
    table = torch.tensor(np.concatenate([plain.E2M1, -plain.E2M1]), device="cuda")
    scale = torch.exp2(s.permute(0, 2, 1, 3).reshape(16 * rt, -1).double() - 127)[:, :4 * kt]
    return (table[codes].view(16 * rt, -1, 32) * scale[:, :, None]).view(16 * rt, -1)[:op.rows, :op.cols].contiguous()


def check(y, x, w):
    x = x.double()
    want, mag = x @ w.t(), x.abs() @ w.abs().t()
    tol = x.shape[1] * 2.0 ** -23 * mag
    assert bool(((y.double() - want).abs() <= tol + HALF[y.dtype] * (want.abs() + tol)).all())


def route(tokens, top_k, experts, uneven, seed):
    """Ids of which some experts get many, the last none, and a few slots are dropped."""
    rng = np.random.default_rng(seed)
    ids = (rng.random((tokens, top_k)) ** uneven * (experts - 1)).astype(np.int32)
    ids[rng.random((tokens, top_k)) < 0.05] = -1
    return torch.from_numpy(ids).cuda()


def test_the_plain_weights():
    w = torch.randn((40, 700)).mul_(3).bfloat16()
    op = nsa.f4_quantize([w.cuda()])
    assert np.array_equal(weights(op, 0).cpu().numpy(), plain.f4_values(*plain.f4(host_f64(w)), 700))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("rows,cols", [(6150, 4097), (4100, 6144)])
def test_one_matrix(rows, cols, dtype):
    """Two strips a wave, eight shares of the columns."""
    op = operand(1, rows, cols, rows)
    w = weights(op, 0)
    for m in (1, 5, 16):
        x = torch.randn((m, cols), device="cuda").bfloat16()
        room = torch.full((m + 1, rows), 7.0, dtype=dtype, device="cuda")
        y = nsa.f4_matmul(x, op, out=room[:m])
        check(y, x, w)
        assert bool((room[m] == 7).all())
        assert torch.equal(nsa.f4_matmul(x, op, out_dtype=dtype), y)


# strips a wave x shares of the columns: experts, rows, columns, tokens, top_k, uneven
EXPERTS = {
    "2 x 1": (40, 850, 500, 60, 4, 2),
    "2 x 2": (20, 900, 1000, 37, 5, 2),
    "4 x 1": (40, 3333, 1001, 80, 4, 3),
    "4 x 2": (33, 2000, 1550, 70, 4, 2),
    "4 x 4": (21, 1600, 3600, 50, 3, 2),
    "many, 2 x 1": (24, 1000, 515, 120, 4, 1.3),
    "many, 2 x 1, whole tiles": (24, 1000, 1024, 120, 4, 1.3),
    "many, a block a CU": (16, 1024, 640, 80, 4, 1.3),
    "many, and one more": (17, 1021, 640, 85, 4, 1.3),
    "many, 2 x 1, passes": (3, 1000, 700, 600, 3, 1.5),
}


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("name", list(EXPERTS))
def test_experts(name, dtype):
    experts, rows, cols, tokens, top_k, uneven = EXPERTS[name]
    op = operand(experts, rows, cols, rows)
    ids = route(tokens, top_k, experts, uneven, 1)
    plan = nsa.moe_sort(ids, experts)
    sizes = plan.sizes()
    n = sum(sizes)
    assert sizes[-1] == 0 and max(sizes) > 16 and n < tokens * top_k
    x = torch.randn((tokens, cols), device="cuda").bfloat16()
    xs = nsa.moe_dispatch(x, plan)
    xs[n:] = float("nan")
    y = torch.full((tokens * top_k, rows), 7.0, dtype=dtype, device="cuda")
    y2 = y.clone()
    nsa.f4_matmul(xs, op, plan=plan, out=y)
    nsa.f4_matmul(x, op, plan=plan, gather=True, out=y2)
    assert torch.equal(y, y2) and bool((y[n:] == 7).all())
    at = 0
    for e, size in enumerate(sizes):
        if size:
            check(y[at:at + size], xs[at:at + size], weights(op, e))
        at += size


@pytest.mark.parametrize("name", ["2 x 2", "4 x 2", "many, 2 x 1, passes"])
def test_captured(name):
    experts, rows, cols, tokens, top_k, uneven = EXPERTS[name]
    op = operand(experts, rows, cols, rows)
    ids = route(tokens, top_k, experts, uneven, 2)
    x = torch.randn((tokens, cols), device="cuda").bfloat16()
    got, want = (torch.zeros((tokens * top_k, rows), device="cuda") for _ in range(2))

    def step(out):
        out.zero_()
        nsa.f4_matmul(x, op, plan=nsa.moe_sort(ids, experts), gather=True, out=out)

    def change(k):
        ids.add_(1).remainder_(experts + 1)
        x.mul_(-1.25)

    replays(lambda: step(got), lambda: step(want), lambda: [(got, want)], change)
