"""The global gradient norm, the clip factor, scaled gradients and the steps that
take the factor, against 64-bit arithmetic.

Bounds.  The norm is formed in double and rounded once: relative error at most
2^-24 for the rounding, plus N 2^-53 for the sum of N squares.  The factor is
one double division of the unrounded norm, rounded once: the same.  A scaled
gradient is the fp32 product, rounded once more for a bf16 output: bit-equal to
that arithmetic on the CPU with the factor the call returned.
"""
import math

import numpy as np
import pytest
import torch

import newton_schulz_03_amd as nsa
import oracle
from parity_util import host_f64

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
SPAN = 16384  # elements of a chunk
NUMELS = [1, 7, 8, 9, 255, 8191, 8192, 8193, 100003, 0, 3 * 8192 + 5, SPAN, SPAN + 1, 4 * SPAN - 1]
U32 = 2.0 ** -24


@pytest.fixture(autouse=True)
def _announce(request):
    print(f"\n[gpu-test] {request.node.name}", flush=True)
    yield
    torch.cuda.synchronize()


def f32(x):
    return float(np.float32(x))


def make(numels, dtypes, seed, std=1e-3):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * std).to(dt).cuda() for n, dt in zip(numels, dtypes)]


def mixed(n):
    return [BF16 if i % 3 else FP32 for i in range(n)]


def want_norm(ts, kind):
    xs = [host_f64(t).ravel() for t in ts]
    if kind == math.inf:
        return max((float(np.max(np.abs(x))) for x in xs if x.size), default=0.0)
    return math.sqrt(math.fsum(float(np.dot(x, x)) for x in xs))


def want_factor(n, max_norm, eps):
    return min(1.0, f32(max_norm) / (n + f32(eps)))


def check_result(r, ts, kind, max_norm, eps=1e-6):
    n = want_norm(ts, kind)
    tol = U32 + sum(t.numel() for t in ts) * 2.0 ** -53
    got = host_f64(r)
    assert abs(got[0] - n) <= tol * n, (got[0], n)
    s = 1.0 if max_norm is None else want_factor(n, max_norm, eps)
    # below 2^-126 the fp32 values are 2^-149 apart whatever their size, so there
    # a rounding is off by up to 2^-150
    assert abs(got[1] - s) <= max(tol * s, 2.0 ** -150), (got[1], s)


@pytest.mark.parametrize("kind", [2, math.inf])
@pytest.mark.parametrize("which", ["bf16", "fp32", "mixed"])
def test_norm_ragged(kind, which):
    dts = {"bf16": [BF16] * len(NUMELS), "fp32": [FP32] * len(NUMELS),
           "mixed": mixed(len(NUMELS))}[which]
    ts = make(NUMELS, dts, 3)
    check_result(nsa.grad_norm_batched(ts, norm_type=kind), ts, kind, None)
    for max_norm in (1e-4, 1e3, 0.0):
        check_result(nsa.grad_norm_batched(ts, max_norm=max_norm, norm_type=kind), ts, kind, max_norm)


@pytest.mark.parametrize("numel", [0, 1, 8, 63, SPAN, SPAN + 1, 2 * SPAN])
def test_norm_of_one_tensor(numel):
    for dt in (BF16, FP32):
        ts = make([numel], [dt], 5)
        for kind in (2, math.inf):
            check_result(nsa.grad_norm_batched(ts, max_norm=0.5, norm_type=kind), ts, kind, 0.5)


@pytest.mark.parametrize("batch", [32, 33, 159, 160, 239, 240, 700, 2500])
def test_norm_and_clip_of_many_tensors(batch):
    # up to 239 tensors (159 into other buffers) travel as kernel arguments, more in
    # a table in the workspace
    rng = np.random.default_rng(batch)
    numels = [int(n) for n in rng.integers(0, 400, batch)]
    ts = make(numels, mixed(batch), batch)
    check_result(nsa.grad_norm_batched(ts, max_norm=1e-2), ts, 2, 1e-2)
    before = [t.clone() for t in ts]
    to = [torch.full_like(t, 7, dtype=FP32) for t in ts]
    r = nsa.grad_clip_batched(ts, 1e-2, out=to)
    check_result(r, before, 2, 1e-2)
    s = r[1].cpu()
    for t, o, b in zip(ts, to, before):
        assert torch.equal(t, b) and torch.equal(o.cpu(), b.cpu().float() * s)
    r = nsa.grad_clip_batched(ts, 1e-2)
    check_result(r, before, 2, 1e-2)
    s = r[1].cpu()
    for t, b in zip(ts, before):
        assert torch.equal(t.cpu(), (b.cpu().float() * s).to(b.dtype))


def test_norm_more_chunks_than_blocks():
    # 2048 blocks take several chunks each
    ts = make([2100 * SPAN + 11, 3 * SPAN], [BF16, FP32], 9)
    for kind in (2, math.inf):
        check_result(nsa.grad_norm_batched(ts, max_norm=0.25, norm_type=kind), ts, kind, 0.25)


def test_more_blocks_than_a_grid_row():
    """The scale pass gives 4096 elements to a block and AdamW 1024; 65536 blocks
    fill a row of their grids.  The elements around that edge and at the end."""
    row = 65536
    g = torch.full((row * 4096 + 5000,), 3.0, dtype=BF16, device="cuda")
    nsa.grad_scale_batched([g], torch.full((1,), 0.5, device="cuda"))
    assert bool((g == 1.5).all())
    n = row * 1024 + 1500
    p, d = torch.full((n,), 2.0, device="cuda"), torch.ones(n, device="cuda")
    m, v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    nsa.adamw_batched([p], [d], [m], [v], lr=0.25, betas=(0.5, 0.5), eps=0.0, weight_decay=0.0)
    # by the formulas, all exact: m = v = 1/2, the corrected moments are 1, p = 2 - 1/4 * 1 / 1
    # up to the roundings of lr / (1 - 1/2), sqrt(1/2) and its inverse: 8 half units
    assert bool((m == 0.5).all()) and bool((v == 0.5).all())
    assert float((p - 1.75).abs().max()) <= 8 * U32


def test_norm_over_the_range_of_fp32():
    # squares beyond fp32's range on either side
    for v, kinds in ((1e25, (2, math.inf)), (1e-25, (2, math.inf)), (3e38, (math.inf,)),
                     (1e-44, (math.inf,))):
        ts = [torch.full((1000,), v, device="cuda")]
        for kind in kinds:
            check_result(nsa.grad_norm_batched(ts, max_norm=1.0, norm_type=kind), ts, kind, 1.0)
    # a norm beyond fp32 is an infinity there
    r = nsa.grad_norm_batched([torch.full((1000,), 3e38, device="cuda")], max_norm=1.0).cpu()
    assert r[0] == math.inf


def test_non_finite_gradients():
    for kind in (2, math.inf):
        ts = make(NUMELS, mixed(len(NUMELS)), 11)
        ts[8][77] = math.inf
        r = nsa.grad_norm_batched(ts, max_norm=1.0, norm_type=kind).cpu()
        assert r[0] == math.inf and r[1] == 0.0
        ts[7][0] = math.nan
        r = nsa.grad_norm_batched(ts, max_norm=1.0, norm_type=kind).cpu()
        assert torch.isnan(r).all()
        nsa.grad_clip_batched(ts, 1.0, norm_type=kind)
        assert all(torch.isnan(t).all() for t in ts)
    z = [torch.zeros(100, device="cuda")]
    r = nsa.grad_norm_batched(z, max_norm=1.0, eps=0.0).cpu()
    assert r[0] == 0.0 and r[1] == 1.0
    r = nsa.grad_norm_batched(z, max_norm=0.0, eps=0.0).cpu()
    assert r[1] == 1.0


@pytest.mark.parametrize("src,dst", [(BF16, BF16), (BF16, FP32), (FP32, BF16), (FP32, FP32)])
@pytest.mark.parametrize("max_norm", [1e-3, 1e3])
def test_clip_into_other_buffers(src, dst, max_norm):
    ts = make(NUMELS, [src] * len(NUMELS), 13)
    before = [t.clone() for t in ts]
    # each output between guards that stay as they were
    room = [torch.full((n + 64,), 7.0, dtype=dst, device="cuda") for n in NUMELS]
    out = [r[32:32 + n] for r, n in zip(room, NUMELS)]
    r = nsa.grad_clip_batched(ts, max_norm, out=out)
    check_result(r, before, 2, max_norm)
    s = r[1].cpu()
    for t, b, o, rm, n in zip(ts, before, out, room, NUMELS):
        assert torch.equal(t, b)
        assert torch.equal(o.cpu(), (b.cpu().float() * s).to(dst))
        assert (rm[:32] == 7).all() and (rm[32 + n:] == 7).all()


def test_inactive_clip_leaves_gradients():
    ts = make(NUMELS, mixed(len(NUMELS)), 15)
    before = [t.clone() for t in ts]
    r = nsa.grad_clip_batched(ts, 1e9)
    assert float(r[1]) == 1.0
    assert all(torch.equal(a, b) for a, b in zip(ts, before))


def test_scale_with_a_factor_from_elsewhere():
    ts = make(NUMELS, mixed(len(NUMELS)), 17)
    before = [t.clone() for t in ts]
    s = torch.tensor([0.3], device="cuda")
    assert nsa.grad_scale_batched(ts, s) is not None
    for t, b in zip(ts, before):
        assert torch.equal(t.cpu(), (b.cpu().float() * s.cpu()).to(b.dtype))


def test_same_bits_every_time_and_on_another_stream():
    ts = make([3_000_017, 1234567], [FP32, BF16], 19)
    a = nsa.grad_norm_batched(ts, max_norm=0.1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b = nsa.grad_norm_batched(ts, max_norm=0.1)
    side.synchronize()
    assert torch.equal(a, b)


def test_capture_and_replay():
    # 40 tensors: the table is written by kernels inside the graph
    for count in (5, 40):
        ts = make([1000 + 131 * i for i in range(count)], mixed(count), 23)
        out = [torch.empty(t.numel(), dtype=BF16, device="cuda") for t in ts]
        ws = torch.empty(nsa.grad_workspace_bytes([t.numel() for t in ts]) + 256, dtype=torch.uint8,
                         device="cuda")
        ws = ws[(-ws.data_ptr()) % 256:]
        res = torch.empty(2, device="cuda")
        nsa.grad_clip_batched(ts, 1e-2, out=out, result=res, workspace=ws)  # warm
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            nsa.grad_clip_batched(ts, 1e-2, out=out, result=res, workspace=ws)
        for k in range(4):
            for t in ts:
                t.mul_(0.7)
            eager_out = [torch.empty_like(o) for o in out]
            eager = nsa.grad_clip_batched(ts, 1e-2, out=eager_out)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(res, eager), k
            assert all(torch.equal(a, b) for a, b in zip(out, eager_out)), k


def adamw_state(numels, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    p = [(torch.randn(n, generator=g) * 0.02).to(dtype).cuda() for n in numels]
    gr = [(torch.randn(n, generator=g) * 1e-3).to(dtype).cuda() for n in numels]
    m = [(torch.randn(n, generator=g) * 1e-3).cuda() for n in numels]
    v = [(torch.randn(n, generator=g) * 1e-3).square().cuda() for n in numels]
    return p, gr, m, v


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_adamw_with_a_factor(dtype):
    """m and v: four fp32 roundings of each term, as without a factor, and one
    more of each gradient (two in g^2) for the scaled product.  p: the bound of
    the plain step with those."""
    numels = [1, 7, 8191, 8192, 8193, 0, 100003]
    p, g, m, v = adamw_state(numels, dtype, 31)
    before = [[host_f64(t) for t in x] for x in (p, g, m, v)]
    r = nsa.grad_norm_batched(g, max_norm=0.05)
    s = float(r[1])
    assert s < 1
    nsa.adamw_batched(p, g, m, v, lr=1e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1, step=3,
                      grad_scale=r[1:])
    lr, b1, b2, eps, wd = (f32(x) for x in (1e-3, 0.9, 0.95, 1e-8, 0.1))
    for i in range(len(numels)):
        p0, g0, m0, v0 = (x[i] for x in before)
        pr, mr, vr = oracle.adamw_step(p0, s * g0, m0, v0, lr=lr, beta1=b1, beta2=b2, eps=eps,
                                       weight_decay=wd, step=3)
        sg = np.abs(s * g0)
        bm = U32 * (4 * b1 * np.abs(m0) + 5 * (1 - b1) * sg) + 1e-38
        bv = U32 * (4 * b2 * v0 + 6 * (1 - b2) * sg * sg) + 1e-38
        assert np.all(np.abs(host_f64(m[i]) - mr) <= bm)
        assert np.all(np.abs(host_f64(v[i]) - vr) <= bv)
        sz, c = lr / (1 - b1 ** 3), 1 / math.sqrt(1 - b2 ** 3)
        d = c * np.sqrt(vr) + eps
        carried = sz * bm / d + sz * np.abs(mr) * (c * bv / (2 * np.sqrt(vr) + 1e-30)) / d ** 2
        upd = np.abs(pr - p0 * (1 - lr * wd))
        bp = U32 * (2 * np.abs(pr) + 8 * upd + 2 * np.abs(p0)) + carried + 1e-38
        got = host_f64(p[i])
        if dtype == BF16:
            bp = bp * (1 + 2.0 ** -7) + 2.0 ** -8 * np.abs(pr)
        assert np.all(np.abs(got - pr) <= bp), float(np.max(np.abs(got - pr) / bp))


@pytest.mark.parametrize("batch,numel", [(83, 100), (84, 100), (250, 3000), (84, 210000), (200, 130000)])
def test_adamw_of_many_tensors_equals_one_at_a_time(batch, numel):
    # up to 83 tensors in one argument table; more in a table in the workspace, or in
    # several launches where each has 8192 blocks of 1024 elements
    rng = np.random.default_rng(batch)
    numels = [int(n) for n in rng.integers(numel - 50, numel + 50, batch)]
    numels[0], numels[batch // 2], numels[-1] = 0, 0, 1
    p, g, m, v = adamw_state(numels, BF16, batch)
    q, n, w = ([x.clone() for x in t] for t in (p, m, v))
    s = torch.full((1,), 0.3, device="cuda")
    nsa.adamw_batched(p, g, m, v, step=2, grad_scale=s)
    for a, b, c, d in zip(q, g, n, w):
        nsa.adamw_batched([a], [b], [c], [d], step=2, grad_scale=s)
    for x, y in ((p, q), (m, n), (v, w)):
        assert all(torch.equal(a, b) for a, b in zip(x, y))


def test_a_factor_of_one_changes_nothing():
    one = torch.ones(1, device="cuda")
    for dtype in (BF16, FP32):
        a = adamw_state([8192 * 3 + 5, 77], dtype, 37)
        b = [[t.clone() for t in x] for x in a]
        nsa.adamw_batched(*a, step=2)
        nsa.adamw_batched(*b, step=2, grad_scale=one)
        assert all(torch.equal(x, y) for p, q in zip(a, b) for x, y in zip(p, q))
        gen = torch.Generator().manual_seed(41)
        ws, gs, ms = ([(torch.randn(sh, generator=gen) * 1e-2).to(dtype).cuda()
                       for sh in ((300, 700), (700, 301), (64, 64))] for _ in range(3))
        ws2, ms2 = [w.clone() for w in ws], [m.clone() for m in ms]
        nsa.step_batched(ws, gs, ms, nesterov=True)
        nsa.step_batched(ws2, gs, ms2, nesterov=True, grad_scale=one)
        assert all(torch.equal(x, y) for x, y in zip(ws + ms, ws2 + ms2))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("nesterov", [False, True])
def test_muon_step_with_a_power_of_two_factor(dtype, nesterov):
    """s = 1/4 multiplies exactly, so the step on g equals, bit for bit, the plain
    step on gradients divided by 4; tall, wide and odd shapes, device and host
    momentum."""
    s = torch.tensor([0.25], device="cuda")
    shapes = ((300, 700), (700, 300), (257, 771), (771, 257), (64, 100), (100, 63))
    gen = torch.Generator().manual_seed(43)
    ws, gs, ms = ([(torch.randn(sh, generator=gen) * 1e-2).to(dtype).cuda() for sh in shapes]
                  for _ in range(3))
    ref_w, ref_m = [w.clone() for w in ws], [m.clone() for m in ms]
    host_w, host_m = [w.clone() for w in ws], [torch.empty(m.shape, dtype=dtype, pin_memory=True).copy_(m)
                                               for m in ms]
    nsa.step_batched(ref_w, [g * 0.25 for g in gs], ref_m, nesterov=nesterov)
    nsa.step_batched(ws, gs, ms, nesterov=nesterov, grad_scale=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ws + ms, ref_w + ref_m))
    nsa.step_batched(host_w, gs, host_m, nesterov=nesterov, grad_scale=s, momentum_host=True)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(host_w, ref_w))
    assert all(torch.equal(a, b.cpu()) for a, b in zip(host_m, ref_m))


def test_muon_momentum_with_a_factor():
    """M' = beta M + s G: two fp32 roundings of s G and one of the sum, then the
    storage rounding."""
    gen = torch.Generator().manual_seed(47)
    for dtype, store in ((BF16, 2.0 ** -8), (FP32, 0.0)):
        w, g, m = ((torch.randn((333, 515), generator=gen) * 1e-2).to(dtype).cuda() for _ in range(3))
        m0, g0 = host_f64(m), host_f64(g)
        r = nsa.grad_norm_batched([g], max_norm=0.7)
        s = float(r[1])
        nsa.step_batched([w], [g], [m], beta=0.95, grad_scale=r[1:])
        want = f32(0.95) * m0 + s * g0
        terms = np.abs(f32(0.95) * m0) + np.abs(s * g0)
        assert np.all(np.abs(host_f64(m) - want) <= 3 * U32 * terms * (1 + store) + store * np.abs(want) + 1e-38)


def test_binding_refuses_what_the_library_cannot_see():
    t = torch.zeros(64, device="cuda")
    for bad in (torch.ones(1), torch.ones(2, device="cuda"), torch.ones(1, device="cuda").double(), 0.5):
        with pytest.raises(ValueError):
            nsa.grad_scale_batched([t], bad)
    with pytest.raises(TypeError):
        nsa.grad_norm_batched([t.half()])
    with pytest.raises(ValueError):
        nsa.grad_norm_batched([t.view(8, 8).t()])
    with pytest.raises(ValueError):
        nsa.grad_norm_batched([t, torch.zeros(3)])
    with pytest.raises(ValueError):
        nsa.grad_clip_batched([t], 1.0, out=[torch.zeros(63, device="cuda")])
    with pytest.raises(nsa.MuonError):
        nsa.grad_norm_batched([t[1:]])  # not 16-byte aligned
    with pytest.raises(nsa.MuonError):
        nsa.grad_norm_batched([t], max_norm=-1.0)
    n = nsa.grad_workspace_bytes([64])
    for bad in (torch.empty(n, dtype=torch.uint8), torch.empty(n, device="cuda"),
                torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            nsa.grad_norm_batched([t], workspace=bad)
    with pytest.raises(nsa.MuonError):
        nsa.grad_norm_batched([t], workspace=torch.empty(n - 1, dtype=torch.uint8, device="cuda"))
