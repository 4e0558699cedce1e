"""Dropout against the generator's plain form: one fp32 product an element, rounded
once, so outputs are equal bits."""
import numpy as np
import pytest
import torch

import expert_plain as plain
import newton_schulz_03_amd as nsa
from test_captured_calls import replays

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
SPAN = 16384
NUMELS = [1, 7, 8, 9, 255, 4095, 4096, 4097, 0, 8193, SPAN - 1, SPAN, SPAN + 1, 3 * SPAN + 5]


@pytest.fixture(autouse=True)
def _announce(request):
    print(f"\n[gpu-test] {request.node.name}", flush=True)
    yield
    torch.cuda.synchronize()


def make(numels, dtypes, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(n, generator=g).to(dt).cuda() for n, dt in zip(numels, dtypes)]


def want(x, i, p, seed, offset, dtype):
    thr = round(p * 65536)
    on = torch.from_numpy(plain.keep(x.numel(), i, seed, offset, thr)).view(x.shape)
    scale = np.float32(65536 / (65536 - thr)) if thr < 65536 else np.float32(0)
    return torch.where(on, x.cpu().float() * torch.tensor(scale), torch.zeros(())).to(dtype)


def same(a, b):
    raw = torch.int16 if a.dtype == BF16 else torch.int32
    return torch.equal(a.cpu().view(raw), b.cpu().view(raw))


DTYPES = {"bf16": [BF16] * len(NUMELS), "fp32": [FP32] * len(NUMELS),
          "mixed": [BF16 if i % 3 else FP32 for i in range(len(NUMELS))]}


@pytest.mark.parametrize("out", [None, BF16, FP32])
@pytest.mark.parametrize("which", list(DTYPES))
@pytest.mark.parametrize("p", [0.1, 0.5, 0.97])
def test_ragged(which, out, p):
    xs = make(NUMELS, DTYPES[which], 3)
    seed, offset = (7 << 40) + 5, (3 << 33) + 11
    wants = [want(x, i, p, seed, offset, out or x.dtype) for i, x in enumerate(xs)]
    if out is None:
        got = nsa.dropout_batched(xs, p, seed=seed, offset=offset)
        assert all(g is x for g, x in zip(got, xs))
    else:
        before = [x.clone() for x in xs]
        to = [torch.full_like(x, 7, dtype=out) for x in xs]
        got = nsa.dropout_batched(xs, p, seed=seed, offset=offset, out=to)
        assert all(g is t for g, t in zip(got, to)) and all(same(x, b) for x, b in zip(xs, before))
    for g, w in zip(got, wants):
        assert same(g, w)


def test_ends_of_p():
    x = make([1000], [FP32], 1)[0]
    x[::3] = float("nan")
    x[1::3] = float("inf")
    for p in (0.0, 1e-6):  # nothing is dropped
        assert same(nsa.dropout_batched([x], p, seed=1, out=[torch.zeros_like(x)])[0], x)
    out = nsa.dropout_batched([x], 1.0, seed=1, out=[torch.ones_like(x)])[0]
    assert not bool(out.any()) and not bool(torch.signbit(out).any())
    p = 65535 / 65536
    assert same(nsa.dropout_batched([x], p, seed=4, out=[torch.zeros_like(x)])[0],
                want(x, 0, p, 4, 0, FP32))


def test_dropped_infinities_and_nans_are_zero():
    for dt in (BF16, FP32):
        x = make([4096], [dt], 1)[0]
        x[::2] = float("nan")
        x[1::2] = float("inf")
        got = nsa.dropout_batched([x], 0.5, seed=9, out=[torch.zeros_like(x)])[0]
        on = torch.from_numpy(plain.keep(4096, 0, 9, 0, 32768)).cuda()
        assert bool((got[~on] == 0).all()) and not bool(torch.isfinite(got[on]).any())


def test_the_gradient_is_the_same_call():
    """Against differences: with whole numbers and p = 1/2 every value is exact."""
    x = torch.arange(-500, 500, device="cuda").float()
    dy = torch.arange(1000, device="cuda").float().remainder_(17)
    drop = lambda v: nsa.dropout_batched([v], 0.5, seed=3, offset=8, out=[torch.empty_like(v)])[0]
    dx, y = drop(dy), drop(x)
    step = (drop(x + 1) - y) * dy
    assert torch.equal(step, dx)


@pytest.mark.parametrize("batch", [159, 160, 239, 240, 700])
def test_many_tensors(batch):
    # tables of up to 239 tensors (159 into other buffers) travel as kernel arguments
    rng = np.random.default_rng(batch)
    xs = make([int(n) for n in rng.integers(0, 300, batch)], [BF16 if i % 2 else FP32 for i in range(batch)], batch)
    wants = [want(x, i, 0.25, 5, 6, x.dtype) for i, x in enumerate(xs)]
    to = [torch.full_like(x, 7) for x in xs]
    for got in (nsa.dropout_batched(xs, 0.25, seed=5, offset=6, out=to), nsa.dropout_batched(xs, 0.25, seed=5, offset=6)):
        assert all(same(g, w) for g, w in zip(got, wants))


@pytest.mark.parametrize("pair", [(BF16, BF16), (FP32, FP32), (FP32, BF16), (BF16, FP32)])
def test_large_and_numbers_on_the_device(pair):
    n = 40_000_003
    x = torch.empty(n, device="cuda").normal_().to(pair[0])
    rng = torch.tensor([-5, 1 << 62], device="cuda")  # as unsigned: 2^64 - 5
    out = torch.zeros(n, dtype=pair[1], device="cuda")
    nsa.dropout_batched([x], 0.3, rng=rng, out=[out])
    assert same(out, want(x, 0, 0.3, (1 << 64) - 5, 1 << 62, pair[1]))


def test_more_than_2_31_elements():
    """The blocks' numbers and addresses past 2^31 elements (4.4 GB of bf16)."""
    n = (1 << 31) + 70_001
    x = torch.ones(n, dtype=BF16, device="cuda")
    nsa.dropout_batched([x], 0.5, seed=1)
    tail = 40_000
    m = 0xFFFFFFFF
    first = (n - tail) // 8 * 8
    block = np.arange(first // 8, (n + 7) // 8, dtype=np.uint64)
    words = plain.philox([block, block * 0, block * 0, block * 0], (1 & m, 0), 7)
    u = np.stack([(w >> np.uint64(16 * h)) & np.uint64(0xFFFF) for w in words for h in (0, 1)], 1).ravel()[:n - first]
    assert torch.equal(x[first:].cpu().float(), torch.from_numpy(np.where(u < 32768, 0.0, 2.0)).float())
    head = plain.keep(4096, 0, 1, 0, 32768)
    assert torch.equal(x[:4096].cpu().float(), torch.from_numpy(np.where(head, 2.0, 0.0)).float())


def test_captured():
    """A replay takes the numbers that the device tensor holds by then."""
    xs = make([5000, 77, 20000], [BF16, FP32, BF16], 2)
    out, wants = ([torch.zeros_like(x) for x in xs] for _ in range(2))
    rng = torch.tensor([3, 4], device="cuda")

    def change(k):
        rng.add_(torch.tensor([0, 1], device="cuda"))
        for x in xs:
            x.mul_(-1.5)

    def eager():
        seed, offset = rng.tolist()
        nsa.dropout_batched(xs, 0.4, seed=seed, offset=offset, out=wants)

    replays(lambda: nsa.dropout_batched(xs, 0.4, rng=rng, out=out), eager, lambda: zip(out, wants), change)


def test_on_another_stream():
    xs = make([300_000], [FP32], 2)
    expect = want(xs[0], 0, 0.4, 1, 2, FP32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        late = torch.empty_like(xs[0])
        for _ in range(50):
            late.copy_(xs[0])
        nsa.dropout_batched([late], 0.4, seed=1, offset=2)
    s.synchronize()
    assert same(late, expect)


def test_binding_refusals():
    x = torch.ones(8, device="cuda")
    for call in (lambda: nsa.dropout_batched([x], 0.5, rng=torch.zeros(2, device="cuda")),
                 lambda: nsa.dropout_batched([x], 0.5, rng=torch.zeros(2, dtype=torch.int64)),
                 lambda: nsa.dropout_batched([x], 0.5, rng=torch.zeros(3, dtype=torch.int64, device="cuda")),
                 lambda: nsa.dropout_batched([x[::2]], 0.5), lambda: nsa.dropout_batched([x], 0.5, out=[]),
                 lambda: nsa.dropout_batched([x], 0.5, out=[x[:7]])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        nsa.dropout_batched([x.half()], 0.5)
    for p in (-0.5, 1.5):
        with pytest.raises(nsa.MuonError):
            nsa.dropout_batched([x], p)
    twin = torch._lazy_clone(x)
    nsa.dropout_batched([twin], 1.0)
    assert bool((x == 1).all()) and not bool(twin.any())
