"""Block-scaled e4m3 operands and their product against 64-bit arithmetic.

Quantization is exact arithmetic up to the one rounding, so operands are
compared value by value and scale by scale with a numpy implementation in
float64.

Products, fp32 output: every product of two e4m3 values and the powers of two
are exact; the sum of K of them is formed in fp32, each of at most K additions
off by at most one unit in the last place of a partial sum, 2^-23 of the sum of
magnitudes (whether it rounds or cuts off); then one rounding to the output
(2^-24), with the old output added in fp32 before it.

Products, bf16 output: the e4m3 matrix instruction first adds 8 consecutive
products on a common grid whose step is at most 2^-13 of the largest of the 8
(measured with two products: the smaller counts at 2^-13 of the larger, and is
lost at 2^-14).  Each product is then off by less than 2^-13 of the group's
largest, the group by less than 8 * 2^-13 = 2^-10 of it, and the sum over the
groups by less than 2^-10 of the sum of magnitudes; the rounding is 2^-8 of the
value.
"""
import math

import numpy as np
import pytest
import torch

import newton_schulz_03_amd as nsa
from parity_util import host_f64

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
BLOCK = 128


@pytest.fixture(autouse=True)
def _announce(request):
    print(f"\n[gpu-test] {request.node.name}", flush=True)
    yield
    torch.cuda.synchronize()


def up(x, a):
    return (x + a - 1) // a * a


def e4m3(x):
    """float64 values (|x| <= 448) rounded to nearest even e4m3 values."""
    a = np.abs(x)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), -6.0)
    # log2 may round up to the next integer just below a power of two
    e = np.where(np.exp2(e) > np.where(a > 0, a, 1.0), np.maximum(e - 1, -6.0), e)
    step = np.exp2(e - 3)
    return np.sign(x) * np.rint(a / step) * step


def quantize(x, block_rows):
    """(values, scale bytes) of float64 x, contracted over its columns."""
    r, k = x.shape
    kp, rp = up(k, BLOCK), up(r, 16)
    v = np.zeros((up(r, block_rows), kp))
    v[:r, :k] = x
    mag = np.where(np.isfinite(v), np.abs(v), 0.0)
    top = mag.reshape(v.shape[0] // block_rows, block_rows, kp // BLOCK, BLOCK).max(axis=(1, 3),
                                                                                  initial=0.0)
    e = np.full(top.shape, -127.0)
    pos = top > 0
    # the smallest e with top <= 448 * 2^e
    c = np.floor(np.log2(np.where(pos, top, 1.0) / 448.0)) - 1
    for _ in range(3):
        c = np.where(top > 448.0 * np.exp2(c), c + 1, c)
    e = np.where(pos, np.maximum(c, -127.0), e)
    er = np.repeat(e, block_rows, axis=0)[:r]
    s = v[:r].reshape(r, kp // BLOCK, BLOCK) * np.exp2(-er)[:, :, None]
    s = s.reshape(r, kp)
    bad = ~np.isfinite(s)
    q = e4m3(np.where(bad, 0.0, s))
    q[bad] = np.nan
    scales = np.zeros((kp // BLOCK, rp), np.int64)
    scales[:, :r] = (er + 127).T
    return q, scales


def values(op):
    """What an operand stands for, in float64, and its scale bytes."""
    q = op[0].cpu().to(FP32).double().numpy()
    s = op[1].cpu().numpy().astype(np.int64)
    r, kp = q.shape
    p = np.exp2(s[:, :r].T.astype(np.float64) - 127)
    return (q.reshape(r, kp // BLOCK, BLOCK) * p[:, :, None]).reshape(r, kp)


def check_operand(op, x, block_rows, what):
    q, s = quantize(x, block_rows)
    got = op[0].cpu().to(FP32).double().numpy()
    assert got.shape == q.shape and tuple(op[1].shape) == s.shape, what
    assert np.array_equal(op[1].cpu().numpy().astype(np.int64), s), what
    assert np.array_equal(got, q, equal_nan=True), what


def matrix(rows, cols, dtype, seed, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g)
    return (x * torch.exp(spread * torch.randn((rows, 1), generator=g))).to(dtype)


SHAPES = [(1, 1), (1, 128), (3, 127), (16, 129), (17, 256), (127, 8), (128, 128), (129, 130),
          (255, 384), (300, 1000), (0, 64), (64, 0), (5, 1003)]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_ragged(dtype, block_rows):
    xs = [matrix(r, c, dtype, 100 + i) for i, (r, c) in enumerate(SHAPES)]
    dev = [x.cuda() for x in xs]
    ops, ops_t = nsa.f8_quantize_batched(dev, block_rows=block_rows, transpose=True)
    only = nsa.f8_quantize_batched(dev, block_rows=block_rows)
    only_t = nsa.f8_quantize_batched(dev, block_rows=block_rows, normal=False, transpose=True)
    for i, x in enumerate(xs):
        h = x.double().numpy()
        check_operand(ops[i], h, block_rows, SHAPES[i])
        check_operand(ops_t[i], np.ascontiguousarray(h.T), block_rows, SHAPES[i])
        for a, b in ((ops[i], only[i]), (ops_t[i], only_t[i])):
            assert torch.equal(a.q.view(torch.uint8), b.q.view(torch.uint8))
            assert torch.equal(a.scales, b.scales)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_edges_of_the_range(block_rows, dtype):
    # block maxima at the steps of the scale, ties between e4m3 values, the
    # largest and smallest fp32 values, zeros, infinities and NaNs
    x = torch.zeros((150, 400))
    g = torch.Generator().manual_seed(7)
    for r in range(128):
        x[r, :128] = torch.randn(128, generator=g) * 2.0 ** (r % 40 - 20)
    tops = [448.0, 448.0 * (1 + 2 ** -23), 447.99, 0.875, 1.75, 1.7500001, 3.4e38, 1e-38, 1e-40, 1e-45, 0.0]
    for r, t in enumerate(tops):
        x[r, 128:256] = torch.linspace(-1, 1, 128) * t
        x[r, 200] = t
    x[20, 128:256] = torch.arange(128) / 16.0 * (1 + 1 / 32)  # around ties
    x[20, 130] = 448.0
    x[21, 128] = 256.0
    x[21, 129:140] = torch.tensor([2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -11, 17.0, 17.5, 18.0, 18.5, 19.0,
                                   -2.0 ** -10, -17.0, 0.0])
    x[22, 300] = math.inf
    x[23, 300:310] = math.nan
    x[24, 256:384] = -math.inf
    x[140, 390] = math.nan
    x = x.to(dtype)
    h = x.double().numpy()
    ops, ops_t = nsa.f8_quantize_batched([x.cuda()], block_rows=block_rows, transpose=True)
    check_operand(ops[0], h, block_rows, "range")
    check_operand(ops_t[0], np.ascontiguousarray(h.T), block_rows, "range, transposed")


def test_quantize_into_given_operands_leaves_the_rest():
    x = matrix(37, 300, BF16, 5).cuda()
    kp, rp = 384, 48
    q = torch.full((256 + 37 * kp + 256,), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((256 + 3 * rp + 256,), 0x55, dtype=torch.uint8, device="cuda")
    op = (q[256:256 + 37 * kp].view(37, kp).view(torch.float8_e4m3fn), s[256:256 + 3 * rp].view(3, rp))
    qt = torch.full((256 + 300 * 128 + 256,), 0x55, dtype=torch.uint8, device="cuda")
    st = torch.full((256 + 304 + 256,), 0x55, dtype=torch.uint8, device="cuda")
    op_t = (qt[256:256 + 300 * 128].view(300, 128).view(torch.float8_e4m3fn), st[256:256 + 304].view(1, 304))
    nsa.f8_quantize_batched([x], transpose=True, out=[op], out_t=[op_t])
    h = host_f64(x)
    check_operand(op, h, 1, "given")
    check_operand(op_t, np.ascontiguousarray(h.T), 1, "given, transposed")
    for t, n in ((q, 37 * kp), (s, 3 * rp), (qt, 300 * 128), (st, 304)):
        assert (t[:256] == 0x55).all() and (t[256 + n:] == 0x55).all()


def operands(shapes, seed, b_rows=1):
    a = [matrix(m, k, FP32, seed + 2 * i, 1.0) for i, (m, n, k) in enumerate(shapes)]
    b = [matrix(n, k, FP32, seed + 2 * i + 1, 1.0) for i, (m, n, k) in enumerate(shapes)]
    return (nsa.f8_quantize_batched([x.cuda() for x in a]),
            nsa.f8_quantize_batched([x.cuda() for x in b], block_rows=b_rows))


def check_product(c, a, b, old=None, what=""):
    x, y = values(a), values(b)
    if x.shape[0] * y.shape[0] * x.shape[1] > 1 << 28:  # the same in float64 on the device
        dx, dy = torch.from_numpy(x).cuda(), torch.from_numpy(y).cuda().t().contiguous()
        want, mag = (dx @ dy).cpu().numpy(), (dx.abs() @ dy.abs()).cpu().numpy()
    else:
        want, mag = x @ y.T, np.abs(x) @ np.abs(y).T
    acc = x.shape[1] * 2.0 ** -23 * mag
    if c.dtype == BF16:
        acc = acc + 2.0 ** -10 * mag
    if old is not None:
        want = want + old
        acc = acc + 2.0 ** -24 * np.abs(want)
    half = 2.0 ** -8 if c.dtype == BF16 else 2.0 ** -24
    tol = acc * (1 + half) + half * np.abs(want) + 1e-38
    off = np.abs(host_f64(c) - want)
    assert np.all(off <= tol), (what, float(np.max(off / tol)))


PRODUCTS = [(1, 1, 1), (1, 300, 129), (300, 1, 500), (7, 9, 128), (16, 64, 64), (128, 128, 128),
            (255, 257, 256), (256, 256, 384), (257, 255, 640), (513, 130, 1000), (0, 40, 30), (40, 0, 30),
            (33, 70, 0), (2, 1024, 2048), (600, 16, 72)]


@pytest.mark.parametrize("out", [BF16, FP32])
@pytest.mark.parametrize("accumulate", [False, True])
def test_matmul_ragged(out, accumulate):
    a, b = operands(PRODUCTS, 1000)
    # each output between guards that stay as they were
    room = [torch.full((16 + m * n + 16,), 3.0, dtype=out, device="cuda") for m, n, _ in PRODUCTS]
    c = [r[16:16 + m * n].view(m, n) for r, (m, n, _) in zip(room, PRODUCTS)]
    g = torch.Generator().manual_seed(3)
    for x in c:
        x.copy_(torch.randn(tuple(x.shape), generator=g))
    old = [host_f64(x) for x in c]
    got = nsa.f8_matmul_batched(a, b, out=c, accumulate=accumulate)
    torch.cuda.synchronize()
    for i, s in enumerate(PRODUCTS):
        assert got[i] is c[i]
        check_product(c[i], a[i], b[i], old[i] if accumulate else None, s)
        assert (room[i][:16] == 3).all() and (room[i][16 + s[0] * s[1]:] == 3).all(), s


# enough work for the 256 x 256 tiles: rests of rows below and above 128, of
# columns, odd numbers of K blocks, a single one and none
LARGE = [(700, 2100, 1500), (1290, 1030, 2048), (257, 2050, 128), (129, 1000, 900), (128, 2304, 1300),
         (384, 1024, 1100), (513, 777, 0), (70, 2000, 2000), (1024, 1025, 640), (33, 600, 700)]


@pytest.mark.parametrize("out", [BF16, FP32])
@pytest.mark.parametrize("accumulate", [False, True])
def test_matmul_large_tiles(out, accumulate):
    a, b = operands(LARGE, 2000, b_rows=128)
    room = [torch.full((16 + m * n + 16,), 3.0, dtype=out, device="cuda") for m, n, _ in LARGE]
    c = [r[16:16 + m * n].view(m, n) for r, (m, n, _) in zip(room, LARGE)]
    g = torch.Generator().manual_seed(5)
    for x in c:
        x.copy_(torch.randn(tuple(x.shape), generator=g))
    old = [host_f64(x) for x in c]
    nsa.f8_matmul_batched(a, b, out=c, accumulate=accumulate)
    torch.cuda.synchronize()
    for i, s in enumerate(LARGE):
        check_product(c[i], a[i], b[i], old[i] if accumulate else None, s)
        assert (room[i][:16] == 3).all() and (room[i][16 + s[0] * s[1]:] == 3).all(), s


@pytest.mark.parametrize("out", [BF16, FP32])
@pytest.mark.parametrize("shapes", [[(2048, 2048, 700)], [(1536, 1500, 1400)],
                                    [(2048 + r, 1100, 500 + r) for r in (0, 20, 64, 100, 150, 192, 200)]])
def test_matmul_smaller_tiles(out, shapes):
    # launches of less than a round, and rests of rows of every kind
    a, b = operands(shapes, 2700, b_rows=128)
    room = [torch.full((16 + m * n + 16,), 3.0, dtype=out, device="cuda") for m, n, _ in shapes]
    c = [x[16:16 + s[0] * s[1]].view(s[:2]) for x, s in zip(room, shapes)]
    g = torch.Generator().manual_seed(7)
    for x in c:
        x.copy_(torch.randn(tuple(x.shape), generator=g))
    old = [host_f64(x) for x in c]
    nsa.f8_matmul_batched(a, b, out=c, accumulate=True)
    torch.cuda.synchronize()
    for i, s in enumerate(shapes):
        check_product(c[i], a[i], b[i], old[i], s)
        assert (room[i][:16] == 3).all() and (room[i][16 + s[0] * s[1]:] == 3).all(), s


@pytest.mark.parametrize("out", [BF16, FP32])
def test_matmul_tiles_of_every_size_give_the_same_bits(out):
    # 2048 rows alone are cut into small tiles, among 16384 into whole ones
    (a,), (b,) = operands([(16384, 2048, 700)], 2800)
    (whole,) = nsa.f8_matmul_batched([a], [b], out_dtype=out)
    for first, rows in ((0, 2048), (4096, 1536), (8192, 2048 + 160)):
        part = (a.q[first:first + rows], a.scales[:, first:first + rows].contiguous())
        (c,) = nsa.f8_matmul_batched([part], [b], out_dtype=out)
        if out == FP32 and rows == 1536:
            # 192 quarter tiles are estimated at 16.9 us and 768 blocks of the kernel of
            # few rows at 16.5: that kernel's four waves share K, another order of the sum
            check_product(c, part, b)
        else:
            assert torch.equal(c, whole[first:first + rows]), (first, rows)


@pytest.mark.parametrize("out", [BF16, FP32])
@pytest.mark.parametrize("m,n", [(1100, 1290), (1290, 1500), (16, 2000), (70, 900)])
def test_matmul_lengths_that_differ(out, m, n):
    # every product's blocks are dealt over the chip, longest sums first
    shapes = [(m, n, k) for k in (130, 256, 4000, 300, 2000, 0, 700)] + [(m // 2, n // 3, 3900)]
    a, b = operands(shapes, 2500, b_rows=128)
    room = [torch.full((16 + r * c + 16,), 3.0, dtype=out, device="cuda") for r, c, _ in shapes]
    c = [x[16:16 + s[0] * s[1]].view(s[:2]) for x, s in zip(room, shapes)]
    nsa.f8_matmul_batched(a, b, out=c)
    torch.cuda.synchronize()
    for i, s in enumerate(shapes):
        check_product(c[i], a[i], b[i], None, s)
        assert (room[i][:16] == 3).all() and (room[i][16 + s[0] * s[1]:] == 3).all(), s


@pytest.mark.parametrize("tiles", [255, 257, 300, 513])
def test_matmul_last_round_in_half_tiles(tiles):
    # one row of tiles more or less than whole rounds of the chip: the bits of a
    # row of C do not depend on where its tile ends
    (a,), (b,) = operands([(256 * tiles - 100, 200, 256)], 3000 + tiles)
    for out in (BF16, FP32):
        (c,) = nsa.f8_matmul_batched([a], [b], out_dtype=out)
        rows = torch.randperm(256 * tiles - 100, generator=torch.Generator().manual_seed(1))[:600]
        rows = torch.cat([rows, torch.arange(256 * tiles - 400, 256 * tiles - 100)])
        part = (a.q[rows.cuda()], a.scales[:, rows.cuda()].contiguous())
        check_product(c[rows.cuda()], (part[0], part[1]), b, what=tiles)


@pytest.mark.parametrize("out", [BF16, FP32])
@pytest.mark.parametrize("accumulate", [False, True])
def test_matmul_outputs_past_the_caches(out, accumulate):
    # more than 256 MB, which passes the caches by; rows at the tiles' edges and others
    m, n = 8300, 8200 if out == FP32 else 16400
    (a,), (b,) = operands([(m, n, 200)], 3500)
    c = torch.ones(m, n, dtype=out, device="cuda")
    nsa.f8_matmul_batched([a], [b], out=[c], accumulate=accumulate)
    rows = torch.cat([torch.arange(250, 260), torch.arange(m - 140, m),
                      torch.randperm(m, generator=torch.Generator().manual_seed(2))[:150]]).cuda()
    part = (a.q[rows], torch.nn.functional.pad(a.scales[:, rows], (0, 4)))  # up to 304
    check_product(c[rows], part, b, np.ones((300, n)) if accumulate else None)


@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 31, 33, 48, 64, 65, 100, 129, 200])
def test_matmul_few_rows(m):
    shapes = [(m, 520, 1280), (m, 136, 256), (m, 33, 4096)]
    a, b = operands(shapes, 50 + m, b_rows=128)
    for out in (BF16, FP32):
        c = nsa.f8_matmul_batched(a, b, out_dtype=out)
        for i, s in enumerate(shapes):
            check_product(c[i], a[i], b[i], what=s)


@pytest.mark.parametrize("m", [3, 20, 50])
@pytest.mark.parametrize("n", [3900, 7000])
def test_matmul_few_rows_many_columns(m, n):
    # wider blocks than the shapes above take
    shapes = [(m, n, 700), (m - 2, 33, 300)]
    a, b = operands(shapes, 60 + m + n, b_rows=128)
    for out in (BF16, FP32):
        c = nsa.f8_matmul_batched(a, b, out_dtype=out)
        for i, s in enumerate(shapes):
            check_product(c[i], a[i], b[i], what=s)


@pytest.mark.parametrize("out", [BF16, FP32])
@pytest.mark.parametrize("shapes", [[(4096, 4000, 300), (8, 64, 24000)],
                                    [(4096, 4000, 300), (8, 64, 24000), (33, 70, 12000), (2048, 2048, 128)]])
def test_matmul_long_sums_of_few_rows_beside_large_products(out, shapes):
    # the few rows' long sums would outlast the tiles: the first call takes both
    # kernels, the second one that of few rows
    a, b = operands(shapes, 70, b_rows=128)
    room = [torch.full((16 + m * n + 16,), 3.0, dtype=out, device="cuda") for m, n, _ in shapes]
    c = [x[16:16 + s[0] * s[1]].view(s[:2]) for x, s in zip(room, shapes)]
    nsa.f8_matmul_batched(a, b, out=c)
    torch.cuda.synchronize()
    for i, s in enumerate(shapes):
        check_product(c[i], a[i], b[i], None, s)
        assert (room[i][:16] == 3).all() and (room[i][16 + s[0] * s[1]:] == 3).all(), s


@pytest.mark.parametrize("k", [1, 128, 129, 256, 320, 512, 640, 896, 1152])
def test_matmul_lengths_of_the_sum(k):
    # one block, two, odd numbers of them
    shapes = [(300, 270, k), (5, 270, k)]
    a, b = operands(shapes, 80 + k)
    c = nsa.f8_matmul_batched(a, b, out_dtype=FP32)
    for i, s in enumerate(shapes):
        check_product(c[i], a[i], b[i], what=s)


def test_matmul_every_value_in_its_place():
    # identity: each row of A alone, scales that differ by row and block
    n = 300
    eye = torch.eye(n)
    b = matrix(n, n, FP32, 9, 2.0)
    (ia,) = nsa.f8_quantize_batched([eye.cuda()])
    (ob,) = nsa.f8_quantize_batched([b.cuda()])
    (c,) = nsa.f8_matmul_batched([ia], [ob], out_dtype=FP32)
    assert np.array_equal(host_f64(c), values(ob)[:, :n].T.astype(np.float32).astype(np.float64))
    (c,) = nsa.f8_matmul_batched([ob], [ia], out_dtype=FP32)
    assert np.array_equal(host_f64(c), values(ob)[:, :n].astype(np.float32).astype(np.float64))


def test_matmul_scales_at_the_ends():
    # the largest and smallest scale bytes, in one operand at a time
    for lo in (1e-36, 1e30):
        x = matrix(40, 200, FP32, 21, 0.0) * lo
        y = matrix(50, 200, FP32, 22, 0.0) / lo
        a = nsa.f8_quantize_batched([x.cuda()])
        b = nsa.f8_quantize_batched([y.cuda()])
        (c,) = nsa.f8_matmul_batched(a, b, out_dtype=FP32)
        check_product(c, a[0], b[0], what=lo)


def test_matmul_nan_stays_in_its_row_and_column():
    x, y = matrix(300, 256, FP32, 31, 0.5), matrix(260, 256, FP32, 32, 0.5)
    x[299, 3] = math.nan
    y[7, 200] = math.inf
    a, b = nsa.f8_quantize_batched([x.cuda()]), nsa.f8_quantize_batched([y.cuda()])
    (c,) = nsa.f8_matmul_batched(a, b, out_dtype=FP32)
    bad = torch.isnan(c).cpu()
    want = torch.zeros(300, 260, dtype=torch.bool)
    want[299] = True
    want[:, 7] = True
    assert torch.equal(bad, want)


def test_operand_and_transpose_of_weights_hold_the_same_values():
    w = matrix(300, 515, BF16, 41)
    (o,), (t,) = nsa.f8_quantize_batched([w.cuda()], block_rows=128, transpose=True)
    assert np.array_equal(values(o)[:, :515], values(t)[:, :300].T)


def test_backward_products_against_the_formula_and_differences():
    """Y = X W^T with the loss <dY, Y>: dX = dY W and dW = dY^T X over the
    operands' values, against the formula; and along random directions against
    differences of the loss in 64 bits (it is linear in X and in W, so a
    difference is exact but for its own rounding)."""
    t, n, k = 77, 200, 330
    x, w, dy = (matrix(r, c, BF16, s, 0.5).cuda() for r, c, s in ((t, k, 51), (n, k, 52), (t, n, 53)))
    (xq,), (xt,) = nsa.f8_quantize_batched([x], transpose=True)
    (wq,), (wt,) = nsa.f8_quantize_batched([w], block_rows=128, transpose=True)
    (dq,), (dt,) = nsa.f8_quantize_batched([dy], transpose=True)
    (y,) = nsa.f8_matmul_batched([xq], [wq], out_dtype=FP32)
    (dx,) = nsa.f8_matmul_batched([dq], [wt], out_dtype=FP32)
    (dw,) = nsa.f8_matmul_batched([dt], [xt], out_dtype=FP32)
    check_product(y, xq, wq, what="forward")
    check_product(dx, dq, wt, what="dX")
    check_product(dw, dt, xt, what="dW")
    rng = np.random.default_rng(5)

    def loss(d, xv, wv):
        return float(np.sum(d * (xv @ wv.T)))

    dv, wv, xv = values(dq)[:, :n], values(wq)[:, :k], values(xq)[:, :k]
    dtv, xtv = values(dt)[:, :t].T, values(xt)[:, :t].T
    for _ in range(4):
        u = rng.standard_normal(xv.shape)
        diff = (loss(dv, xv + 0.5 * u, wv) - loss(dv, xv - 0.5 * u, wv))
        got = float(np.sum(host_f64(dx) * u))
        bound = n * 2.0 ** -23 * float(np.sum((np.abs(dv) @ np.abs(wv)) * np.abs(u))) + 1e-9 * abs(loss(dv, xv, wv))
        assert abs(got - diff) <= bound, (got, diff, bound)
        u = rng.standard_normal(wv.shape)
        diff = (loss(dtv, xtv, wv + 0.5 * u) - loss(dtv, xtv, wv - 0.5 * u))
        got = float(np.sum(host_f64(dw) * u))
        bound = 128 * 2.0 ** -23 * float(np.sum((np.abs(dtv).T @ np.abs(xtv)) * np.abs(u))) + 1e-9 * abs(loss(dtv, xtv, wv))
        assert abs(got - diff) <= bound, (got, diff, bound)


def test_weight_gradient_sums_over_micro_batches():
    n, k = 130, 260
    dw = torch.zeros((n, k), device="cuda")
    want, tol = np.zeros((n, k)), np.zeros((n, k))
    for step, t in enumerate((100, 0, 257)):
        x, dy = matrix(t, k, BF16, 60 + step, 0.5).cuda(), matrix(t, n, BF16, 70 + step, 0.5).cuda()
        xt = nsa.f8_quantize_batched([x], normal=False, transpose=True)
        dt = nsa.f8_quantize_batched([dy], normal=False, transpose=True)
        nsa.f8_matmul_batched(dt, xt, out=[dw], accumulate=True)
        a, b = values(dt[0]), values(xt[0])
        want += a @ b.T
        tol += a.shape[1] * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T)
        tol += 2.0 ** -24 * 2 * np.abs(want)
    assert np.all(np.abs(host_f64(dw) - want) <= tol + 1e-38)


def test_streams_batches_and_repeats():
    shapes = [(40 + 3 * i, 64 + 8 * (i % 5), 200) for i in range(70)]  # a table of several pieces
    a, b = operands(shapes, 400)
    first = nsa.f8_matmul_batched(a, b)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        second = nsa.f8_matmul_batched(a, b)
    third = nsa.f8_matmul_batched(a, b)  # at the same time, with a workspace of its own
    torch.cuda.synchronize()
    for i, s in enumerate(shapes):
        assert torch.equal(first[i], second[i]) and torch.equal(first[i], third[i])
        if i % 10 == 0:
            check_product(first[i], a[i], b[i], what=s)


def test_capture_and_replay():
    xs = [matrix(r, 300, BF16, 500 + r, 0.5).cuda() for r in (20, 150, 0, 64)]
    ws = [matrix(260, 300, BF16, 600 + i, 0.5).cuda() for i in range(4)]
    wq = nsa.f8_quantize_batched(ws, block_rows=128)

    def forward():
        return nsa.f8_matmul_batched(nsa.f8_quantize_batched(xs), wq)

    forward()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = forward()
    for k in range(4):
        for x in xs:
            x.mul_(-1.5)
        want = forward()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want)), k


def test_a_training_step_of_two_experts():
    """All of it as a training loop has it: quantized weights and tokens, the
    forward product, both backward products over two micro-batches, the clip
    into bf16 gradients, the Muon step on them, the weights quantized again.
    Each part is held to 64-bit arithmetic on what the part before it gave."""
    n, k = 130, 264
    ws = [(matrix(n, k, BF16, 700 + e, 0.0).float() * 0.05).to(BF16).cuda() for e in range(2)]
    ms = [torch.zeros_like(w) for w in ws]
    dws = [torch.zeros((n, k), device="cuda") for _ in ws]
    wq, wt = nsa.f8_quantize_batched(ws, block_rows=128, transpose=True)
    for mb, tokens in enumerate(((50, 0), (33, 140))):
        xs = [matrix(t, k, BF16, 710 + 10 * mb + e, 0.3).cuda() for e, t in enumerate(tokens)]
        xq, xt = nsa.f8_quantize_batched(xs, transpose=True)
        ys = nsa.f8_matmul_batched(xq, wq)
        dys = [(y.float() - 0.1).to(BF16) for y in ys]  # of the loss sum (y - 0.1)^2 / 2
        dq, dt = nsa.f8_quantize_batched(dys, transpose=True)
        dxs = nsa.f8_matmul_batched(dq, wt)
        old = [host_f64(d) for d in dws]
        nsa.f8_matmul_batched(dt, xt, out=dws, accumulate=True)
        for e in range(2):
            check_product(ys[e], xq[e], wq[e], what="y")
            check_product(dxs[e], dq[e], wt[e], what="dx")
            check_product(dws[e], dt[e], xt[e], old[e], what="dw")
    gs = [torch.empty_like(w) for w in ws]
    r = nsa.grad_clip_batched(dws, 0.5, out=gs)
    norm = math.sqrt(sum(float(np.sum(host_f64(d) ** 2)) for d in dws))
    assert abs(float(r[0]) - norm) <= 2.0 ** -23 * norm
    for d, g in zip(dws, gs):
        assert torch.equal(g.cpu(), (d.cpu() * r[1].cpu()).to(BF16))
    ref_w, ref_m = [w.clone() for w in ws], [m.clone() for m in ms]
    nsa.step_batched(ref_w, gs, ref_m)  # the step on the clipped gradients is the plain step
    nsa.step_batched(ws, gs, ms, grad_scale=torch.ones(1, device="cuda"))
    assert all(torch.equal(a, b) for a, b in zip(ws + ms, ref_w + ref_m))
    again = nsa.f8_quantize_batched(ws, block_rows=128, out=wq)
    assert again[0][0] is wq[0].q
    for w, o in zip(ws, again):
        check_operand(o, host_f64(w), 128, "weights after the step")


def test_new_outputs_are_ordinary_tensors():
    # pieces of one allocation: shapes, neighbours, in-place work, gradients, lifetime
    xs = [matrix(r, c, BF16, 40 + r, 1.0).cuda() for r, c in ((3, 130), (0, 40), (70, 300), (20, 0))]
    ops, ops_t = nsa.f8_quantize_batched(xs, transpose=True)
    for x, o, t in zip(xs, ops, ops_t):
        r, c = x.shape
        assert o.q.dtype == torch.float8_e4m3fn and o.scales.dtype == torch.uint8
        assert o.q.shape == (r, up(c, BLOCK)) and o.scales.shape == (up(c, BLOCK) // BLOCK, up(r, 16))
        assert t.q.shape == (c, up(r, BLOCK)) and t.scales.shape == (up(r, BLOCK) // BLOCK, up(c, 16))
        for y in (*o, *t):
            assert y.is_contiguous() and y.device == x.device and not y.requires_grad
            assert y.numel() == 0 or y.data_ptr() % 16 == 0
    c = nsa.f8_matmul_batched(ops, ops, out_dtype=FP32)
    assert [tuple(y.shape) for y in c] == [(3, 3), (0, 0), (70, 70), (20, 20)]
    kept = [y.clone() for y in c]
    c[2].mul_(2)
    assert torch.equal(c[2], 2 * kept[2]) and torch.equal(c[0], kept[0]) and torch.equal(c[3], kept[3])
    w = c[2].requires_grad_()
    (w * w).sum().backward()
    assert torch.equal(w.grad, 2 * w.detach())
    last = c[3]
    del c, w
    torch.cuda.synchronize()
    junk = [torch.full((1 << 16,), 9.0, device="cuda") for _ in range(8)]
    assert torch.equal(last, kept[3]) and len(junk) == 8


def test_binding_refusals_on_the_gpu():
    a, b = operands([(5, 6, 200)], 900)
    with pytest.raises(ValueError):
        nsa.f8_matmul_batched(a, nsa.f8_quantize_batched([matrix(6, 300, FP32, 1).cuda()]))
    with pytest.raises(ValueError):
        nsa.f8_matmul_batched(a, b, out=[torch.zeros(6, 5, device="cuda")])
    with pytest.raises(TypeError):
        nsa.f8_matmul_batched(a, b, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        nsa.f8_matmul_batched([(a[0].q, a[0].scales[:, :8])], b)
    with pytest.raises(ValueError):
        nsa.f8_matmul_batched([(a[0].q[:, :128], a[0].scales)], b)
    with pytest.raises(TypeError):
        nsa.f8_matmul_batched([(a[0].q.view(torch.uint8), a[0].scales)], b)
    with pytest.raises(ValueError):
        nsa.f8_quantize_batched([torch.zeros(5, 300, device="cuda")], out=[nsa.f8_empty(6, 300, "cuda")])
    with pytest.raises(ValueError):
        nsa.f8_quantize_batched([torch.zeros(300, 5, device="cuda").t()])
    with pytest.raises(nsa.MuonError):
        nsa.f8_quantize_batched([torch.zeros(5, 300, device="cuda")], block_rows=64)
