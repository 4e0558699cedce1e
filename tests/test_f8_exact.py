"""Products of block-scaled e4m3 operands that are exact, bit for bit.

Values are 0, +-1 and +-2, scales 1, 2 and 4: the products of a block lie within two
binades of each other, far inside the window in which the e4m3 matrix instruction adds
8 of them, and every partial sum is an integer below 2^24.  Whatever the order of the
sum, fp32 holds it, so both output types have one right answer: the integer, rounded
once.  One lost, doubled or misplaced product shows.

On the CPU: the shapes reach every kernel and tile size (tests/host/f8_plan_show.cpp,
compiled host-only against the library's ABI source, says what each call takes)."""
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import newton_schulz_03_amd as nsa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "newton_schulz_03_amd", "csrc")
BF16, FP32 = torch.bfloat16, torch.float32
BLOCK = 128

CASES = {
    # the kernel of few rows, every block shape
    "16 rows, 16 columns": [(5, 200, 300)],
    "16 rows, 32 columns": [(5, 3901, 700)],
    "16 rows, 64 columns": [(9, 7000, 1100)],
    "32 rows, 16 columns": [(20, 201, 129)],
    "32 rows, 32 columns": [(20, 3900, 6144)],
    "32 rows, 64 columns": [(31, 7001, 1100)],
    "64 rows, 16 columns": [(50, 200, 1), (200, 136, 1280), (64, 33, 4096)],
    "64 rows, 32 columns": [(64, 3900, 700)],
    "64 rows, 64 columns": [(50, 7002, 700)],
    "few rows, lengths that differ": [(16, 2000, k) for k in (130, 256, 4000, 300, 2000, 0, 700)],
    "few rows, many products": [(1 + i % 9, 520, 256 + 128 * (i % 7)) for i in range(60)],
    # tiles of 256, 128 and 64 rows
    "whole tiles": [(16384, 2048, 640)],
    "quarter tiles": [(2048, 2048, 2048)],
    "half tiles": [(2048, 2303, 1100)],
    "whole and half tiles": [(4196, 2304, 300)],
    "whole and quarter tiles": [(4197, 4094, 640)],
    "tiles of all kinds": [(4196, 1101, 2048), (2100, 2303, 2048)],
    "tiles of all kinds, dealt": [(2100, 4096, 4000), (356, 2304, 4000), (8, 64, 6144)],
    "tiles dealt over the chip": [(1290, 1500, k) for k in (130, 256, 4000, 300, 2000, 0, 700)],
    "long sums": [(700, 2100, 6144)] * 4,
    "one block, two, three": [(1290, 1500, k) for k in (1, 129, 300, 400, 513, 700)],
    "rests of rows": [(2048 + r, 1100, 500 + r) for r in (1, 20, 64, 65, 100, 128, 150, 192, 193, 255)],
    # both kernels
    "quarter tiles and few rows": [(2048, 2048, 2048), (8, 64, 3000)],
    "half tiles and few rows": [(2048, 4096, 300), (8, 2048, 6144), (8, 2047, 6144)],
    "whole tiles and few rows": [(2048, 4096, 300), (2048, 1100, 300), (1, 2048, 6144)],
    "all tiles and few rows": [(4196, 2048, 640), (2100, 2304, 640), (64, 64, 6144)],
    # outputs that pass the caches by
    "past the caches": [(8300, 16400, 200)],
}


@pytest.mark.skipif(shutil.which("hipcc") is None, reason="hipcc not found")
def test_the_cases_reach_every_kernel_and_tile(tmp_path):
    exe = tmp_path / "f8_plan_show"
    build = subprocess.run(
        ["hipcc", "--offload-host-only", "-x", "hip", "-O1", "-std=c++17",
         "-I", os.path.join(ROOT, "include"), "-I", CSRC,
         os.path.join(ROOT, "tests", "host", "f8_plan_show.cpp"), "-o", str(exe)],
        capture_output=True, text=True, timeout=300)
    assert build.returncode == 0, build.stderr[-3000:]
    for dtype in "01":
        seen = set()
        for shapes in CASES.values():
            args = [dtype, "0"] + [str(x) for s in shapes for x in s]
            run = subprocess.run([str(exe)] + args, capture_output=True, text=True, timeout=60)
            assert run.returncode == 0, run.stderr
            full, half, quarter, spread, nt, blocks, mt, wide, dealt = (int(x) for x in run.stdout.split())
            tiles = [k for k, n in (("full", full), ("half", half), ("quarter", quarter)) if n]
            seen.update(tiles)
            if spread:
                seen.update("dealt " + k for k in tiles)
            if nt:
                seen.add("past the caches")
            if blocks:
                seen.add((mt, wide))
                if dealt:
                    seen.add("dealt blocks")
                if tiles:
                    seen.update("blocks and " + k for k in tiles)
        want = {"full", "half", "quarter", "dealt full", "dealt quarter", "past the caches",
                "dealt blocks", "blocks and full", "blocks and half", "blocks and quarter"}
        want |= {(mt, nt) for mt in (1, 2, 4) for nt in (1, 2, 4)}
        assert want <= seen, want - seen


def up(x, a):
    return (x + a - 1) // a * a


def operand(rows, k, gen):
    """An operand of rows x k on the device, and what it stands for (float32, exact)."""
    kp, rp = up(k, BLOCK), up(rows, 16)
    v = torch.randint(-2, 3, (rows, k), generator=gen, device="cuda").float()
    v = torch.nn.functional.pad(v, (0, kp - k))
    e = torch.randint(0, 3, (kp // BLOCK, rows), generator=gen, device="cuda")
    s = torch.zeros((kp // BLOCK, rp), dtype=torch.uint8, device="cuda")
    s[:, :rows] = (e + 127).to(torch.uint8)
    x = (v.view(rows, kp // BLOCK, BLOCK) * torch.exp2(e.t().float())[:, :, None]).view(rows, kp)
    return (v.to(torch.float8_e4m3fn), s), x


@pytest.mark.gpu
@pytest.mark.parametrize("out", [BF16, FP32])
@pytest.mark.parametrize("name", CASES)
def test_exact_products(name, out):
    print(f"\n[gpu-test] {name} {out}", flush=True)
    shapes = CASES[name]
    gen = torch.Generator(device="cuda").manual_seed(len(name) + len(shapes))
    a, x = zip(*(operand(m, k, gen) for m, n, k in shapes))
    b, y = zip(*(operand(n, k, gen) for m, n, k in shapes))
    want = []
    for p, q in zip(x, y):
        # a sum of at most 6144 products of at most 4 * 16
        assert p.shape[1] * 64 < 1 << 24
        want.append((p.double() @ q.double().t().contiguous()).float())
    got = nsa.f8_matmul_batched(a, b, out_dtype=out)
    torch.cuda.synchronize()
    for s, c, w in zip(shapes, got, want):
        assert bool((c == w.to(out)).all()), s
    old = [torch.randint(-64, 65, tuple(w.shape), generator=gen, device="cuda").float() for w in want]
    into = [o.clone().to(out) for o in old]
    del got
    nsa.f8_matmul_batched(a, b, out=into, accumulate=True)
    torch.cuda.synchronize()
    for s, c, w, o in zip(shapes, into, want, old):
        assert bool((c == (w + o).to(out)).all()), s


@pytest.mark.gpu
@pytest.mark.parametrize("m,n", [(48, 40), (2048, 2304)])  # few rows; tiles
@pytest.mark.parametrize("out", [BF16, FP32])
def test_each_k_counts_once(m, n, out):
    """Row r of A holds a single 1, at column r % k: the product is column r % k of B,
    scales included, in every row and column of the result."""
    gen = torch.Generator(device="cuda").manual_seed(m)
    k = 384
    at = torch.arange(m, device="cuda") % k
    v = torch.zeros((m, k), device="cuda")
    v[torch.arange(m, device="cuda"), at] = 1
    s = torch.zeros((k // BLOCK, up(m, 16)), dtype=torch.uint8, device="cuda")
    s[:, :m] = 127
    b, y = operand(n, k, gen)
    (c,) = nsa.f8_matmul_batched([(v.to(torch.float8_e4m3fn), s)], [b], out_dtype=out)
    assert bool((c == y[:, at].t().to(out)).all())


@pytest.mark.gpu
@pytest.mark.parametrize("m,n", [(300, 260), (2048, 2304)])  # few rows; tiles
@pytest.mark.parametrize("out", [BF16, FP32])
def test_nan_stays_in_its_row_and_column(m, n, out):
    gen = torch.Generator(device="cuda").manual_seed(n)
    (qa, sa), x = operand(m, 300, gen)
    (qb, sb), y = operand(n, 300, gen)
    qa.view(torch.uint8)[m - 1, 3] = 0x7f
    qb.view(torch.uint8)[7, 299] = 0xff
    (c,) = nsa.f8_matmul_batched([(qa, sa)], [(qb, sb)], out_dtype=out)
    want = (x.double() @ y.double().t().contiguous()).to(out)
    want[m - 1], want[:, 7] = float("nan"), float("nan")
    assert np.array_equal(c.float().cpu().numpy(), want.float().cpu().numpy(), equal_nan=True)


def column_scales(n):
    """Exponents that differ by row of B, and the scale bytes of its one block."""
    e = torch.tensor([-100, -60, -20, 0, 20, 60, 100], device="cuda")[torch.arange(n, device="cuda") % 7]
    s = torch.zeros((1, up(n, 16)), dtype=torch.uint8, device="cuda")
    s[0, :n] = (e + 127).to(torch.uint8)
    return e, s


@pytest.mark.gpu
@pytest.mark.parametrize("m,n", [(255, 70), (2048, 2304)])  # few rows; tiles
@pytest.mark.parametrize("out", [BF16, FP32])
def test_every_scale_byte(m, n, out):
    """Each scale byte 0 .. 254 in some row of A, against scales of 2^-100 to 2^100 in B:
    exact wherever 2^-126 <= 2^(e + f), 512 * 2^(e + f) < 2^127 (the sum of 128 products
    of at most 4) and, for fp32 results, the operand's values are below 2^128."""
    gen = torch.Generator(device="cuda").manual_seed(m)
    v = torch.randint(-2, 3, (m, BLOCK), generator=gen, device="cuda").float()
    w = torch.randint(-2, 3, (n, BLOCK), generator=gen, device="cuda").float()
    byte = torch.arange(m, device="cuda") % 255
    s = torch.zeros((1, up(m, 16)), dtype=torch.uint8, device="cuda")
    s[0, :m] = byte.to(torch.uint8)
    f, t = column_scales(n)
    (c,) = nsa.f8_matmul_batched([(v.to(torch.float8_e4m3fn), s)], [(w.to(torch.float8_e4m3fn), t)],
                                 out_dtype=out)
    e = (byte - 127)[:, None] + f[None, :]
    held = (e >= -126) & (e + 9 < 127)
    if out == FP32:
        held &= (byte < 254)[:, None]
    want = (v.double() @ w.double().t().contiguous()) * torch.exp2(e.double())
    assert int(held.sum()) > m * n // 2
    assert bool((c.double() == want)[held].all())


@pytest.mark.gpu
@pytest.mark.parametrize("m,n", [(40, 70), (2048, 2304)])  # few rows; tiles
def test_magnitudes_next_to_the_largest_fp32_value(m, n):
    """248 * 2^120 = 3.3e38 and above round up to the operand value 2^128.  The scaled
    instruction of bf16 results takes it; fp32 results take operands as fp32 holds them,
    so there it is infinite.  No other row notices."""
    x = torch.ones((m, BLOCK), device="cuda")
    x[3] = 0
    x[3, 5] = 3.4e38
    x[7, 9] = -248.0 * 2.0 ** 120
    x[7, :9] = 0
    x[7, 10:] = 0
    x[8] = 0
    x[8, 1] = 247.0 * 2.0 ** 120  # rounds down, to 240 * 2^120
    (a,) = nsa.f8_quantize_batched([x])
    assert a.scales[0, [3, 7, 8]].tolist() == [247] * 3
    assert a.q.float()[[3, 7, 8], [5, 9, 1]].tolist() == [256.0, -256.0, 240.0]
    gen = torch.Generator(device="cuda").manual_seed(n)
    w = torch.randint(1, 3, (n, BLOCK), generator=gen, device="cuda").float()
    t = torch.zeros((1, up(n, 16)), dtype=torch.uint8, device="cuda")
    t[0, :n] = 127 - 20
    b = (w.to(torch.float8_e4m3fn), t)
    stands = x.double()
    stands[3, 5], stands[7, 9], stands[8, 1] = 2.0 ** 128, -2.0 ** 128, 240 * 2.0 ** 120
    want = (stands @ w.double().t().contiguous()) * 2.0 ** -20
    (c,) = nsa.f8_matmul_batched([a], [b], out_dtype=BF16)
    assert bool((c.double() == want.float().to(BF16).double()).all())
    (c,) = nsa.f8_matmul_batched([a], [b], out_dtype=FP32)
    assert not bool(torch.isfinite(c[[3, 7]]).any())
    rest = torch.ones(m, dtype=torch.bool, device="cuda")
    rest[3] = rest[7] = False
    assert bool((c.double() == want)[rest].all())
