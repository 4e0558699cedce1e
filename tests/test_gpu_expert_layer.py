"""The operators of an expert layer one after another, as a program uses them: a
training pass (sort, dispatch, e4m3 products, dropout, combine, and all of their
gradients) and a decode step on 4-bit weights.

Each stage is held to its own definition in 64 bits on what the GPU's previous
stage left, with the bounds of that stage's own tests: copies, masks and
rounded products are equal; e4m3 products lose at most 2^-10 of the sum of
magnitudes (8 products on a common grid of 2^-13 of the largest) with bf16 results and
K 2^-23 with fp32 ones, 4-bit ones K 2^-23, sums of n values n 2^-24, each
then half a step of the type.
"""
import numpy as np
import pytest
import torch

import expert_plain as plain
import newton_schulz_03_amd as nsa
from parity_util import host_f64

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, FP32: 2.0 ** -24}


def values(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).cuda()


def near(got, want, tol):
    assert np.all(np.abs(host_f64(got) - want) <= tol + HALF[got.dtype] * (np.abs(want) + tol))


def value(op, rows, cols):
    """The float64 values of an e4m3 operand."""
    q, s = host_f64(op.q.float()), op.scales.cpu().numpy().astype(np.float64)
    p = np.exp2(s[:, :rows].T - 127)
    return (q.reshape(rows, q.shape[1] // 128, 128) * p[:, :, None]).reshape(q.shape)[:, :cols]


def products(a, b, out):
    """a[i] b[i]^T of e4m3 operands against their values."""
    for x, y, o in zip(a, b, out):
        k = x.q.shape[1]
        u, v = value(x, o.shape[0], k), value(y, o.shape[1], k)
        mag = np.abs(u) @ np.abs(v).T
        near(o, u @ v.T, (2.0 ** -10 if o.dtype == BF16 else k * 2.0 ** -23) * mag)


def test_a_training_pass():
    tokens, top_k, experts, hidden, ffn = 300, 3, 5, 256, 384
    rng = np.random.default_rng(1)
    # a token may name an expert twice, some slots are dropped, one expert has no rows
    ids = rng.choice([0, 1, 2, 4, -1], (tokens, top_k), p=[0.4, 0.2, 0.2, 0.1, 0.1])
    ids = torch.from_numpy(ids.astype(np.int64)).cuda()
    x, gate = values((tokens, hidden), BF16, 1), torch.rand((tokens, top_k), device="cuda")
    up = [values((ffn, hidden), BF16, 10 + e, 0.05) for e in range(experts)]
    down = [values((hidden, ffn), BF16, 20 + e, 0.05) for e in range(experts)]
    dout = values((tokens, hidden), BF16, 2, 1e-2)
    upq, upq_t = nsa.f8_quantize_batched(up, block_rows=128, transpose=True)
    downq, downq_t = nsa.f8_quantize_batched(down, block_rows=128, transpose=True)

    # forward
    plan = nsa.moe_sort(ids, experts)
    want_plan = plain.plan(ids.cpu().numpy(), experts)
    assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(plan, want_plan))
    sizes = plan.sizes()
    n = sum(sizes)
    slots = want_plan[3][:n]
    split = lambda t: list(torch.split(t[:n], sizes))
    xs = nsa.moe_dispatch(x, plan, out=torch.empty((n, hidden), dtype=BF16, device="cuda"))
    assert torch.equal(xs, x[torch.from_numpy(slots // top_k).cuda()])
    xq, xq_t = nsa.f8_quantize_batched(split(xs), transpose=True)
    hs = nsa.f8_matmul_batched(xq, upq)
    products(xq, upq, hs)
    act = [torch.relu(h) for h in hs]
    drop = nsa.dropout_batched(act, 0.25, seed=7, offset=3, out=[torch.empty_like(a) for a in act])
    on = [torch.from_numpy(plain.keep(a.numel(), i, 7, 3, 16384)).view(a.shape).cuda() for i, a in enumerate(act)]
    scale = torch.tensor(np.float32(4 / 3), device="cuda")
    masked = lambda ts: [torch.where(m, t.float() * scale, torch.zeros_like(scale)).to(BF16) for m, t in zip(on, ts)]
    assert all(torch.equal(a, b) for a, b in zip(drop, masked(act)))
    hq, hq_t = nsa.f8_quantize_batched(drop, transpose=True)
    ys = torch.empty((n, hidden), dtype=BF16, device="cuda")
    nsa.f8_matmul_batched(hq, downq, out=split(ys))
    products(hq, downq, split(ys))
    out = nsa.moe_combine(ys, plan, weights=gate)
    sums, mags = np.zeros((tokens, hidden)), np.zeros((tokens, hidden))
    terms = host_f64(ys) * host_f64(gate).ravel()[slots][:, None]
    np.add.at(sums, slots // top_k, terms)
    np.add.at(mags, slots // top_k, np.abs(terms))
    near(out, sums, top_k * 2.0 ** -24 * mags)

    # backward
    dys, dgate = nsa.moe_combine_backward(dout, ys, plan, gate)
    assert torch.equal(dys, (gate.flatten()[torch.from_numpy(slots).cuda()][:, None]
                             * dout.float()[torch.from_numpy(slots // top_k).cuda()]).to(BF16))
    dots = np.zeros(tokens * top_k)
    sizes_ = np.zeros(tokens * top_k)
    pair = host_f64(dout)[slots // top_k] * host_f64(ys)
    dots[slots], sizes_[slots] = pair.sum(1), np.abs(pair).sum(1)
    assert np.all(np.abs(host_f64(dgate).ravel() - dots) <= hidden * 2.0 ** -24 * sizes_)
    dyq, dyq_t = nsa.f8_quantize_batched(split(dys), transpose=True)
    dh = nsa.f8_matmul_batched(dyq, downq_t)
    products(dyq, downq_t, dh)
    ddown = nsa.f8_matmul_batched(dyq_t, hq_t, out_dtype=FP32)
    products(dyq_t, hq_t, ddown)
    dact = nsa.dropout_batched(dh, 0.25, seed=7, offset=3, out=[torch.empty_like(h) for h in dh])
    assert all(torch.equal(a, b) for a, b in zip(dact, masked(dh)))
    dhs = [torch.where(h > 0, d, torch.zeros_like(d)) for h, d in zip(hs, dact)]
    dhq, dhq_t = nsa.f8_quantize_batched(dhs, transpose=True)
    dxs = torch.empty((n, hidden), dtype=BF16, device="cuda")
    nsa.f8_matmul_batched(dhq, upq_t, out=split(dxs))
    products(dhq, upq_t, split(dxs))
    dup = nsa.f8_matmul_batched(dhq_t, xq_t, out_dtype=FP32)
    products(dhq_t, xq_t, dup)
    dx = nsa.moe_combine(dxs, plan)
    sums, mags = np.zeros((tokens, hidden)), np.zeros((tokens, hidden))
    np.add.at(sums, slots // top_k, host_f64(dxs))
    np.add.at(mags, slots // top_k, np.abs(host_f64(dxs)))
    near(dx, sums, top_k * 2.0 ** -24 * mags)

    # the step of the expert without rows sees a zero gradient
    assert not bool(dup[3].any()) and not bool(ddown[3].any())
    norm, factor = nsa.grad_clip_batched(dup + ddown, 1.0).tolist()
    assert norm > 0 and 0 < factor <= 1


@pytest.mark.parametrize("tokens", [1, 6, 50])
def test_a_decode_step(tokens):
    top_k, experts, hidden, ffn = 4, 20, 320, 200
    ids = torch.topk(values((tokens, experts), FP32, tokens), top_k, dim=1).indices
    gate = torch.rand((tokens, top_k), device="cuda")
    x = values((tokens, hidden), BF16, 1)
    # as the step leaves them: up projections stored hidden x ffn
    up = [values((hidden, ffn), BF16, 10 + e, 0.05) for e in range(experts)]
    down = [values((hidden, ffn), BF16, 40 + e, 0.05) for e in range(experts)]
    upq, downq = nsa.f4_quantize(up, transpose=True), nsa.f4_quantize(down)
    plan = nsa.moe_sort(ids, experts)
    h = nsa.f4_matmul(x, upq, plan=plan, gather=True)
    a = torch.nn.functional.silu(h.float()).to(BF16)
    y = nsa.f4_matmul(a, downq, plan=plan, out_dtype=FP32)
    out = nsa.moe_combine(y, plan, weights=gate)

    offsets, _, _, slots = plain.plan(ids.cpu().numpy(), experts)
    for e in range(experts):
        p = slice(offsets[e], offsets[e + 1])
        for got, rows, w in ((h[p], host_f64(x)[slots[p] // top_k], host_f64(up[e]).T),
                             (y[p], host_f64(a)[p], host_f64(down[e]))):
            w = plain.f4_values(*plain.f4(w), w.shape[1])
            mag = np.abs(rows) @ np.abs(w).T
            near(got, rows @ w.T, w.shape[1] * 2.0 ** -23 * mag)
    terms = host_f64(y) * host_f64(gate).ravel()[slots][:, None]
    sums, mags = np.zeros((tokens, hidden)), np.zeros((tokens, hidden))
    np.add.at(sums, slots // top_k, terms)
    np.add.at(mags, slots // top_k, np.abs(terms))
    near(out, sums, top_k * 2.0 ** -24 * mags)
