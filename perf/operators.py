"""Operators around the optimizer step, measured against their plain forms.

  norm      the global norm of a ragged batch of gradients, and the clip factor
  clip      the same, and the gradients times that factor
  adamw     the AdamW step on gradients that take the clip factor as they are read
  quantize  block-scaled e4m3 operands of a batch of matrices: one power-of-two
            scale per 1 x 128 or 128 x 128 block, for the matrix, its transpose
            or both
  matmul    C_i = A_i B_i^T over such operands, ragged over experts

Gradients lie in one flat bucket, every tensor at a 16-byte boundary, as data-
parallel training keeps them; the plain forms work on the whole bucket (the
gaps hold zeros) and the framework's calls on the list of tensors.
"""
import math
import random

import torch

own = False

HIDDEN, FFN, EXPERTS, LAYERS = 6144, 2048, 384, 74
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
NONEXPERT = [HIDDEN, HIDDEN, EXPERTS * HIDDEN] * LAYERS + [HIDDEN]
RAGGED = [1, 7, 8, 9, 255, 8191, 8192, 8193, 100003, 0, 24581]


def listed():
    return [
        # the gradient of one norm weight: the smallest call, all latency
        {"name": "norm, one weight", "op": "norm", "set": "one", "dtype": "bf16", "kind": "l2"},
        # every parameter that Muon does not cover: two norm weights and a router per layer
        {"name": "norm, non-expert", "op": "norm", "set": "nonexpert", "dtype": "bf16", "kind": "l2"},
        # one rank's expert gradients as fp32 sums over micro-batches
        {"name": "norm, experts fp32", "op": "norm", "set": "experts48", "dtype": "fp32", "kind": "l2"},
        # a small model's ragged parameters, odd sizes and an empty one
        {"name": "clip, ragged", "op": "clip", "set": "ragged", "dtype": "fp32", "out": "fp32", "kind": "l2"},
        # fp32 sums of expert gradients, clipped into the bf16 gradients that the step reads
        {"name": "clip, experts to bf16", "op": "clip", "set": "experts24", "dtype": "fp32", "out": "bf16", "kind": "l2"},
        # fp32 parameters of odd sizes
        {"name": "adamw, ragged", "op": "adamw", "set": "ragged", "dtype": "fp32"},
        # the model's non-expert parameters
        {"name": "adamw, non-expert", "op": "adamw", "set": "nonexpert", "dtype": "bf16"},
        # the tokens of 32 experts, for the forward product and the weight gradient
        {"name": "quantize, tokens", "op": "quantize", "batch": 32, "rows": 256, "spread": 255, "shape_seed": 3,
         "cols": HIDDEN, "dtype": "bf16", "block_rows": 1, "normal": True, "transpose": True},
        # expert weights after the step, for the forward product and the input gradient
        {"name": "quantize, weights", "op": "quantize", "batch": 16, "rows": FFN, "spread": 0, "shape_seed": 0,
         "cols": HIDDEN, "dtype": "bf16", "block_rows": 128, "normal": True, "transpose": True},
        # a few tokens for each expert: the weights' bytes bound it
        {"name": "matmul, few tokens", "op": "matmul", "batch": 32, "m": 4, "spread": 4, "shape_seed": 1,
         "n": FFN, "k": HIDDEN, "ragged": "m", "out": "bf16", "accumulate": False},
        # the up projection of 16 experts over their tokens
        {"name": "matmul, forward", "op": "matmul", "batch": 16, "m": 1024, "spread": 500, "shape_seed": 2,
         "n": FFN, "k": HIDDEN, "ragged": "m", "out": "bf16", "accumulate": False},
        # the weight gradient of 8 experts, summed in fp32 over micro-batches
        {"name": "matmul, weight gradient", "op": "matmul", "batch": 8, "m": FFN, "spread": 1000, "shape_seed": 4,
         "n": HIDDEN, "k": 4000, "ragged": "k", "out": "fp32", "accumulate": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["norm", "clip", "adamw", "quantize", "matmul"])
    seed = rng.randrange(1 << 30)
    if op in ("norm", "clip", "adamw"):
        case = {"op": op, "set": "drawn", "tensors": _log(rng, 1, 300),
                "elements": _log(rng, 1000, 150_000_000), "shape_seed": seed,
                "dtype": rng.choice(["bf16", "fp32"])}
        if op != "adamw":
            case["kind"] = rng.choice(["l2", "l2", "max"])
        if op == "clip":
            case["out"] = rng.choice(["bf16", "fp32"])
        return case
    if op == "quantize":
        rows = _log(rng, 1, 4096)
        cols = _log(rng, 16, 8192)
        batch = min(_log(rng, 1, 64), max(1, 190_000_000 // (rows * cols)))
        normal, transpose = rng.choice([(True, False), (False, True), (True, True)])
        return {"op": op, "batch": batch, "rows": rows, "spread": rng.choice([0, rows // 2]), "shape_seed": seed,
                "cols": cols, "dtype": rng.choice(["bf16", "fp32"]), "block_rows": rng.choice([1, 128]),
                "normal": normal, "transpose": transpose}
    m, n, k = _log(rng, 1, 4096), _log(rng, 16, 8192), _log(rng, 16, 8192)
    batch = min(_log(rng, 1, 64), max(1, 190_000_000_000 // (m * n * k)), max(1, 400_000_000 // (n * k)))
    ragged = rng.choice(["m", "k"])
    return {"op": op, "batch": batch, "m": m, "spread": (m if ragged == "m" else k) // 2, "shape_seed": seed,
            "n": n, "k": k, "ragged": ragged, "out": rng.choice(["bf16", "fp32"]), "accumulate": rng.random() < 0.3}


# ---------------------------------------------------------------------------
# Sizes
# ---------------------------------------------------------------------------

def _numels(case):
    if case["set"] == "one":
        return [HIDDEN]
    if case["set"] == "nonexpert":
        return list(NONEXPERT)
    if case["set"].startswith("experts"):
        return [FFN * HIDDEN] * int(case["set"][len("experts"):])
    if case["set"] == "ragged":
        return list(RAGGED)
    r = random.Random(case["shape_seed"])
    w = [r.random() ** 3 + 1e-6 for _ in range(case["tensors"])]
    return [max(1, int(case["elements"] * x / sum(w))) for x in w]


def _around(case, base):
    """`base` give or take `spread` for each of the batch; where it may reach 0, one of them is 0."""
    r = random.Random(case["shape_seed"])
    got = [max(0, base + r.randint(-case["spread"], case["spread"])) for _ in range(case["batch"])]
    if case["spread"] >= base and case["batch"] > 1:
        got[-1] = 0
    return got


def _shapes(case):
    """(m, n, k) of each product."""
    if case["ragged"] == "m":
        return [(m, case["n"], case["k"]) for m in _around(case, case["m"])]
    return [(case["m"], case["n"], k) for k in _around(case, case["k"])]


def _up(x, a):
    return (x + a - 1) // a * a


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _bucket(numels, dtype, fill):
    """A flat bucket and its tensors, each at a multiple of 8 elements; the gaps hold zeros."""
    offs, total = [], 0
    for n in numels:
        offs.append(total)
        total += _up(n, 8)
    flat = fill(total).to(dtype)
    gaps = [(o + n, o + _up(n, 8)) for o, n in zip(offs, numels) if n % 8]
    for a, b in gaps:
        flat[a:b] = 0
    return flat, [flat[o:o + n] for o, n in zip(offs, numels)]


def _e4m3(x, block_rows):
    """Plain e4m3 operand of x (R x K, contracted over its columns): the values
    (R x Kp, Kp = K up to a multiple of 128, zeros there) and the scale bytes
    (Kp/128 x R up to a multiple of 16, zeros there).  A block's scale 2^e is the
    smallest power of two, at least 2^-127, with its largest finite magnitude
    at most 448 * 2^e; what is not finite becomes NaN."""
    r, k = x.shape
    kp, rp = _up(k, 128), _up(r, 16)
    v = torch.zeros((_up(r, block_rows), kp), dtype=torch.float32, device=x.device)
    v[:r, :k] = x.float()
    blocks = v.view(v.shape[0] // block_rows, block_rows, kp // 128, 128)
    mag = torch.where(torch.isfinite(blocks), blocks.abs(), torch.zeros_like(blocks)).amax(dim=(1, 3))
    _, ex = torch.frexp(mag)  # mag = f * 2^ex, 1/2 <= f < 1; 448 = 7/8 * 2^9
    mag_f = torch.ldexp(mag.double(), -ex)
    e = (ex - 9 + (mag_f > 0.875).int()).clamp(min=-127)
    e = torch.where(mag > 0, e, torch.full_like(e, -127))
    # 2^-e in two factors, each a normal number
    h = torch.div(-e, 2, rounding_mode="floor")
    inv = [torch.ldexp(torch.ones_like(mag), p)[:, None, :, None] for p in (h, -e - h)]
    s = blocks * inv[0] * inv[1]
    s = torch.where(torch.isfinite(s), s, torch.full_like(s, math.nan))
    q = s.view(v.shape)[:r].to(torch.float8_e4m3fn)
    scales = torch.zeros((kp // 128, rp), dtype=torch.uint8, device=x.device)
    scales[:, :r] = (e + 127).to(torch.uint8).repeat_interleave(block_rows, 0)[:r].t()
    return q, scales


def _value(q, scales, dtype=torch.float32):
    """The values that an operand stands for."""
    r, kp = q.shape
    p = torch.ldexp(torch.ones((), dtype=torch.float64, device=q.device), scales[:, :r].t().int() - 127).to(dtype)
    return (q.to(dtype).view(r, kp // 128, 128) * p[:, :, None]).view(r, kp)


def _room(shapes, dev, whole):
    """Buffers for the operands of (rows, contracted) shapes, as views of two allocations."""
    qs = [(r, _up(k, 128)) for r, k in shapes]
    ss = [(_up(k, 128) // 128, _up(r, 16)) for r, k in shapes]
    got = []
    for sizes, dtype in ((qs, torch.float8_e4m3fn), (ss, torch.uint8)):
        flat = torch.zeros(sum(a * b for a, b in sizes), dtype=torch.uint8, device=dev).view(dtype)
        whole.append(flat)
        got.append([p.view(s) for p, s in zip(flat.split([a * b for a, b in sizes]), sizes)])
    return list(zip(*got))


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(shape, std, dtype=torch.float32):
        return torch.empty(shape, dtype=torch.float32, device=dev).normal_(0.0, std, generator=gen).to(dtype)

    st = {"case": case}
    if case["op"] in ("norm", "clip", "adamw"):
        numels, dt = _numels(case), DTYPES[case["dtype"]]
        st["flat"], st["grads"] = _bucket(numels, dt, lambda n: normal(n, 1e-3))
        if case["op"] != "adamw":
            # half of the gradients' expected norm (l2) or largest magnitude (max): the clip is active
            st["max_norm"] = 0.5e-3 * math.sqrt(max(1, sum(numels))) if case["kind"] == "l2" else 1e-3
            st["norm_type"] = 2.0 if case["kind"] == "l2" else math.inf
        if case["op"] == "clip":
            st["out"], st["outs"] = _bucket(numels, DTYPES[case["out"]],
                                            lambda n: torch.zeros(n, device=dev))
        if case["op"] == "adamw":
            st["p"], st["ps"] = _bucket(numels, dt, lambda n: normal(n, 0.02))
            st["m"], st["ms"] = _bucket(numels, torch.float32, lambda n: normal(n, 1e-3))
            st["v"], st["vs"] = _bucket(numels, torch.float32, lambda n: normal(n, 1e-3).square_())
            st["scale"] = torch.empty(1, device=dev).uniform_(0.2, 0.9, generator=gen)
            st["hyper"] = dict(lr=1e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1, step=10)
        return st
    if case["op"] == "quantize":
        # rows of different size, as tokens and output channels have
        st["xs"] = [normal((r, case["cols"]), 1.0).mul_(torch.exp(normal((r, 1), 1.0))).to(DTYPES[case["dtype"]])
                    for r in _around(case, case["rows"])]
        # the operands' buffers, kept from step to step: all values of a batch in
        # one allocation, all scales in another
        st["whole"] = []
        st["out"] = _room([tuple(x.shape) for x in st["xs"]], dev, st["whole"]) if case["normal"] else None
        st["out_t"] = _room([tuple(x.shape[::-1]) for x in st["xs"]], dev, st["whole"]) if case["transpose"] else None
        return st
    shapes = _shapes(case)
    b_rows = 128 if case["ragged"] == "m" else 1  # the second operand: weights, in 128 x 128 blocks, or tokens
    st["a"] = [_e4m3(normal((m, k), 1.0), 1) for m, n, k in shapes]
    st["b"] = [_e4m3(normal((n, k), 0.02), b_rows) for m, n, k in shapes]
    st["c"] = [normal((m, n), 1.0, DTYPES[case["out"]]) for m, n, k in shapes]
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(st):
    return globals()["_run_" + st["case"]["op"]](st)


def _plain_norm(flat, st):
    x = flat.float()
    if st["norm_type"] == math.inf:
        n = x.abs().amax()
    else:
        n = (x * x).sum(dtype=torch.float64).sqrt().float()
    return torch.stack([n, torch.clamp(st["max_norm"] / (n + 1e-6), max=1.0)])


def _run_norm(st):
    if own:
        import newton_schulz_03_amd as nsa
        return nsa.grad_norm_batched(st["grads"], max_norm=st["max_norm"], norm_type=st["norm_type"])
    return _plain_norm(st["flat"], st)


def _run_clip(st):
    if own:
        import newton_schulz_03_amd as nsa
        r = nsa.grad_clip_batched(st["grads"], st["max_norm"], norm_type=st["norm_type"], out=st["outs"])
    else:
        r = _plain_norm(st["flat"], st)
        st["out"].copy_(st["flat"].float() * r[1])
    return r, st["out"]


def _run_adamw(st):
    h = st["hyper"]
    if own:
        import newton_schulz_03_amd as nsa
        nsa.adamw_batched(st["ps"], st["grads"], st["ms"], st["vs"], grad_scale=st["scale"], **h)
    else:
        (b1, b2), t = h["betas"], h["step"]
        g = st["flat"].float() * st["scale"]
        p = st["p"].float() * (1 - h["lr"] * h["weight_decay"])
        st["m"].mul_(b1).add_(g * (1 - b1))
        st["v"].mul_(b2).add_(g * g * (1 - b2))
        den = st["v"].sqrt() / math.sqrt(1 - b2 ** t) + h["eps"]
        st["p"].copy_(p - h["lr"] / (1 - b1 ** t) * (st["m"] / den))
    return st["p"], st["m"], st["v"]


def _run_quantize(st):
    c = st["case"]
    if own:
        import newton_schulz_03_amd as nsa
        nsa.f8_quantize_batched(st["xs"], block_rows=c["block_rows"], normal=c["normal"],
                                transpose=c["transpose"], out=st["out"], out_t=st["out_t"])
    else:
        [(o[0].copy_(y[0]), o[1].copy_(y[1])) for x, o in zip(st["xs"], st["out"] or [])
         for y in [_e4m3(x, c["block_rows"])]]
        [(o[0].copy_(y[0]), o[1].copy_(y[1])) for x, o in zip(st["xs"], st["out_t"] or [])
         for y in [_e4m3(x.t(), c["block_rows"])]]
    return st["whole"]


def _run_matmul(st):
    c = st["case"]
    if own:
        import newton_schulz_03_amd as nsa
        nsa.f8_matmul_batched(st["a"], st["b"], out=st["c"], accumulate=c["accumulate"])
    else:
        [o.copy_(y + o.float() if c["accumulate"] else y) for a, b, o in zip(st["a"], st["b"], st["c"])
         for y in [_value(*a) @ _value(*b).t()]]
    return st["c"]


# ---------------------------------------------------------------------------
# What a pass cannot do without, and its result in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] in ("norm", "clip", "adamw"):
        n, e = sum(_numels(case)), 2 if case["dtype"] == "bf16" else 4
        if case["op"] == "norm":
            return {"bytes": n * e + 8, "flops": 2 * n}
        if case["op"] == "clip":
            return {"bytes": n * (e + (2 if case["out"] == "bf16" else 4)) + 8, "flops": 3 * n}
        return {"bytes": n * (3 * e + 16), "flops": 16 * n}
    if case["op"] == "quantize":
        e, byt = 2 if case["dtype"] == "bf16" else 4, 0
        for r in _around(case, case["rows"]):
            c = case["cols"]
            byt += r * c * e
            byt += (r * _up(c, 128) + _up(c, 128) // 128 * r) if case["normal"] else 0
            byt += (c * _up(r, 128) + _up(r, 128) // 128 * c) if case["transpose"] else 0
        return {"bytes": byt, "flops": 0}
    byt = flops = 0
    e = 2 if case["out"] == "bf16" else 4
    for m, n, k in _shapes(case):
        byt += m * n * e * (2 if case["accumulate"] else 1)
        byt += (m + n) * (k + k // 128) if m and k else 0
        flops += 2 * m * n * k
    return {"bytes": byt, "flops": flops}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("norm", "clip"):
        x = st["flat"].double()
        n = torch.linalg.vector_norm(x, ord=st["norm_type"])
        s = torch.minimum(st["max_norm"] / (n + 1e-6), torch.ones_like(n))
        r = torch.stack([n, s])
        return r if case["op"] == "norm" else (r, x.mul_(s))
    if case["op"] == "adamw":
        h = st["hyper"]
        (b1, b2), t = h["betas"], h["step"]
        g = st["flat"].double().mul_(st["scale"].double())
        m = st["m"].double().mul_(b1).add_(g, alpha=1 - b1)
        v = st["v"].double().mul_(b2).addcmul_(g, g, value=1 - b2)
        del g
        upd = (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt_() + h["eps"])
        return st["p"].double().mul_(1 - h["lr"] * h["weight_decay"]).sub_(upd, alpha=h["lr"]), m, v
    if case["op"] == "quantize":
        br = case["block_rows"]

        def one(x):
            r, k = x.shape
            x = torch.nn.functional.pad(x.double(), (0, _up(k, 128) - k, 0, _up(r, br) - r))
            top = torch.nn.functional.max_pool2d(x.abs()[None, None], (br, 128))[0, 0] if x.numel() else \
                x.new_zeros((x.shape[0] // br, x.shape[1] // 128))
            e = torch.ceil(torch.log2(top / 448.0)).clamp(min=-127.0)
            e = e + (top > 448.0 * torch.exp2(e)).double() - (top <= 448.0 * torch.exp2(e - 1)).double()
            e = e.clamp(min=-127.0).repeat_interleave(br, 0)[:r]
            v = (x[:r].view(r, x.shape[1] // 128, 128) * torch.exp2(-e)[:, :, None]).view(r, x.shape[1])
            s = torch.nn.functional.pad((e + 127).t(), (0, _up(r, 16) - r)).to(torch.uint8)
            return v, s

        got = []
        for wanted, xs in ((case["normal"], st["xs"]), (case["transpose"], [x.t() for x in st["xs"]])):
            if wanted:
                vs, ss = zip(*(one(x) for x in xs))
                got += [torch.cat([v.reshape(-1) for v in vs]), torch.cat([s.reshape(-1) for s in ss])]
        return got
    got = []
    for a, b, c in zip(st["a"], st["b"], st["c"]):
        y = _value(*a, dtype=torch.float64) @ _value(*b, dtype=torch.float64).t()
        got.append(y + c.double() if case["accumulate"] else y)
    return got
