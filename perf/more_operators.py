"""Operators of the expert layers, measured against their plain forms.

  sort      token slots sorted by expert: the plan that the others read
  dispatch  the plan, and the tokens' rows copied to their sorted places
  combine   the experts' rows back at their tokens, weighted and summed
  backward  the gradient of that: of the rows, and of the weights
  dropout   a ragged batch of tensors, the mask from a counter-based generator
  product   rows times matrices of 4-bit weights with group scales, each expert's
            rows with its own matrix, or all rows with one

Experts are chosen by scores that favour some of them; a share of the slots may
be dropped (an id of -1), as a capacity limit or padding does.
"""
import functools
import math
import random

import numpy as np
import torch

own = False

HIDDEN, FFN, EXPERTS, TOP_K = 6144, 2048, 384, 8
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
GROUP = 32


def listed():
    return [
        # one token of a generated text: all latency
        {"name": "sort, one token", "op": "sort", "tokens": 1, "top_k": TOP_K, "experts": EXPERTS, "drop": 0.0, "ids": "int32"},
        # a sequence of the longest training length, with slots over the capacity dropped; ids as torch.topk gives them
        {"name": "sort, 65536 tokens", "op": "sort", "tokens": 65536, "top_k": TOP_K, "experts": EXPERTS, "drop": 0.05, "ids": "int64"},
        # the tokens of a micro-batch on their way to the experts
        {"name": "dispatch, bf16", "op": "dispatch", "tokens": 4096, "top_k": TOP_K, "experts": EXPERTS, "drop": 0.0, "ids": "int32",
         "cols": HIDDEN, "dtype": "bf16"},
        # the micro-batch back from them
        {"name": "combine, bf16", "op": "combine", "tokens": 4096, "top_k": TOP_K, "experts": EXPERTS, "drop": 0.0, "ids": "int32",
         "cols": HIDDEN, "dtype": "bf16", "weighted": True},
        # the gradient of dispatch in a small model with rows of odd length and dropped slots
        {"name": "combine, fp32, odd rows", "op": "combine", "tokens": 1000, "top_k": 2, "experts": 16, "drop": 0.1, "ids": "int64",
         "cols": 1001, "dtype": "fp32", "weighted": False},
        # the micro-batch's gradient on its way to the experts, and the router's
        {"name": "backward, bf16", "op": "backward", "tokens": 4096, "top_k": TOP_K, "experts": EXPERTS, "drop": 0.02, "ids": "int32",
         "cols": HIDDEN, "dtype": "bf16"},
        # the hidden rows of a few small experts, the smallest call
        {"name": "dropout, few", "op": "dropout", "batch": 3, "rows": 5, "spread": 4, "shape_seed": 1, "cols": 333, "dtype": "fp32",
         "out": "fp32", "p": 0.1, "device": False},
        # the hidden rows of 48 experts between their products
        {"name": "dropout, experts", "op": "dropout", "batch": 48, "rows": 700, "spread": 400, "shape_seed": 2, "cols": FFN, "dtype": "bf16",
         "out": "bf16", "p": 0.4, "device": True},
        # fp32 rows of odd length, as bf16 for the product that follows
        {"name": "dropout, fp32 to bf16", "op": "dropout", "batch": 16, "rows": 600, "spread": 600, "shape_seed": 3, "cols": FFN + 1,
         "dtype": "fp32", "out": "bf16", "p": 0.25, "device": False},
        # one token through a dense projection
        {"name": "product, one token", "op": "product", "tokens": 1, "top_k": 1, "experts": 1, "drop": 0.0, "rows": HIDDEN, "cols": HIDDEN,
         "gather": False, "out": "bf16"},
        # one token's experts, their up projection; the token's row is read where it is
        {"name": "product, one token's experts", "op": "product", "tokens": 1, "top_k": TOP_K, "experts": EXPERTS, "drop": 0.0, "rows": FFN,
         "cols": HIDDEN, "gather": True, "out": "bf16"},
        # 128 texts at once, the experts' down projection: nearly every expert has rows
        {"name": "product, 128 tokens' experts", "op": "product", "tokens": 128, "top_k": TOP_K, "experts": EXPERTS, "drop": 0.0,
         "rows": HIDDEN, "cols": FFN, "gather": False, "out": "fp32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["sort", "dispatch", "combine", "backward", "dropout", "product"])
    if op == "dropout":
        cols, rows = _log(rng, 1, 8192), _log(rng, 1, 4096)
        return {"op": op, "batch": min(_log(rng, 1, 64), max(1, 66_000_000 // (rows * cols))), "rows": rows,
                "spread": rng.choice([0, rows // 2, rows]), "shape_seed": rng.randrange(1 << 30), "cols": cols,
                "dtype": rng.choice(["bf16", "fp32"]), "out": rng.choice(["bf16", "fp32"]),
                "p": round(rng.uniform(0.01, 0.9), 3), "device": rng.random() < 0.5}
    experts = _log(rng, 2, 512)
    top_k = min(rng.randint(1, 10), experts)
    case = {"op": op, "top_k": top_k, "experts": experts, "drop": rng.choice([0.0, 0.0, 0.03, 0.3])}
    if op == "product":
        case["rows"], case["cols"] = _log(rng, 64, 8192), _log(rng, 64, 8192)
        if rng.random() < 0.3:
            case["experts"] = case["top_k"] = 1
        case["experts"] = min(case["experts"], max(1, 2_400_000_000 // (case["rows"] * case["cols"])))
        case["top_k"] = min(case["top_k"], case["experts"])
        case["tokens"] = _log(rng, 1, 128)
        return {**case, "gather": rng.random() < 0.5, "out": rng.choice(["bf16", "fp32"])}
    case["ids"] = rng.choice(["int32", "int64"])
    if op == "sort":
        return {**case, "tokens": _log(rng, 1, 524288 // top_k)}
    cols = _log(rng, 16, 8192)
    case.update(cols=cols, dtype=rng.choice(["bf16", "fp32"]), tokens=_log(rng, 1, max(2, min(65536, 100_000_000 // (cols * top_k)))))
    if op == "combine":
        case["weighted"] = rng.random() < 0.6
    return case


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _up(x, a):
    return (x + a - 1) // a * a


def _sizes(case):
    """Rows of each tensor of a dropout; where they may be 0, one of them is."""
    r = random.Random(case["shape_seed"])
    got = [max(0, case["rows"] + r.randint(-case["spread"], case["spread"])) for _ in range(case["batch"])]
    if case["spread"] >= case["rows"] and case["batch"] > 1:
        got[-1] = 0
    return got


def _route(case, gen, dev):
    """Expert ids (tokens x top_k) by scores that favour some experts, a share of the slots -1."""
    t, k, e = case["tokens"], case["top_k"], case["experts"]
    score = torch.randn((t, e), generator=gen, device=dev) + 0.5 * torch.randn((1, e), generator=gen, device=dev)
    ids = torch.topk(score, k, dim=1).indices
    lost = torch.rand((t, k), generator=gen, device=dev) < case["drop"]
    return torch.where(lost, torch.full_like(ids, -1), ids).to(getattr(torch, case.get("ids", "int32")))


def _codes(w):
    """Plain 4-bit weights of w (R x K, contracted over its columns): codes
    (R x Kp, one a byte, Kp: K up to a multiple of 128, zeros there) and scale
    bytes e + 127 (R x Kp/32).  The scale 2^e of a group of 32 is the smallest
    power of two, from 2^-125 to 2^125, with the group's largest magnitude at
    most 6 * 2^e; values are rounded to the nearest, ties to the even code."""
    r, k = w.shape
    v = torch.nn.functional.pad(w.float(), (0, _up(k, 128) - k)).view(r, -1, GROUP)
    f, ex = torch.frexp(v.abs().amax(dim=2))  # 6 = 3/4 * 2^3
    e = torch.where(f > 0, ex - 3 + (f > 0.75).int(), torch.full_like(ex, -125)).clamp(-125, 125)
    m = torch.ldexp(v, -e[:, :, None])
    a = m.abs()
    code = sum((a > b).to(torch.uint8) for b in (0.25, 1.25, 2.5, 5.0))
    code += sum((a >= b).to(torch.uint8) for b in (0.75, 1.75, 3.5))
    return (code + 8 * (m < 0).to(torch.uint8)).view(r, -1), (e + 127).to(torch.uint8)


def _operand(code, scale, q, s):
    """Lays codes and scales out as the product takes them, into q (R/16 x Kp/128 x
    64 x 16 bytes) and s (R/16 x Kp/512 rounded up x 16 x 16): a tile of 16 rows
    and 128 columns is 1024 bytes, byte b of its chunk 16 c + r holds columns
    32 (b / 4) + 8 c + 2 (b % 4) and the next one of row r, the first in the low
    half; the scales of row r and of 512 columns are 16 bytes.  Rows past R are
    code 0 with scale 1."""
    r, kp = code.shape
    rp, kt = _up(r, 16), kp // 128
    code = torch.nn.functional.pad(code, (0, 0, 0, rp - r))
    pair = code[:, 0::2] | code[:, 1::2] << 4
    q.copy_(pair.view(rp // 16, 16, kt, 4, 4, 4).permute(0, 2, 4, 1, 3, 5).reshape(q.shape))
    scale = torch.nn.functional.pad(scale, (0, _up(kp, 512) // GROUP - kp // GROUP, 0, rp - r), value=127)
    s.copy_(scale.view(rp // 16, 16, -1, 16).transpose(1, 2))


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(shape, std, dtype=torch.float32):
        return torch.empty(shape, dtype=torch.float32, device=dev).normal_(0.0, std, generator=gen).to(dtype)

    st = {"case": case}
    if case["op"] == "dropout":
        st["xs"] = [normal((r, case["cols"]), 1.0, DTYPES[case["dtype"]]) for r in _sizes(case)]
        st["out"] = [torch.zeros(x.shape, dtype=DTYPES[case["out"]], device=dev) for x in st["xs"]]
        st["state"] = torch.randint(1 << 62, (2,), generator=gen, device=dev)
        st["seed"], st["offset"] = st["state"].tolist()
        return st
    ids = st["ids"] = _route(case, gen, dev)
    t, k, e = case["tokens"], case["top_k"], case["experts"]
    if case["op"] == "sort":
        return st
    if case["op"] == "product":
        r, kp = case["rows"], _up(case["cols"], 128)
        st["q"] = torch.empty((e, _up(r, 16) // 16, kp // 128, 64, 16), dtype=torch.uint8, device=dev)
        st["s"] = torch.empty((e, _up(r, 16) // 16, _up(kp, 512) // 512, 16, 16), dtype=torch.uint8, device=dev)
        for q, s in zip(st["q"], st["s"]):
            _operand(*_codes(normal((r, case["cols"]), 0.02)), q, s)
        st["x"] = normal((t if case["gather"] else t * k, case["cols"]), 1.0, torch.bfloat16)
        st["y"] = torch.zeros((t * k, r), dtype=DTYPES[case["out"]], device=dev)
        st["plan"] = _plan(ids, e)
        # the experts with rows and where those begin and end, as a program knows
        # them that runs an expert at a time
        st["spans"] = [(i, a, b) for i, (a, b) in enumerate(zip(st["plan"][0].tolist(), st["plan"][0].tolist()[1:])) if a < b]
        return st
    dt, h = DTYPES[case["dtype"]], case["cols"]
    if case["op"] == "dispatch":
        st["x"] = normal((t, h), 1.0, dt)
        st["xs"] = torch.zeros((t * k, h), dtype=dt, device=dev)
        return st
    st["plan"] = _plan(ids, e)
    st["ys"] = normal((t * k, h), 1.0, dt)
    st["w"] = torch.softmax(normal((t, k), 1.0), dim=1)
    if case["op"] == "backward":
        st["dout"] = normal((t, h), 1e-3, dt)
        st["dys"] = torch.zeros((t * k, h), dtype=dt, device=dev)
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(st):
    return globals()["_run_" + st["case"]["op"]](st)


def _plan(ids, experts):
    """The plan in plain operations: offsets (experts + 1), the experts with rows
    (their number, their ids, then -1), the sorted row of each slot, the slot of
    each sorted row."""
    key = torch.where((ids >= 0) & (ids < experts), ids, torch.full_like(ids, experts)).flatten()
    key, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(key, torch.arange(experts + 1, device=ids.device, dtype=key.dtype))
    kept = key < experts
    place = torch.arange(key.numel(), device=ids.device)
    rows = torch.empty_like(order).scatter_(0, order, torch.where(kept, place, torch.full_like(place, -1)))
    slots = torch.where(kept, order, torch.full_like(order, -1))
    full = offsets[1:] > offsets[:-1]
    n = full.sum().view(1)
    at = torch.sort((~full).int(), stable=True).indices
    active = torch.cat([n, torch.where(torch.arange(experts, device=ids.device) < n, at, torch.full_like(at, -1))])
    return tuple(v.int() for v in (offsets, active, rows.view(ids.shape), slots))


def _own_plan(nsa, st):
    return nsa.MoePlan(*st["plan"])


def _run_sort(st):
    if own:
        import newton_schulz_03_amd as nsa
        return tuple(nsa.moe_sort(st["ids"], st["case"]["experts"]))
    return _plan(st["ids"], st["case"]["experts"])


def _run_dispatch(st):
    if own:
        import newton_schulz_03_amd as nsa
        plan = nsa.moe_sort(st["ids"], st["case"]["experts"])
        return tuple(plan) + (nsa.moe_dispatch(st["x"], plan, out=st["xs"]),)
    plan = _plan(st["ids"], st["case"]["experts"])
    got = st["x"][plan[3].clamp(min=0) // st["case"]["top_k"]]
    st["xs"].copy_(torch.where((plan[3] >= 0)[:, None], got, st["xs"]))
    return plan + (st["xs"],)


def _run_combine(st):
    weighted = st["case"]["weighted"]
    if own:
        import newton_schulz_03_amd as nsa
        return nsa.moe_combine(st["ys"], _own_plan(nsa, st), weights=st["w"] if weighted else None)
    rows = st["plan"][2]
    y = st["ys"][rows.clamp(min=0)].float()
    y = torch.where((rows >= 0)[:, :, None], y, torch.zeros_like(y))
    return ((y * st["w"][:, :, None] if weighted else y).sum(1)).to(st["ys"].dtype)


def _run_backward(st):
    if own:
        import newton_schulz_03_amd as nsa
        return nsa.moe_combine_backward(st["dout"], st["ys"], _own_plan(nsa, st), st["w"], dys=st["dys"])
    _, _, rows, slots = st["plan"]
    t = st["dout"].float()
    at = slots.clamp(min=0)
    dy = t[at // st["case"]["top_k"]] * st["w"].flatten()[at][:, None]
    st["dys"].copy_(torch.where((slots >= 0)[:, None], dy, st["dys"].float()))
    dw = (st["ys"][rows.clamp(min=0)].float() * t[:, None, :]).sum(2)
    return st["dys"], torch.where(rows >= 0, dw, torch.zeros_like(dw))


M32 = 0xFFFFFFFF


def _philox_round(state, r):
    c, k = state
    p, q = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57  # 64-bit products, their low halves exact
    c = ((q >> 32 & M32) ^ c[1] ^ k[0], q & M32, (p >> 32 & M32) ^ c[3] ^ k[1], p & M32)
    return c, ((k[0] + 0x9E3779B9) & M32, (k[1] + 0xBB67AE85) & M32)


def _keep(n, i, seed, offset, thr, dev):
    """Which of n elements of tensor i stay: 16 bits an element, eight to a block of
    Philox 4x32 with 7 rounds, counter (block, tensor, offset), key seed."""
    b = torch.arange((n + 7) // 8, dtype=torch.int64, device=dev)
    c = (b, *(torch.full_like(b, v) for v in (i, offset & M32, offset >> 32)))
    c, _ = functools.reduce(_philox_round, range(7), (c, (seed & M32, seed >> 32)))
    u = torch.stack([c[0] & 0xFFFF, c[0] >> 16, c[1] & 0xFFFF, c[1] >> 16, c[2] & 0xFFFF, c[2] >> 16, c[3] & 0xFFFF, c[3] >> 16], dim=1)
    return u.view(-1)[:n] >= thr


def _run_dropout(st):
    c = st["case"]
    if own:
        import newton_schulz_03_amd as nsa
        if c["device"]:
            return nsa.dropout_batched(st["xs"], c["p"], rng=st["state"], out=st["out"])
        return nsa.dropout_batched(st["xs"], c["p"], seed=st["seed"], offset=st["offset"], out=st["out"])
    thr = round(c["p"] * 65536)
    [o.copy_(torch.where(_keep(x.numel(), i, st["seed"], st["offset"], thr, x.device).view(x.shape), x.float() * (65536 / (65536 - thr)),
                         torch.zeros((), device=x.device)))
     for i, (x, o) in enumerate(zip(st["xs"], st["out"]))]
    return st["out"]


def _weights(q, s, rows, cols):
    """The values (rows x cols) that the laid out weights of one matrix stand for."""
    tr, kt = q.shape[:2]
    q = q.view(tr, kt, 4, 16, 4, 4).permute(0, 3, 1, 4, 2, 5).reshape(16 * tr, kt * 64, 1)
    codes = torch.cat([q & 15, q >> 4], dim=2).view(16 * tr, kt * 128)
    scale = torch.ldexp(torch.ones((), device=q.device), s.transpose(1, 2).reshape(16 * tr, -1).int() - 127)[:, :kt * 4]
    value = torch.tensor(E2M1 + [-v for v in E2M1], device=q.device)[codes.int()]
    return (value.view(16 * tr, kt * 4, GROUP) * scale[:, :, None]).view(16 * tr, -1)[:rows, :cols]


def _run_product(st):
    c = st["case"]
    if own:
        import newton_schulz_03_amd as nsa
        w = nsa.F4Operand(st["q"], st["s"], c["rows"], c["cols"])
        if c["experts"] == 1 and c["drop"] == 0:  # a matrix that every row takes needs no plan
            return nsa.f4_matmul(st["x"], w, out=st["y"])
        return nsa.f4_matmul(st["x"], w, plan=_own_plan(nsa, st), gather=c["gather"], out=st["y"])
    x = st["x"][st["plan"][3].clamp(min=0) // c["top_k"]] if c["gather"] else st["x"]
    [st["y"][a:b].copy_(x[a:b].float() @ _weights(st["q"][e], st["s"][e], c["rows"], c["cols"]).t())
     for e, a, b in st["spans"]]
    return st["y"]


# ---------------------------------------------------------------------------
# What a pass cannot do without, and its result in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "dropout":
        n = sum(_sizes(case)) * case["cols"]
        return {"bytes": n * sum(2 if case[d] == "bf16" else 4 for d in ("dtype", "out")), "flops": n}
    t, k, e = case["tokens"], case["top_k"], case["experts"]
    n = t * k
    kept = n * (1 - case["drop"])
    if case["op"] == "product":
        r, c = case["rows"], case["cols"]
        # experts that have rows: the expectation for equally likely ones
        some = e * (1 - (1 - 1 / e) ** kept) if e > 1 else 1
        return {"bytes": int(some * r * c * (1 / 2 + 1 / GROUP) + (t if case["gather"] else kept) * c * 2
                             + kept * r * (2 if case["out"] == "bf16" else 4)), "flops": int(2 * kept * r * c)}
    plan = n * (4 if case["ids"] == "int32" else 8) + 8 * n + 8 * (e + 1)
    if case["op"] == "sort":
        return {"bytes": plan, "flops": 0}
    row = case["cols"] * (2 if case["dtype"] == "bf16" else 4)
    if case["op"] == "dispatch":
        return {"bytes": int(plan + (t + kept) * row), "flops": 0}
    if case["op"] == "combine":
        return {"bytes": int((t + kept) * row + n * (8 if case["weighted"] else 4)), "flops": int(2 * kept * case["cols"])}
    return {"bytes": int((t + 2 * kept) * row + 12 * n), "flops": int(3 * kept * case["cols"])}


def _exact_plan(ids, experts):
    ids = ids.cpu().numpy().astype(np.int64)
    flat = ids.ravel()
    slots = np.full(flat.size, -1, np.int64)
    rows = np.full(flat.size, -1, np.int64)
    kept = np.flatnonzero((flat >= 0) & (flat < experts))
    order = kept[np.lexsort((kept, flat[kept]))]
    slots[:order.size] = order
    rows[order] = np.arange(order.size)
    counts = np.bincount(flat[kept], minlength=experts)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    active = np.full(experts + 1, -1, np.int64)
    some = np.flatnonzero(counts)
    active[0] = some.size
    active[1:1 + some.size] = some
    return [torch.from_numpy(v.astype(np.int32)) for v in (offsets, active, rows.reshape(ids.shape), slots)]


def _exact_keep(n, i, seed, offset, thr):
    """_keep again, in unsigned 64-bit integers of the host."""
    u64 = np.uint64
    mask, half = u64(M32), u64(32)
    x = [np.arange((n + 7) // 8, dtype=u64), u64(i), u64(offset & M32), u64(offset >> 32)]
    k0, k1 = seed & M32, seed >> 32
    for _ in range(7):
        a, b = x[0] * u64(0xD2511F53), x[2] * u64(0xCD9E8D57)
        x = [(b >> half) ^ x[1] ^ u64(k0), b & mask, (a >> half) ^ x[3] ^ u64(k1), a & mask]
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    words = np.stack([np.broadcast_to(v, x[0].shape) for v in x], axis=1).astype("<u4")
    return np.ascontiguousarray(words).view("<u2").ravel()[:n] >= thr


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "dropout":
        thr = round(case["p"] * 65536)
        got = []
        for i, x in enumerate(st["xs"]):
            keep = torch.from_numpy(_exact_keep(x.numel(), i, st["seed"], st["offset"], thr)).to(x.device)
            got.append(x.double().mul_(65536).div_(65536 - thr).masked_fill_(~keep.view(x.shape), 0.0))
        return got
    t, k, e = case["tokens"], case["top_k"], case["experts"]
    plan = _exact_plan(st["ids"], e)
    if case["op"] == "sort":
        return tuple(plan)
    n = int(plan[0][-1])
    slot = plan[3][:n].long().cuda()
    if case["op"] == "dispatch":
        xs = torch.zeros((t * k, case["cols"]), dtype=torch.float64, device="cuda")
        xs[:n] = st["x"].double().index_select(0, slot // k)
        return tuple(plan) + (xs,)
    if case["op"] == "product":
        values = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
        y = torch.zeros((t * k, case["rows"]), dtype=torch.float64, device="cuda")
        bounds = plan[0].tolist()
        r, kp = case["rows"], _up(case["cols"], 128)
        row = torch.arange(r, device="cuda")[:, None]
        col = torch.arange(case["cols"], device="cuda")[None, :]
        # where row and column lie in the laid out matrix, element by element
        at = ((row // 16 * (kp // 128) + col // 128) * 64 + 16 * (col % 32 // 8) + row % 16) * 16 + 4 * (col % 128 // 32) + col % 8 // 2
        sat = ((row // 16 * (_up(kp, 512) // 512) + col // 512) * 16 + row % 16) * 16 + col % 512 // 32
        for i in range(e):
            a, b = bounds[i], bounds[i + 1]
            if a == b:
                continue
            byte = st["q"][i].flatten()[at].int()
            code = torch.where(col % 2 == 1, byte >> 4, byte & 15)
            w = values[(code & 7).long()] * torch.exp2(st["s"][i].flatten()[sat].double() - 127)
            w = torch.where(code >= 8, -w, w)
            x = st["x"].double()
            y[a:b] = (x.index_select(0, slot[a:b] // k) if case["gather"] else x[a:b]) @ w.t()
        return y
    if case["op"] == "combine":
        w = st["w"].double().flatten()[slot] if case["weighted"] else torch.ones(n, dtype=torch.float64, device="cuda")
        out = torch.zeros((t, case["cols"]), dtype=torch.float64, device="cuda")
        return out.index_add_(0, slot // k, st["ys"][:n].double() * w[:, None])
    dy = torch.zeros((t * k, case["cols"]), dtype=torch.float64, device="cuda")
    d = st["dout"].double().index_select(0, slot // k)
    dy[:n] = d * st["w"].double().flatten()[slot][:, None]
    dw = torch.zeros(t * k, dtype=torch.float64, device="cuda")
    dw[slot] = (d * st["ys"][:n].double()).sum(1)
    return dy, dw.view(t, k)
