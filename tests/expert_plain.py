"""Plain forms, in numpy and 64 bits, of the operators of the expert layers."""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def plan(ids, experts):
    """(offsets, active, rows, slots) by counting, one slot at a time."""
    flat = np.asarray(ids, dtype=np.int64).ravel()
    of = [[] for _ in range(experts)]
    for s, e in enumerate(flat.tolist()):
        if 0 <= e < experts:
            of[e].append(s)
    order = [s for group in of for s in group]
    offsets = np.concatenate([[0], np.cumsum([len(g) for g in of])])
    rows = np.full(flat.size, -1)
    rows[order] = np.arange(len(order))
    slots = np.full(flat.size, -1)
    slots[:len(order)] = order
    some = [e for e in range(experts) if of[e]]
    active = np.array([len(some)] + some + [-1] * (experts - len(some)))
    return offsets, active, rows.reshape(np.shape(ids)), slots


def philox(counter, key, rounds):
    """The four words (uint64 arrays below 2^32) of Philox 4x32 for 4 counter words and 2 key words."""
    u, m = np.uint64, 0xFFFFFFFF
    c, k = [np.asarray(v, dtype=np.uint64) for v in counter], list(key)
    for _ in range(rounds):
        p, q = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        c = [(q >> u(32)) ^ c[1] ^ u(k[0]), q & u(m), (p >> u(32)) ^ c[3] ^ u(k[1]), p & u(m)]
        k = [(k[0] + 0x9E3779B9) & m, (k[1] + 0xBB67AE85) & m]
    return c


def keep(n, tensor, seed, offset, threshold):
    """Which of n elements of the list's tensor number `tensor` stay."""
    m = 0xFFFFFFFF
    block = np.arange((n + 7) // 8, dtype=np.uint64)
    one = np.ones_like(block)
    words = philox([block, one * np.uint64(tensor), one * np.uint64(offset & m), one * np.uint64(offset >> 32)],
                   (seed & m, seed >> 32), 7)
    halves = [(w >> np.uint64(16 * h)) & np.uint64(0xFFFF) for w in words for h in (0, 1)]
    return np.stack(halves, axis=1).ravel()[:n] >= threshold


def e2m1(x):
    """Codes of the nearest e2m1 values of float64 x (zeros keep their sign), ties to the even
    code; saturates."""
    a = np.abs(x)[..., None]
    d = np.abs(a - E2M1)
    best = d.min(axis=-1, keepdims=True)
    near = d == best  # one or two neighbours
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(near.sum(-1) > 1, even.argmax(-1), near.argmax(-1))
    return code + 8 * np.signbit(x)


def f4(w):
    """(codes, scale bytes) of float64 w (R x K), contracted over its columns: R x Kp and
    R x Kp / 32, Kp = K up to a multiple of 128."""
    r, k = w.shape
    kp = -(-k // 128) * 128
    v = np.zeros((r, kp))
    v[:, :k] = w
    v = v.reshape(r, kp // 32, 32)
    bad = ~np.isfinite(v).all(axis=2)
    v = np.where(bad[:, :, None], 0.0, v)
    top = np.abs(v).max(axis=2)
    e = np.full(top.shape, -125)
    for x in range(-125, 125):  # the smallest exponent that holds the largest magnitude
        e = np.where(top > 6.0 * 2.0 ** x, x + 1, e)
    codes = e2m1(v * np.exp2(-e.astype(np.float64))[:, :, None])
    codes = np.where(bad[:, :, None], 0, codes)
    return codes.reshape(r, kp), np.where(bad, 255, e + 127)


def f4_layout(codes, scales):
    """Codes and scale bytes as an operand holds them, element by element."""
    r, kp = codes.shape
    rt, kt, quads = -(-r // 16), kp // 128, -(-kp // 512)
    q = np.zeros((rt, kt, 64, 16), dtype=np.uint8)
    s = np.full((rt, quads, 16, 16), 127, dtype=np.uint8)
    row, col = np.meshgrid(np.arange(r), np.arange(kp), indexing="ij")
    at = (row // 16, col // 128, 16 * (col % 32 // 8) + row % 16, 4 * (col % 128 // 32) + col % 8 // 2)
    np.bitwise_or.at(q, at, (codes << (4 * (col % 2))).astype(np.uint8))
    row, group = np.meshgrid(np.arange(r), np.arange(kp // 32), indexing="ij")
    s[row // 16, group // 16, row % 16, group % 16] = scales
    return q, s


def f4_values(codes, scales, cols):
    """The values that codes and scale bytes stand for, without the padding."""
    v = np.where(codes >= 8, -1.0, 1.0) * E2M1[codes & 7]
    p = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    with np.errstate(invalid="ignore"):
        return (v.reshape(len(v), -1, 32) * p[:, :, None]).reshape(v.shape)[:, :cols]
