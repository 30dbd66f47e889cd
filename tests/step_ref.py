"""Plain 64-bit implementations of a training turn's calls (numpy), for their tests."""
import numpy as np

LOW = (1 << 32) - 1


def scores(x, sigmoid):
    if sigmoid:
        with np.errstate(over="ignore"):
            return 1 / (1 + np.exp(-x))
    top = x.max(1, keepdims=True)
    e = np.exp(x - np.where(np.isneginf(top), 0, top))
    z = e.sum(1, keepdims=True)
    return e / np.where(z == 0, 1, z)


def select(x, bias, k, sigmoid, groups=1, top_groups=1, renormalize=False, scale=1.0):
    """(ids, weights) row by row, from the definition."""
    x = x.astype(np.float64)
    s = scores(x, sigmoid)
    rows, e = x.shape
    ids, w = np.full((rows, k), -1), np.zeros((rows, k))
    size = e // groups
    for r in range(rows):
        value = s[r] + (0 if bias is None else bias.astype(np.float64))
        taken = set(range(groups))
        if top_groups < groups:
            of = []
            for g in range(groups):
                vals = sorted((value[i] for i in range(g * size, (g + 1) * size) if not np.isneginf(x[r, i])), reverse=True)
                of.append(sum(vals[:2]) if vals else -np.inf)
            taken = set(sorted(range(groups), key=lambda g: (-of[g], g))[:top_groups])
        rank = x[r] if bias is None else value
        live = [i for i in range(e) if not np.isneginf(x[r, i]) and i // size in taken]
        best = sorted(live, key=lambda i: (-rank[i], i))[:k]
        ids[r, :len(best)] = best
        w[r, :len(best)] = s[r, best]
    if renormalize:
        z = w.sum(1, keepdims=True)
        w = w / np.where(z == 0, 1, z)
    return ids.astype(np.int32), w * scale


def select_grad(x, ids, dw, sigmoid, renormalize, scale=1.0):
    """(gradient, a bound of what its terms add up to without their signs)"""
    x, dw = x.astype(np.float64), dw.astype(np.float64)
    s = scores(x, sigmoid)
    ds, most = np.zeros_like(s), np.zeros_like(s)
    for r in range(len(x)):
        js = [j for j in range(ids.shape[1]) if 0 <= ids[r, j] < x.shape[1]]
        sel = np.array([s[r, ids[r, j]] for j in js])
        total = sel.sum() if renormalize else 1.0
        total = total if total else 1.0
        mean = sum(dw[r, j] * v for j, v in zip(js, sel)) / total if renormalize else 0.0
        for j in js:
            ds[r, ids[r, j]] += (dw[r, j] - mean) / total * scale
            most[r, ids[r, j]] += (abs(dw[r, j]) + np.abs(dw[r, js]).max()) / total * abs(scale)
    if sigmoid:
        return s * (1 - s) * ds, s * most
    return s * (ds - (ds * s).sum(1, keepdims=True)), s * (most + (most * s).sum(1, keepdims=True))


def order(ids, experts):
    flat = ids.reshape(-1)
    offsets = np.zeros(experts + 1, np.int32)
    slots = np.full(flat.shape, -1, np.int32)
    at = 0
    for e in range(experts):
        offsets[e] = at
        mine = np.nonzero(flat == e)[0]
        slots[mine] = np.arange(at, at + len(mine))
        at += len(mine)
    offsets[experts] = at
    return offsets, slots.reshape(ids.shape)


def logprobs(x, scale):
    """(log p, lse, entropy, largest) of the rows; rows without an open token: -inf, -inf, 0."""
    z = x.astype(np.float64) * scale
    top = z.max(1, keepdims=True)
    d = z - np.where(np.isneginf(top), 0, top)
    e = np.exp(d)
    s = e.sum(1, keepdims=True)
    none = s == 0
    logs = np.log(np.where(none, 1, s))
    lp = np.where(none, -np.inf, d - logs)
    p = e / np.where(none, 1, s)
    ent = -(p * np.where(p > 0, lp, 0)).sum(1)
    return lp, np.where(none, -np.inf, top + logs)[:, 0], ent, p


def dither(index, seed, step):
    """The two 16-bit numbers of elements `index` (uint64 array)."""
    i = index.astype(np.uint64)
    key = (seed * 0x9E3779B1 + step * 0x6A09E667) & LOW
    m = np.uint64(LOW)
    x = ((i & m) * np.uint64(0x9E3779B1) + ((i >> np.uint64(32)) * np.uint64(0xBB67AE85) & m) + np.uint64(key)) & m
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(0x6A09E667)) & m
    x = ((x ^ (x >> np.uint64(15))) * np.uint64(0x3C6EF373)) & m
    x = x ^ (x >> np.uint64(16))
    return (x & np.uint64(0xFFFF)).astype(np.float64) / 65536, (x >> np.uint64(16)).astype(np.float64) / 65536


GRID = np.array([i * 2.0 ** -9 for i in range(8)] + [(8 + f) * 2.0 ** (e - 10) for e in range(1, 16) for f in range(8)][:-1])


def to8(x, r, keep):
    """(codes, scale bytes) of a state `x` (float32 values as float64): by the grid of e4m3 values."""
    n = len(x)
    nb = -(-n // 32)
    b = np.zeros(nb * 32)
    b[:n] = x
    b = b.reshape(nb, 32)
    codes, byte = np.zeros((nb, 32), np.uint8), np.zeros(nb, np.uint8)
    r = np.broadcast_to(r, (n,))
    rr = np.zeros(nb * 32)
    rr[:n] = r
    rr = rr.reshape(nb, 32)
    for i in range(nb):
        if not np.isfinite(b[i]).all():
            byte[i] = 255
            continue
        top = np.abs(b[i]).max()
        e = 0
        if top:
            while e < 254 and top / 2.0 ** (e - 127) > 448:
                e += 1
        byte[i] = e
        y = np.abs(b[i]) / 2.0 ** (e - 127)
        low = np.searchsorted(GRID, y, side="right") - 1
        gap = np.where(low + 1 < len(GRID), GRID[np.minimum(low + 1, len(GRID) - 1)] - GRID[low], np.inf)
        up = (y - GRID[low]) / gap + rr[i] >= 1
        code = low + up
        if keep:
            code = np.where((y > 0) & (code == 0), 1, code)
        codes[i] = code | (np.signbit(b[i]) * 128)
    return codes.reshape(-1)[:n], byte


def from8(codes, byte):
    mag = np.concatenate([GRID, [np.nan]])[codes & 127]
    v = np.where(codes & 128, -mag, mag)
    unit = np.where(byte == 255, np.nan, 2.0 ** (byte.astype(np.float64) - 127))
    return v * np.repeat(unit, 32)[:len(codes)]
