"""Plain 64-bit reference of the 4-bit weight format and its products (numpy)."""
import numpy as np

MX, NV = 0, 1
GRID = np.array([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
VALUES = np.concatenate([GRID, -GRID])
MIN_SCALE, MAX_SCALE = 2.0 ** -100, 2.0 ** 117


def block(fmt):
    return 32 if fmt == MX else 16


def e4m3_grid():
    g = [i * 2.0 ** -9 for i in range(8)]
    for e in range(1, 16):
        g += [(8 + f) * 2.0 ** (e - 10) for f in range(8)]
    return np.array(g[:127], dtype=np.float64)     # 0 .. 448; byte 127 is NaN


E4M3 = np.concatenate([e4m3_grid(), [np.nan]])
E4M3 = np.concatenate([E4M3, -E4M3])
E8M0 = np.concatenate([2.0 ** (np.arange(255, dtype=np.float64) - 127), [np.nan]])


def bf16(bits):
    return (np.asarray(bits, dtype=np.uint32) << 16).view(np.float32)


def to_bf16(x):
    """fp64 -> the nearest bf16 (ties to even), as fp64 values; no overflow handling beyond inf."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(all="ignore"):
        f = x.astype(np.float32)
        # round to odd into fp32 first, so that the second rounding sees which side x was on
        b = f.view(np.uint32).astype(np.int64)
        err = x - f.astype(np.float64)
        low = (b & 1) == 0
        away = np.where(np.signbit(x), err < 0, err > 0)
        b = np.where(np.isfinite(f) & (err != 0) & low, np.where(away, b + 1, b - 1), b)
        r = (b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000
        r = np.where(np.isnan(f), 0x7FC00000, r)
        return r.astype(np.uint32).view(np.float32).astype(np.float64)


def nearest(y, grid):
    """Index of the nearest grid value (ties to the even index, beyond the end to the last)."""
    mid = (grid[1:] + grid[:-1]) / 2
    lo, hi = np.searchsorted(mid, y, side="left"), np.searchsorted(mid, y, side="right")
    return np.where(lo == hi, lo, np.where(lo % 2 == 0, lo, hi))


def calibrate(x):
    x = np.abs(np.asarray(x, dtype=np.float64))
    top = x[np.isfinite(x)].max(initial=0.0)
    if top == 0:
        return np.float32(1)
    return np.float32(min(max(float(np.float32(top / 2688)), MIN_SCALE), MAX_SCALE))


def quantize(x, fmt, s=1.0):
    """(packed codes [rows, (cols+1)//2], scale bytes [rows, blocks]) of x (fp32 or bf16 values)."""
    x = np.asarray(x, dtype=np.float32).astype(np.float64)
    rows, cols = x.shape
    B = block(fmt)
    nb = -(-cols // B)
    v = np.zeros((rows, nb * B))
    v[:, :cols] = x
    v = v.reshape(rows, nb, B)
    with np.errstate(all="ignore"):
        amax = np.abs(v).max(-1)
        bad = ~np.isfinite(v).all(-1)
        if fmt == MX:
            safe = np.where(bad | (amax == 0), 1.0, amax)
            e = np.frexp(safe)[1] - 1
            byte = np.where(amax == 0, 0, np.maximum(e - 2 + 127, 0))
            byte = np.where(bad, 255, byte)
            unit = 2.0 ** (np.where(bad, 0, byte) - 127.0)
            mag = nearest(np.where(bad[..., None], 0, np.abs(v)) / unit[..., None], GRID)
        else:
            s = float(np.float32(s))
            bad = bad | (not (MIN_SCALE <= s <= MAX_SCALE))
            byte = nearest(np.where(bad, 0, amax) / (6 * s if s > 0 else 1.0), e4m3_grid())
            unit = e4m3_grid()[byte] * s
            live = (byte > 0) & ~bad
            y = np.where(live[..., None], np.abs(v), 0) / np.where(live, unit, 1.0)[..., None]
            mag = nearest(y, GRID)
            byte = np.where(bad, 127, byte)
    code = np.where(bad[..., None], 0, mag | (np.signbit(v) << 3)).astype(np.uint8)
    code = code.reshape(rows, nb * B)
    code[:, cols:] = 0
    w = (cols + 1) // 2
    packed = (code[:, 0::2] | (code[:, 1::2] << 4))[:, :w]
    return np.ascontiguousarray(packed), byte.astype(np.uint8)


def unit_values(codes, scales, cols, fmt):
    """Values [rows, cols] in fp64 without the tensor scale."""
    codes = np.asarray(codes, dtype=np.uint8)[:, : (cols + 1) // 2]
    c = np.empty((codes.shape[0], codes.shape[1] * 2), dtype=np.uint8)
    c[:, 0::2], c[:, 1::2] = codes & 15, codes >> 4
    unit = (E8M0 if fmt == MX else E4M3)[np.asarray(scales)]
    unit = np.repeat(unit, block(fmt), axis=1)[:, :cols]
    return VALUES[c[:, :cols]] * unit


def product(x, w, offsets=None, grad=False):
    """(x w^T or x w, the sum of the terms' sizes) in fp64; rows outside the groups NaN."""
    x, w = np.asarray(x, dtype=np.float64), np.asarray(w, dtype=np.float64)
    g = 1 if offsets is None else len(offsets) - 1
    n = w.shape[0] // g
    off = [0, x.shape[0]] if offsets is None else list(offsets)
    out = np.full((x.shape[0], w.shape[1] if grad else n), np.nan)
    size = np.zeros_like(out)
    for i in range(g):
        a, b = off[i], off[i + 1]
        p = w[i * n:(i + 1) * n]
        p = p if grad else p.T
        out[a:b] = x[a:b] @ p
        size[a:b] = np.abs(x[a:b]) @ np.abs(p)
    return out, size
