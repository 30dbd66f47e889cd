"""The 4-bit weight operators as they are measured: cases, inputs, a plain
form of each in elementary torch operations, and the calls of the library.

A 4-bit tensor holds rows of e2m1 codes, two a byte (the even element in the
low nibble), with one scale for each block of a row:

  mx  blocks of 32, scale 2^(byte - 127)
  nv  blocks of 16, scale an e4m3 value, times one fp32 scale of the tensor

Kinds of a case:

  roundtrip  quantise a bf16 / fp32 tensor, and read the 4 bits back
  read       read a 4-bit tensor back
  linear     y = x w^T, x bf16 and w in 4 bits; `groups` weights, the rows of
             x sorted by weight (experts)
  linear4    the same with x quantised within the call
  grad       dx = dy w, the gradient of `linear` with respect to x
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = {"mx": 32, "nv": 16}
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
MOST_FLOPS = 2.0 * 8192 * 14336 * 4096


def listed():
    return [
        # the 4096 x 4096 tensor of the smallest refit workload, as a trainer quantises it each step
        {"name": "roundtrip_4096", "kind": "roundtrip", "rows": 4096, "cols": 4096, "dtype": "bf16", "fmt": "mx"},
        # gate matrices of 16 experts (an EP=8 share of a 128-expert layer), fp32 masters, scale taken from the data
        {"name": "roundtrip_masters", "kind": "roundtrip", "rows": 12288, "cols": 2048, "dtype": "fp32", "fmt": "nv"},
        # ragged rows: an odd length that ends inside a byte and inside a block
        {"name": "read_odd", "kind": "read", "rows": 1001, "cols": 1999, "dtype": "fp32", "fmt": "nv"},
        # an embedding matrix of 151936 x 2048 read back whole
        {"name": "read_embedding", "kind": "read", "rows": 151936, "cols": 2048, "dtype": "bf16", "fmt": "mx"},
        # one token through a square projection: latency counts
        {"name": "decode_one", "kind": "linear", "m": 1, "n": 4096, "k": 4096, "groups": 1, "fmt": "mx", "dtype": "bf16"},
        # a decode batch through an up projection
        {"name": "decode_batch", "kind": "linear", "m": 24, "n": 14336, "k": 4096, "groups": 1, "fmt": "nv", "dtype": "bf16"},
        # a long prefill through an up projection
        {"name": "prefill", "kind": "linear", "m": 8192, "n": 14336, "k": 4096, "groups": 1, "fmt": "mx", "dtype": "bf16"},
        # 2048 tokens sent to 8 of 128 experts each, ragged, some experts empty
        {"name": "experts", "kind": "linear", "m": 16384, "n": 768, "k": 2048, "groups": 128, "fmt": "nv", "dtype": "bf16"},
        # the prefill with its activations in 4 bits too
        {"name": "prefill_4bit", "kind": "linear4", "m": 8192, "n": 14336, "k": 4096, "groups": 1, "fmt": "mx", "dtype": "bf16"},
        # odd sizes, a reduction that ends inside a tile, fp32 results
        {"name": "ragged_4bit", "kind": "linear4", "m": 333, "n": 1000, "k": 2080, "groups": 1, "fmt": "mx", "dtype": "fp32"},
        # backward through a down projection
        {"name": "grad_down", "kind": "grad", "m": 4096, "n": 4096, "k": 14336, "groups": 1, "fmt": "mx", "dtype": "bf16"},
        # backward through the experts, fp32 gradients
        {"name": "grad_experts", "kind": "grad", "m": 16384, "n": 768, "k": 2048, "groups": 128, "fmt": "nv", "dtype": "fp32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["roundtrip", "read", "linear", "linear4", "grad"])
    fmt = "mx" if kind == "linear4" else rng.choice(["mx", "nv"])
    dtype = rng.choice(["bf16", "fp32"])
    if kind in ("roundtrip", "read"):
        cols = _log(rng, 1, 16384)
        if rng.random() < 0.6:
            cols = max(32, cols // 32 * 32)
        rows = min(_log(rng, 1, 65536), (96 << 20) // cols)
        return {"kind": kind, "rows": rows, "cols": cols, "dtype": dtype, "fmt": fmt}
    groups = 1 if rng.random() < 0.6 else _log(rng, 2, 128)
    top = 16384 if groups == 1 else 2048
    n, k = _log(rng, 16, top), _log(rng, 32, top)
    if rng.random() < 0.7:
        n, k = max(16, n // 16 * 16), max(32, k // 32 * 32)
    m = min(_log(rng, 1, 16384), int(MOST_FLOPS / 2 / n / k))
    return {"kind": kind, "m": m, "n": n, "k": k, "groups": groups, "fmt": fmt, "dtype": dtype}


def work(case):
    fmt = case["fmt"]
    held = lambda rows, cols: rows * (-(-cols // 2) + -(-cols // BLOCK[fmt]))  # noqa: E731
    size = 2 if case["dtype"] == "bf16" else 4
    if case["kind"] in ("roundtrip", "read"):
        n = case["rows"] * case["cols"]
        read = n * size if case["kind"] == "roundtrip" else 0
        return {"bytes": read + held(case["rows"], case["cols"]) + n * size, "flops": 0}
    m, n, k = case["m"], case["n"], case["k"]
    used = min(case["groups"], m) if case["groups"] > 1 else 1
    into, out = (n, k) if case["kind"] == "grad" else (k, n)
    return {"bytes": 2 * m * into + used * held(n, k) + size * m * out, "flops": 2.0 * m * n * k}


# ------------------------------------------------------------ plain forms

def _blocks(x, b):
    """x [rows, cols] as [rows, blocks, b], the last block filled with zeros."""
    rows, cols = x.shape
    nb = -(-cols // b)
    if nb * b != cols:
        x = torch.nn.functional.pad(x, (0, nb * b - cols))
    return x.reshape(rows, nb, b)


def _round_e2m1(y):
    """Magnitudes y >= 0 to the nearest of 0 .5 1 1.5 2 3 4 6, ties to the even code."""
    y = torch.where(y < 2, torch.round(y * 2) / 2, torch.where(y < 4, torch.round(y), torch.round(y / 2) * 2))
    return y.clamp(max=6.0)


def _quantise(x, fmt, s=None):
    """(codes [rows, blocks, b] uint8, scale bytes [rows, blocks] uint8, s) of x."""
    v = _blocks(x.float(), BLOCK[fmt])
    amax = v.abs().amax(-1)
    if fmt == "mx":
        exps = (amax.view(torch.int32) >> 23) - 2
        scales = exps.clamp(min=0).to(torch.uint8)
        # the two halves of 2^(127 - byte): each a normal number, and x times the first exact or tiny
        up = 127 - scales.to(torch.int32)
        half = up >> 1
        one = lambda e: ((e + 127) << 23).view(torch.float32)[..., None]  # noqa: E731
        mag = _round_e2m1(v.abs() * one(half) * one(up - half))
    else:
        if s is None:
            s = (amax.amax().double() / 2688).clamp(2.0 ** -100, 2.0 ** 117).float().reshape(1)
            s = torch.where(amax.amax() == 0, torch.ones_like(s), s)
        t = amax.double() / (6 * s.double())   # next to a border 32 bits decide wrongly
        step = torch.exp2(torch.floor(torch.log2(t.clamp(min=2.0 ** -6))) - 3)
        step = torch.where(t >= step * 16, step * 2, step)
        held = (torch.round(t / step) * step).clamp(max=448.0)
        scales = held.float().to(torch.float8_e4m3fn).view(torch.uint8)
        y = v.abs().double() / (held * s.double())[..., None]
        mag = _round_e2m1(torch.where(held[..., None] == 0, 0.0, y)).float()
    code = torch.where(mag < 2, mag * 2, torch.where(mag < 4, mag + 2, mag / 2 + 4)).to(torch.uint8)
    return code | (torch.signbit(v).to(torch.uint8) << 3), scales, s


def _pack(code, cols):
    """Codes [rows, blocks, b] as bytes [rows, stride], the stride a multiple of 16."""
    rows = code.shape[0]
    c = code.reshape(rows, -1)
    packed = c[:, 0::2] | (c[:, 1::2] << 4)
    stride = -(-(-(-cols // 2)) // 16) * 16
    out = torch.zeros(rows, stride, dtype=torch.uint8, device=code.device)
    w = min(stride, packed.shape[1])
    out[:, :w] = packed[:, :w]
    return out


def _values(codes, scales, s, cols, fmt):
    """The values [rows, cols] of a packed tensor, in fp32."""
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    packed = codes[:, : -(-cols // 2)]
    c = torch.stack((packed & 15, packed >> 4), -1).reshape(codes.shape[0], -1)[:, :cols]
    v = _blocks(table[c.int()], BLOCK[fmt])
    if fmt == "mx":
        v = v * scales.view(torch.float8_e8m0fnu).float()[..., None]
    else:
        v = v * scales.view(torch.float8_e4m3fn).float()[..., None] * s
    return v.reshape(codes.shape[0], -1)[:, :cols]


def _decoded_scales(scales, fmt):
    return scales.view(torch.float8_e8m0fnu if fmt == "mx" else torch.float8_e4m3fn)


def _product(a, w, state, transposed):
    """a w^T (or a w), the rows of a by their group's w; fp32."""
    c = state["case"]
    g, n, k = c["groups"], c["n"], c["k"]
    if g == 1:
        return a.float() @ (w.t() if transposed else w)
    # rows of each group side by side in a padded batch
    off = state["offsets"].long()
    row = torch.arange(a.shape[0], device=a.device)
    group = torch.searchsorted(off[1:], row, right=True)
    at = row - off[group]
    batch = torch.zeros(g, state["longest"], a.shape[1], device=a.device)
    batch[group, at] = a.float()
    w = w.reshape(g, n, k)
    return torch.bmm(batch, w.transpose(1, 2).contiguous() if transposed else w)[group, at]


# -------------------------------------------------------------------- cases

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _weights(rows, cols, g):
    """Weights as a model holds them: normal, rows of different size."""
    w = torch.randn(rows, cols, device="cuda", generator=g)
    size = torch.exp(0.3 * torch.randn(rows, 1, device="cuda", generator=g))
    return w.mul_(size.mul_(0.02))


def _acts(m, k, g):
    """Activations: normal, a few columns far larger."""
    x = torch.randn(m, k, device="cuda", generator=g)
    big = torch.rand(k, device="cuda", generator=g) < 0.004
    return (x * torch.where(big, 12.0, 1.0)).bfloat16()


def _counts(m, groups, seed):
    """Rows of each group: Zipf shares in a shuffled order, so some groups are empty."""
    r = np.random.RandomState(seed % (1 << 31))
    p = 1.0 / np.arange(1, groups + 1) ** 0.8
    p = r.permutation(p / p.sum())
    p[r.rand(groups) < 0.05] = 0
    p = p / p.sum() if p.sum() else np.full(groups, 1.0 / groups)
    return r.multinomial(m, p)


def prepare(case, seed):
    return _with_handles(_inputs(case, seed))


def _inputs(case, seed):
    g = _generator(seed)
    state = {"case": dict(case)}
    fmt = case["fmt"]
    if case["kind"] == "roundtrip":
        state["x"] = _weights(case["rows"], case["cols"], g).to(TYPES[case["dtype"]])
        return state
    rows = case["rows"] if case["kind"] == "read" else case["n"] * case["groups"]
    cols = case["cols"] if case["kind"] == "read" else case["k"]
    w = _weights(rows, cols, g).bfloat16()
    s = (w.float().abs().max() / 2688).reshape(1) if fmt == "nv" else None
    code, scales = [], []
    for part in w.split(max(1, (32 << 20) // cols)):   # the plain quantiser's 64-bit steps are large
        a, b, _ = _quantise(part, fmt, s)
        code.append(_pack(a, cols))
        scales.append(b)
    state.update(codes=torch.cat(code), scales=torch.cat(scales), tensor_scale=s)
    if case["kind"] == "read":
        return state
    m = case["m"]
    state["x"] = _acts(m, case["n"] if case["kind"] == "grad" else case["k"], g)
    if case["groups"] > 1:
        counts = _counts(m, case["groups"], seed)
        off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        state["offsets"] = torch.from_numpy(off).cuda()
        state["longest"] = int(counts.max())
    return state


def _with_handles(state):
    """The buffers and handles that a program keeps from call to call."""
    if own:
        from bit_exact_xor_amd import dcr
        c = state["case"]
        fmt = dcr.FP4_MX if c["fmt"] == "mx" else dcr.FP4_NV
        if c["kind"] == "roundtrip":
            state["q"] = dcr.Fp4Tensor(c["rows"], c["cols"], fmt)
        elif c["kind"] == "read":
            state["q"] = dcr.Fp4Tensor(c["rows"], c["cols"], fmt, codes=state["codes"], scales=state["scales"],
                                       tensor_scale=state["tensor_scale"])
        else:
            state["q"] = dcr.Fp4Tensor(c["n"] * c["groups"], c["k"], fmt, codes=state["codes"],
                                       scales=state["scales"], tensor_scale=state["tensor_scale"])
            if c["kind"] == "linear4":
                state["xq"] = dcr.Fp4Tensor(c["m"], c["k"], fmt)
        state["workspace"] = dcr.fp4_workspace()
    return state


def run(state):
    c = state["case"]
    kind, fmt, out = c["kind"], c["fmt"], TYPES[c["dtype"]]
    if own:
        return _run_own(state, kind, out)
    if kind == "roundtrip":
        code, scales, s = _quantise(state["x"], fmt)
        v = _values(_pack(code, c["cols"]), scales, s, c["cols"], fmt).to(out)
        got = {"values": v, "scales": _decoded_scales(scales, fmt)}
        return {**got, "tensor_scale": s} if fmt == "nv" else got
    w = _values(state["codes"], state["scales"], state["tensor_scale"], c["cols"] if kind == "read" else c["k"], fmt)
    if kind == "read":
        return w.to(out)
    x = state["x"]
    if kind == "linear4":
        code, scales, s = _quantise(x, fmt)
        x = _values(_pack(code, c["k"]), scales, s, c["k"], fmt)
    return _product(x, w, state, kind != "grad").to(out)


def _run_own(state, kind, out):
    from bit_exact_xor_amd import dcr
    c, q, ws = state["case"], state["q"], state["workspace"]
    if kind == "roundtrip":
        y = torch.empty(c["rows"], c["cols"], dtype=out, device="cuda")
        nv = c["fmt"] == "nv"
        dcr.dcr_fp4_quantize(state["x"], q, dcr.FP4_CALIBRATE if nv else 0, ws)
        dcr.dcr_fp4_dequantize(q, y)
        got = {"values": y, "scales": _decoded_scales(q.scales, c["fmt"])}
        return {**got, "tensor_scale": q.tensor_scale} if nv else got
    if kind == "read":
        y = torch.empty(c["rows"], c["cols"], dtype=out, device="cuda")
        dcr.dcr_fp4_dequantize(q, y)
        return y
    y = torch.empty(c["m"], c["k"] if kind == "grad" else c["n"], dtype=out, device="cuda")
    off = state.get("offsets")
    if kind == "linear":
        dcr.dcr_fp4_matmul(state["x"], q, y, off, ws)
    elif kind == "linear4":
        dcr.dcr_fp4_quantize(state["x"], state["xq"])
        dcr.dcr_fp4_matmul_q(state["xq"], q, y, off, ws)
    else:
        dcr.dcr_fp4_matmul_grad(state["x"], q, y, off, ws)
    return y


# ------------------------------------------------------ the definition, in 64 bits

GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _nearest(y, grid):
    """Index of the nearest grid value to y >= 0; a tie goes to the even index, and past the end to the last."""
    grid = torch.as_tensor(grid, dtype=torch.float64, device=y.device)
    mid = (grid[1:] + grid[:-1]) / 2
    low, high = torch.searchsorted(mid, y), torch.searchsorted(mid, y, right=True)
    return torch.where(low == high, low, torch.where(low % 2 == 0, low, high))


def _e4m3_grid():
    sub = [i * 2.0 ** -9 for i in range(8)]
    return sub + [(8 + f) * 2.0 ** (e - 10) for e in range(1, 16) for f in range(8) if not (e == 15 and f == 7)]


def _exact_quantise(x, fmt):
    """(values in fp64 without the tensor's scale, block scales, the tensor's scale) of x."""
    rows, cols = x.shape
    b = BLOCK[fmt]
    nb = -(-cols // b)
    v = torch.zeros(rows, nb * b, dtype=torch.float64, device=x.device)
    v[:, :cols] = x.double()
    v = v.view(rows, nb, b)
    top = v.abs().max(-1).values
    s = 1.0
    if fmt == "mx":
        exps = torch.frexp(top).exponent - 1
        held = torch.exp2(torch.where(top == 0, -127, (exps - 2).clamp(min=-127)).double())
    else:
        most = float(top.max())
        s = float(np.float32(min(max(most / 2688, 2.0 ** -100), 2.0 ** 117))) if most else 1.0
        grid = torch.tensor(_e4m3_grid(), dtype=torch.float64, device=x.device)
        held = grid[_nearest(top / (6 * s), grid)]
    unit = torch.where(held == 0, 1.0, held * s)
    y = torch.where(held[..., None] == 0, 0.0, v.abs() / unit[..., None])
    mag = torch.tensor(GRID, dtype=torch.float64, device=x.device)[_nearest(y, GRID)]
    q = torch.copysign(mag, v) * held[..., None] * s
    return q.view(rows, nb * b)[:, :cols], held, s


def _exact_values(state, cols, fmt):
    codes, scales = state["codes"], state["scales"]
    rows = codes.shape[0]
    grid = torch.tensor(GRID + [-v for v in GRID], dtype=torch.float64, device=codes.device)
    c = torch.empty(rows, codes.shape[1] * 2, dtype=torch.uint8, device=codes.device)
    c[:, 0::2], c[:, 1::2] = codes & 15, codes >> 4
    v = grid[c[:, :cols].int()]
    at = torch.arange(cols, device=codes.device) // BLOCK[fmt]
    if fmt == "mx":
        unit = torch.exp2(scales.double() - 127)
    else:
        grid = torch.tensor(_e4m3_grid(), dtype=torch.float64, device=codes.device)
        unit = grid[scales.int()] * state["tensor_scale"].double()
    return v.mul_(unit[:, at])


def exact(case, seed):
    state = _inputs(case, seed)
    fmt, kind = case["fmt"], case["kind"]
    if kind == "roundtrip":
        v, held, s = _exact_quantise(state["x"], fmt)
        got = {"values": v, "scales": held}
        return {**got, "tensor_scale": torch.tensor([s], dtype=torch.float64)} if fmt == "nv" else got
    if kind == "read":
        return _exact_values(state, case["cols"], fmt)
    w = _exact_values(state, case["k"], fmt)
    x = _exact_quantise(state["x"], fmt)[0] if kind == "linear4" else state["x"].double()
    if case["groups"] == 1:
        return x @ (w if kind == "grad" else w.t())
    out = torch.zeros(case["m"], case["k"] if kind == "grad" else case["n"], dtype=torch.float64, device=x.device)
    off = state["offsets"].tolist()
    for i in range(case["groups"]):
        a, b = off[i], off[i + 1]
        part = w[i * case["n"]:(i + 1) * case["n"]]
        if b > a:
            out[a:b] = x[a:b] @ (part if kind == "grad" else part.t())
    return out


if __name__ == "__main__":
    print(*listed(), *(draw(random.Random(i)) for i in range(6)), sep="\n")
