"""4-bit weights on the GPU against a plain 64-bit implementation."""
import numpy as np
import pytest
import torch

from bit_exact_xor_amd import dcr
from tests import fp4_ref as R

pytestmark = pytest.mark.gpu
FORMATS = [R.MX, R.NV]
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def up(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def source(kind, rows, cols, dtype, rng):
    x = rng.standard_normal((rows, cols))
    if kind == "wide":
        x *= 2.0 ** rng.integers(-140, 120, (rows, cols))
    elif kind == "borders":      # values on and next to the borders of the codes
        x = rng.choice([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.9], (rows, cols)) * rng.choice([-1, 1], (rows, cols))
        x *= 1 + rng.integers(-1, 2, (rows, cols)) * 2.0 ** -8
    elif kind == "tiny":         # subnormal numbers and zeros of both signs
        x = rng.integers(-4, 5, (rows, cols)) * 2.0 ** -133
        x[:, ::3] = -0.0
        x[::2] = 0.0
    elif kind == "holes":        # NaN and infinities in some blocks
        m = rng.random((rows, cols))
        x[m < 0.004], x[(m > 0.004) & (m < 0.008)], x[(m > 0.008) & (m < 0.012)] = np.nan, np.inf, -np.inf
    t = torch.from_numpy(x.astype(np.float32)).to(TYPES[dtype])
    return t


KINDS = ["normal", "wide", "borders", "tiny", "holes"]
SHAPES = [(1, 1), (1, 31), (3, 33), (2, 64), (5, 100), (65, 768), (17, 2050), (4, 14336)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", KINDS)
def test_quantize_bytes(fmt, dtype, kind):
    """Codes and scales are the reference's bytes; nothing else is written."""
    rng = np.random.default_rng(KINDS.index(kind))
    for rows, cols in SHAPES:
        x = source(kind, rows, cols, dtype, rng)
        s = [0.0123, 2.0 ** -6, 3.0e-4][cols % 3]
        w, nb = (cols + 1) // 2, dcr.fp4_blocks(cols, fmt)
        for pad in (0, 5, 16):
            codes = torch.full((rows, w + pad), 0xA5, dtype=torch.uint8, device="cuda")
            scales = torch.full((rows, nb + pad), 0x5A, dtype=torch.uint8, device="cuda")
            q = dcr.Fp4Tensor(rows, cols, fmt, codes=codes, scales=scales,
                              tensor_scale=torch.tensor([s], device="cuda"))
            dcr.dcr_fp4_quantize(x.cuda(), q)
            c, b = R.quantize(x.float().numpy(), fmt, s)
            gc, gb = codes.cpu().numpy(), scales.cpu().numpy()
            assert np.array_equal(gb[:, :nb], b), (rows, cols, pad)
            assert np.array_equal(gc[:, :w], c), (rows, cols, pad)
            assert (gc[:, w:] == 0xA5).all() and (gb[:, nb:] == 0x5A).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_quantize_strided_source(fmt, dtype):
    rng = np.random.default_rng(3)
    big = source("normal", 9, 300, dtype, rng).cuda()
    for view in (big[:, 8:200], big[:, 1:130], big[::2, 3:4], big[2:3, 5:], big[:, :256]):
        q = dcr.Fp4Tensor(view.shape[0], view.shape[1], fmt, tensor_scale=torch.tensor([.01], device="cuda"))
        dcr.dcr_fp4_quantize(view, q)
        c, b = R.quantize(view.float().cpu().numpy(), fmt, .01)
        assert np.array_equal(q.scales.cpu().numpy(), b)
        assert np.array_equal(q.codes.cpu().numpy()[:, :c.shape[1]], c)


@pytest.mark.parametrize("s", [0.0, -1.0, float("nan"), float("inf"), 2.0 ** -101, 2.0 ** 118, 2.0 ** -100, 2.0 ** 117,
                               1e-6, 1e3, 0.25])
def test_nv_tensor_scales(s):
    """Outside the range every block is NaN; inside it saturates or vanishes as the reference does."""
    rng = np.random.default_rng(5)
    x = source("normal", 33, 176, "fp32", rng) * (s * 700 if 0 < s < 1 else 1.0)
    q = dcr.Fp4Tensor(33, 176, R.NV, tensor_scale=torch.tensor([s], device="cuda"))
    dcr.dcr_fp4_quantize(x.cuda(), q)
    c, b = R.quantize(x.numpy(), R.NV, s)
    assert np.array_equal(q.scales.cpu().numpy(), b)
    assert np.array_equal(q.codes.cpu().numpy()[:, :c.shape[1]], c)
    if not R.MIN_SCALE <= s <= R.MAX_SCALE:
        assert (b == 127).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (7, 33), (768, 2048), (3, 100001)])
def test_calibrate(dtype, rows, cols):
    rng = np.random.default_rng(rows)
    ws = dcr.fp4_workspace()
    for kind in ("normal", "holes", "zero", "huge"):
        x = source("holes" if kind == "holes" else "normal", rows, cols, dtype, rng)
        x = x * 0 if kind == "zero" else x * 1e37 if kind == "huge" else x
        q = dcr.Fp4Tensor(rows, cols, R.NV, tensor_scale=torch.tensor([float("nan")], device="cuda"))
        dcr.dcr_fp4_quantize(x.cuda(), q, dcr.FP4_CALIBRATE, ws)
        s = R.calibrate(x.float().numpy())
        assert float(q.tensor_scale) == float(s), kind
        c, b = R.quantize(x.float().numpy(), R.NV, s)
        assert np.array_equal(q.scales.cpu().numpy(), b), kind
        assert np.array_equal(q.codes.cpu().numpy()[:, :c.shape[1]], c), kind


def random_fp4(rows, cols, fmt, rng, lo=None, hi=None, s=0.37):
    """Random codes and scale bytes, and their values in fp64 without the tensor scale."""
    w = (cols + 1) // 2
    codes = rng.integers(0, 256, (rows, -(-w // 16) * 16), dtype=np.uint8)
    lo, hi = (lo, hi) if lo is not None else (118, 130) if fmt == R.MX else (40, 80)
    scales = rng.integers(lo, hi + 1, (rows, dcr.fp4_blocks(cols, fmt))).astype(np.uint8)
    q = dcr.Fp4Tensor(rows, cols, fmt, codes=up(codes), scales=up(scales), tensor_scale=torch.tensor([s], device="cuda"))
    return q, R.unit_values(codes, scales, cols, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_dequantize(fmt, dtype):
    """Every scale byte; each value rounded once to fp32, then once to bf16."""
    rng = np.random.default_rng(7)
    B = R.block(fmt)
    for rows, cols in [(256, B), (1, 1), (3, 33), (5, 1999), (64, 768), (2, 16384)]:
        q, v = random_fp4(rows, cols, fmt, rng)
        if rows == 256:
            q.scales.copy_(up(np.arange(256, dtype=np.uint8)[:, None]))
            v = R.unit_values(q.codes.cpu().numpy(), q.scales.cpu().numpy(), cols, fmt)
        with np.errstate(all="ignore"):
            e = v.astype(np.float32)
            if fmt == R.NV:
                e = e * np.float32(0.37)
            e = e.astype(np.float64) if dtype == "fp32" else R.to_bf16(e)
        for pad in (0, 3, 8):
            y = torch.full((rows, cols + pad), 7.0, dtype=TYPES[dtype], device="cuda")
            dcr.dcr_fp4_dequantize(q, y[:, :cols])
            got = f64(y)
            assert np.array_equal(got[:, :cols], e, equal_nan=True), (rows, cols, pad)
            assert np.array_equal(np.signbit(got[:, :cols]) | np.isnan(e), np.signbit(e) | np.isnan(e))
            assert (got[:, cols:] == 7.0).all()


# ------------------------------------------------------------------ products
#
# Two kinds of data.  "whole": x small whole numbers (or quarters, in 4 bits),
# weights multiples of a sixteenth below 2^5, reductions to 4096: every partial
# sum is a multiple of 2^-4 below 2^20, exact in fp32, so fp32 results are
# equal to the reference's in any order.
# "normal": each of the red - 1 additions and the products' alignment rounds
# at most 2^-23 of the running sum of sizes (twice half a step, should the
# instruction truncate), plus the tensor scale's 2^-24 and the result's half
# step.

def whole_fp4(rows, cols, fmt, rng):
    return random_fp4(rows, cols, fmt, rng, 127, 129, 1.0) if fmt == R.MX else random_fp4(rows, cols, fmt, rng, 56, 64, 1.0)


def bound(size, ref, red, dtype):
    b = size * (red + 8) * 2.0 ** -23 + np.abs(ref) * 2.0 ** -24
    return b + np.abs(ref) * (torch.finfo(TYPES[dtype]).eps / 2) + 2.0 ** -126


def run_product(op, x, q, y, off, ws):
    if op == "matmul":
        dcr.dcr_fp4_matmul(x, q, y, off, ws)
    elif op == "grad":
        dcr.dcr_fp4_matmul_grad(x, q, y, off, ws)
    else:
        dcr.dcr_fp4_matmul_q(x, q, y, off, ws)


def check_product(op, fmt, m, n, k, dtype, data, groups=1, off=None, seed=0, x_pad=0, y_pad=0, x_shift=0):
    rng = np.random.default_rng(seed + 1000 * m + n + 7 * k)
    ws = dcr.fp4_workspace()
    q, w = (whole_fp4 if data == "whole" else random_fp4)(n * groups, k, fmt, rng)
    s = 1.0 if fmt == R.MX else float(q.tensor_scale)
    red, outs = (n, k) if op == "grad" else (k, n)
    if op == "matmul_q":
        x, xv = (whole_fp4 if data == "whole" else random_fp4)(m, k, R.MX, rng)
        if data == "whole":
            x, xv = random_fp4(m, k, R.MX, rng, 126, 127)
    else:
        xv = rng.integers(-2, 3, (m, red)).astype(np.float64) if data == "whole" else rng.standard_normal((m, red))
        big = torch.full((m, x_shift + red + x_pad), float("nan"), dtype=torch.bfloat16, device="cuda")
        x = big[:, x_shift:x_shift + red]
        x.copy_(up(xv))
        xv = f64(x)
    y = torch.full((m, outs + y_pad), 99.0, dtype=TYPES[dtype], device="cuda")
    o = None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda")
    run_product(op, x, q, y[:, :outs], o, ws)
    got = f64(y)
    ref, size = R.product(xv, w, off, op == "grad")
    left = np.isnan(ref)
    ref, size = ref * s, size * s
    assert (got[:, outs:] == 99.0).all(), "wrote past the rows' ends"
    assert (got[:, :outs][left] == 99.0).all(), "wrote rows of no group"
    g, r = got[:, :outs][~left], ref[~left]
    if data == "whole" and dtype == "fp32":
        assert np.array_equal(g, r), f"{(g != r).sum()} of {g.size} differ"
    elif data == "whole":
        assert np.array_equal(g, R.to_bf16(r))
    else:
        assert (np.abs(g - r) <= bound(size[~left], r, red, dtype)).all(), np.abs(g - r).max()
    y2 = torch.full_like(y, 99.0)
    run_product(op, x, q, y2[:, :outs], o, ws)
    assert torch.equal(y, y2), "the same call gave other bits"


OPS = [("matmul", R.MX), ("matmul", R.NV), ("matmul_q", R.MX), ("grad", R.MX), ("grad", R.NV)]
SIZES = [(1, 1, 1), (1, 16, 32), (1, 4096, 4096), (2, 100, 2048), (3, 7, 33), (5, 768, 2050), (16, 512, 256), (17, 130, 96),
         (24, 1030, 1024), (33, 64, 4096), (64, 256, 160), (65, 129, 257), (100, 1000, 2080), (128, 128, 128),
         (200, 320, 448), (255, 513, 515), (256, 768, 2048), (300, 2048, 768), (512, 1024, 512), (1030, 300, 288),
         (130, 64, 75), (70, 72, 33), (40, 8, 1), (300, 256, 31)]


@pytest.mark.parametrize("op,fmt", OPS)
@pytest.mark.parametrize("m,n,k", SIZES)
def test_product_whole_numbers(op, fmt, m, n, k):
    check_product(op, fmt, m, n, k, "fp32", "whole")
    check_product(op, fmt, m, n, k, "bf16", "whole", seed=1)


@pytest.mark.parametrize("op,fmt", OPS)
@pytest.mark.parametrize("m,n,k", [(1, 512, 2048), (7, 33, 45), (40, 300, 1000), (300, 520, 640), (513, 1024, 768)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_product_normal(op, fmt, m, n, k, dtype):
    check_product(op, fmt, m, n, k, dtype, "normal")


@pytest.mark.parametrize("op,fmt", OPS)
@pytest.mark.parametrize("x_shift,x_pad,y_pad", [(0, 8, 8), (8, 0, 0), (1, 0, 1), (0, 3, 5), (2, 6, 0)])
def test_product_strides(op, fmt, x_shift, x_pad, y_pad):
    for m, n, k in [(1, 70, 64), (9, 96, 320), (70, 256, 256), (260, 260, 130), (256, 256, 512)]:
        check_product(op, fmt, m, n, k, "fp32", "whole", x_shift=x_shift, x_pad=x_pad, y_pad=y_pad)


@pytest.mark.parametrize("op,fmt", OPS)
@pytest.mark.parametrize("off,m", [([0, 3, 3, 10, 11], 11), ([2, 2, 2, 2, 2], 5), ([5, 70, 70, 400, 420], 450),
                                   ([0, 0, 0, 0, 300], 300), ([0, 256, 512, 768, 1024], 1024), ([1, 2, 3, 4, 5], 9)])
@pytest.mark.parametrize("n,k", [(96, 160), (256, 512), (33, 70)])
def test_product_groups(op, fmt, off, m, n, k):
    check_product(op, fmt, m, n, k, "fp32", "whole", groups=4, off=off)


@pytest.mark.parametrize("op,fmt", OPS)
def test_product_many_groups(op, fmt):
    rng = np.random.default_rng(0)
    counts = rng.integers(0, 5, 200) * rng.integers(0, 3, 200)
    off = np.concatenate([[0], np.cumsum(counts)]).tolist()
    check_product(op, fmt, off[-1] + 2, 48, 64, "fp32", "whole", groups=200, off=off)


@pytest.mark.parametrize("op,fmt", OPS)
def test_product_one_group_with_offsets(op, fmt):
    check_product(op, fmt, 20, 64, 96, "fp32", "whole", groups=1, off=[3, 17])


@pytest.mark.parametrize("op,fmt", OPS)
def test_product_bad_offsets_stay_inside(op, fmt):
    """Offsets outside 0 .. m or descending: held to the buffers; rows around them untouched."""
    rng = np.random.default_rng(1)
    q, _ = whole_fp4(3 * 32, 64, fmt, rng)
    red, outs = (32, 64) if op == "grad" else (64, 32)
    x = random_fp4(20, 64, R.MX, rng)[0] if op == "matmul_q" else torch.ones(20, red, dtype=torch.bfloat16, device="cuda")
    whole = torch.full((60, outs), 5.0, device="cuda")
    y = whole[20:40]
    for off in ([-7, 10, 1000, 2 ** 31 - 1], [19, 3, 8, 2], [-5, -4, -3, -2], [50, 60, 70, 80]):
        run_product(op, x, q, y, torch.tensor(off, dtype=torch.int32, device="cuda"), dcr.fp4_workspace())
        torch.cuda.synchronize()
        assert (whole[:20] == 5.0).all() and (whole[40:] == 5.0).all()


@pytest.mark.parametrize("op,fmt", OPS)
def test_product_empty(op, fmt):
    ws = dcr.fp4_workspace()
    for m, n, k in [(0, 8, 32), (3, 0, 32), (3, 8, 0)]:
        q = dcr.Fp4Tensor(n, k, fmt)
        red, outs = (n, k) if op == "grad" else (k, n)
        x = dcr.Fp4Tensor(m, k, fmt) if op == "matmul_q" else torch.ones(m, red, dtype=torch.bfloat16, device="cuda")
        y = torch.full((m, outs), 4.0, device="cuda")
        run_product(op, x, q, y, None, ws)
        if m and outs:
            assert (y == 0).all()      # a sum of nothing


@pytest.mark.parametrize("op,fmt", OPS)
@pytest.mark.parametrize("m", [1, 40, 300])
def test_product_nan_reaches_its_results_only(op, fmt, m):
    """A NaN scale, and NaN or infinity in x: in the results that use them, nowhere else."""
    rng = np.random.default_rng(2)
    n, k = 288, 320
    q, w = whole_fp4(n, k, fmt, rng)
    q.scales[5, 2] = 255 if fmt == R.MX else 127
    w = R.unit_values(q.codes.cpu().numpy(), q.scales.cpu().numpy(), k, fmt)
    red, outs = (n, k) if op == "grad" else (k, n)
    if op == "matmul_q":
        x, xv = random_fp4(m, k, R.MX, rng, 126, 127)
        x.scales[m - 1, 3] = 255
        xv = R.unit_values(x.codes.cpu().numpy(), x.scales.cpu().numpy(), k, R.MX)
    else:
        xv = rng.integers(1, 3, (m, red)).astype(np.float64)
        xv[m - 1, 3] = np.nan
        xv[m // 2, 7] = np.inf
        x = up(xv).bfloat16()
    y = torch.empty(m, outs, device="cuda")
    run_product(op, x, q, y, None, dcr.fp4_workspace())
    with np.errstate(all="ignore"):
        ref = np.stack([(xv[i][None, :] * (w.T if op == "grad" else w)).sum(-1) for i in range(m)])
    got = f64(y)
    fin = np.isfinite(ref)
    assert np.array_equal(np.isfinite(got), fin)
    assert np.array_equal(got[fin], ref[fin])
    assert np.array_equal(np.isnan(got), np.isnan(ref))


def test_gradient_against_differences():
    """<dx, d> equals the difference quotient of <dy, y(x + h d)> (whole numbers: no rounding anywhere)."""
    rng = np.random.default_rng(4)
    ws = dcr.fp4_workspace()
    for fmt in FORMATS:
        q, _ = whole_fp4(96, 160, fmt, rng)
        x, d = (rng.integers(-1, 2, (13, 160)) for _ in range(2))
        dy = up(rng.integers(-2, 3, (13, 96))).bfloat16()
        ys = []
        for h in (-1, 1):
            y = torch.empty(13, 96, device="cuda")
            dcr.dcr_fp4_matmul(up(x + h * d).bfloat16(), q, y, None, ws)
            ys.append((y.double() * dy.double()).sum().item())
        dx = torch.empty(13, 160, device="cuda")
        dcr.dcr_fp4_matmul_grad(dy, q, dx, None, ws)
        assert (dx.double().cpu().numpy() * d).sum() == (ys[1] - ys[0]) / 2


# ------------------------------------------------- streams, graphs, together

def test_side_stream_and_graph():
    """Quantise, product and gradient on a stream of their own, then captured
    together and replayed between eager calls: every replay gives the eager bits."""
    rng = np.random.default_rng(6)
    ws, ws2 = dcr.fp4_workspace(), dcr.fp4_workspace()
    w = up(rng.standard_normal((512, 640)).astype(np.float32))
    q = dcr.Fp4Tensor(512, 640, R.NV)
    qx, qw = dcr.Fp4Tensor(40, 640, R.MX), dcr.Fp4Tensor(512, 640, R.MX)
    x = torch.empty(40, 640, dtype=torch.bfloat16, device="cuda")
    y, dx, y4 = torch.empty(40, 512, device="cuda"), torch.empty(40, 640, device="cuda"), torch.empty(40, 512, device="cuda")

    def step(work):
        dcr.dcr_fp4_quantize(w, q, dcr.FP4_CALIBRATE, work)
        dcr.dcr_fp4_matmul(x, q, y, None, work)
        dcr.dcr_fp4_matmul_grad(y.bfloat16(), q, dx, None, work)
        dcr.dcr_fp4_quantize(x, qx)
        dcr.dcr_fp4_quantize(w, qw)
        dcr.dcr_fp4_matmul_q(qx, qw, y4, None, work)

    xs = [up(rng.standard_normal((40, 640))).bfloat16() for _ in range(4)]
    want = []
    for v in xs:
        x.copy_(v)
        step(ws)
        want.append([t.clone() for t in (y, dx, y4, q.codes, q.scales)])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        x.copy_(xs[1])
        step(ws)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((y, dx, y4, q.codes, q.scales), want[1]))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(ws2)
    for i in (2, 0, 3, 2):
        x.copy_(xs[i])
        y.zero_(), dx.zero_(), y4.zero_(), q.codes.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((y, dx, y4, q.codes, q.scales), want[i])), i
        step(ws)


def test_stream_argument():
    """An explicit stream orders the call behind that stream's work."""
    s = torch.cuda.Stream()
    q = dcr.Fp4Tensor(64, 128, R.MX)
    with torch.cuda.stream(s):
        x = torch.zeros(64, 128, device="cuda")
        for _ in range(50):
            x += 1
    dcr.dcr_fp4_quantize(x, q, stream=s)
    y = torch.empty(64, 128, device="cuda")
    dcr.dcr_fp4_dequantize(q, y, stream=s)
    s.synchronize()
    c, b = R.quantize(np.full((64, 128), 50.0), R.MX)
    assert np.array_equal(q.scales.cpu().numpy(), b)
    assert np.array_equal(f64(y), R.unit_values(c, b, 128, R.MX))


def test_far_offsets():
    """Rows past 2^32 bytes into codes, x and results."""
    rng = np.random.default_rng(8)
    rows, cols = 3, 96
    stride = (1 << 31) + 64
    codes = torch.empty(2 * stride + 64, dtype=torch.uint8, device="cuda").as_strided((rows, 64), (stride, 1))
    scales = torch.empty(2 * stride + 64, dtype=torch.uint8, device="cuda").as_strided((rows, 6), (stride, 1))
    x = source("normal", rows, cols, "bf16", rng)
    q = dcr.Fp4Tensor(rows, cols, R.NV, codes=codes, scales=scales, tensor_scale=torch.tensor([.01], device="cuda"))
    xs = torch.empty(2 * (1 << 30) + 4096, dtype=torch.bfloat16, device="cuda").as_strided((rows, cols), (1 << 30, 1))
    xs.copy_(x)
    dcr.dcr_fp4_quantize(xs, q)
    c, b = R.quantize(x.float().numpy(), R.NV, .01)
    assert np.array_equal(codes.cpu().numpy()[:, :48], c) and np.array_equal(scales.cpu().numpy(), b)
    y = torch.empty(2 * (1 << 30) + 4096, dtype=torch.float32, device="cuda").as_strided((rows, rows), (1 << 30, 1))
    dcr.dcr_fp4_matmul(xs, q, y, None, dcr.fp4_workspace())
    w = R.unit_values(c, b, cols, R.NV)
    ref, size = R.product(f64(x), w)
    assert (np.abs(f64(y) - ref * .01) <= bound(size * .01, ref * .01, cols, "fp32") + np.abs(ref) * 1e-9).all()


# -------------------------------------------------------------- refit in 4 bits

@pytest.mark.parametrize("fmt", FORMATS)
def test_refit_then_product(fmt):
    """Quantise, encode, transfer, apply in place, multiply: after every refit
    the receiver holds the sender's bytes and its products are the sender's."""
    from bit_exact_xor_amd import pipeline
    rng = np.random.default_rng(9)
    shapes = [(768, 2048), (130, 96), (33, 70), (512, 512)]
    link = pipeline.Fp4Refit(shapes, fmt)
    w = [up((0.02 * rng.standard_normal(s)).astype(np.float32)) for s in shapes]
    sent = []
    for step in range(4):
        if step:
            for t in w:      # a small update of some of the weights, as a training step makes
                t += up((rng.random(t.shape) < 0.02) * rng.choice([-1, 1], t.shape) * 2e-3).float()
        sent.append(link.refit([w[0].bfloat16()] + w[1:], calibrate=step == 3))
        assert link.version == step + 1
        for i, (t, s) in enumerate(zip(w, shapes)):
            src = (w[0].bfloat16() if i == 0 else t).float().cpu().numpy()
            sc = 1.0 if fmt == R.MX else float(link.held[i].tensor_scale)
            if fmt == R.NV and step in (0, 3):
                assert sc == float(R.calibrate(src))
            c, b = R.quantize(src, fmt, sc)
            assert np.array_equal(link.held[i].codes.cpu().numpy()[:, :c.shape[1]], c)
            assert np.array_equal(link.held[i].scales.cpu().numpy(), b)
            assert torch.equal(link.held[i].codes, link.sent[i].codes)
            x = up(rng.integers(-2, 3, (5, s[1]))).bfloat16()
            y = torch.empty(5, s[0], device="cuda")
            dcr.dcr_fp4_matmul(x, link.sent[i], y, None, link.fp4_workspace)
            assert torch.equal(link.matmul(i, x, torch.float32), y)
            ref, size = R.product(f64(x), R.unit_values(c, b, s[1], fmt))
            assert (np.abs(f64(y) - ref * sc) <= bound(size * sc, ref * sc, s[1], "fp32")).all()
    assert sent[1] < sent[0] / 4 and sent[2] < sent[0] / 4      # 2 % of elements moved: few bytes travel
    with pytest.raises(ValueError):
        link.refit(w[:2])


def test_refit_of_unchanged_weights_sends_nothing():
    from bit_exact_xor_amd import pipeline
    link = pipeline.Fp4Refit([(64, 96)], R.NV)
    w = [torch.ones(64, 96, device="cuda")]
    assert link.refit(w) > 0
    assert link.refit(w) == 0 and link.refit(w) == 0


def test_refit_of_experts():
    """A stack of experts, refitted and multiplied by groups."""
    from bit_exact_xor_amd import pipeline
    rng = np.random.default_rng(11)
    link = pipeline.Fp4Refit([(8 * 48, 64)], R.MX)
    w = up(rng.standard_normal((8 * 48, 64)).astype(np.float32))
    off = [0, 3, 3, 10, 11, 40, 41, 60, 64]
    x = up(rng.integers(-2, 3, (64, 64))).bfloat16()
    for _ in range(2):
        link.refit([w])
        c, b = R.quantize(w.cpu().numpy(), R.MX)
        y = link.matmul(0, x, torch.float32, torch.tensor(off, dtype=torch.int32, device="cuda"))
        ref, size = R.product(f64(x), R.unit_values(c, b, 64, R.MX), off)
        assert (np.abs(f64(y) - ref) <= bound(size, ref, 64, "fp32")).all()
        w = w * 1.01


@pytest.mark.parametrize("op,fmt", OPS[:3])
@pytest.mark.parametrize("m,n,k", [(1, 14336, 2304), (16, 12400, 2592), (11, 6500, 4064), (8, 6400, 2304), (4, 1000, 3616),
                                   (13, 4096, 4096), (16, 16400, 512)])
def test_product_few_rows(op, fmt, m, n, k):
    """Wide and narrow weights, sums of several turns of a wave, scales with and without borders of their own."""
    check_product(op, fmt, m, n, k, "fp32", "whole")
    check_product(op, fmt, m, n, k, "bf16", "normal")


@pytest.mark.parametrize("op,fmt", OPS[:3])
@pytest.mark.parametrize("n,k", [(1024, 2304), (1650, 2080), (96, 4096), (3000, 512)])
def test_product_few_rows_of_groups(op, fmt, n, k):
    check_product(op, fmt, 33, n, k, "fp32", "whole", groups=8, off=[1, 1, 5, 23, 24, 24, 24, 30, 31])
    check_product(op, fmt, 2, n, k, "fp32", "whole", groups=8, off=[0, 0, 0, 1, 1, 1, 2, 2, 2])


def test_tensor_keeps_its_buffers():
    q = dcr.Fp4Tensor(4, 64)
    for name in ("codes", "scales", "tensor_scale", "rows"):
        with pytest.raises(AttributeError):
            setattr(q, name, None)


def padded(q, code_pad, scale_pad):
    """q in buffers with longer rows; what lies between its rows must not matter."""
    rows, w, nb = q.rows, (q.cols + 1) // 2, dcr.fp4_blocks(q.cols, q.fmt)
    codes = torch.full((rows, w + code_pad), 0x77, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, nb + scale_pad), 255 if q.fmt == R.MX else 127, dtype=torch.uint8, device="cuda")
    codes[:, :w], scales[:, :nb] = q.codes[:, :w], q.scales[:, :nb]
    if q.cols % 2:
        codes[:, w - 1] |= 0x70
    return dcr.Fp4Tensor(rows, q.cols, q.fmt, codes=codes, scales=scales, tensor_scale=q.tensor_scale)


@pytest.mark.parametrize("op,fmt", OPS)
@pytest.mark.parametrize("m", [2, 20, 70, 300])
def test_product_weight_strides(op, fmt, m):
    """Rows of codes and scales at any distance, on borders of 8 and 16 bytes among them, NaN scales between them."""
    rng = np.random.default_rng(m)
    ws = dcr.fp4_workspace()
    for n, k in [(100, 96), (130, 384), (300, 640), (257, 289), (64, 4000), (280, 2336)]:
        q, w = whole_fp4(n, k, fmt, rng)
        red, outs = (n, k) if op == "grad" else (k, n)
        if op == "matmul_q":
            x, xv = random_fp4(m, k, R.MX, rng, 126, 127)
        else:
            xv = rng.integers(-2, 3, (m, red)).astype(np.float64)
            x = up(xv).bfloat16()
        want = R.product(xv, w, None, op == "grad")[0]
        nb, cb = dcr.fp4_blocks(k, fmt), (k + 1) // 2
        for code_pad, scale_pad in [(0, 1), (1, 0), (-cb % 16, 3), (-cb % 16, -nb % 16), (-cb % 16 + 16, -nb % 8 + 8), (8, 5)]:
            y = torch.full((m, outs), 9.0, device="cuda")
            v = padded(x, -cb % 16, -nb % 8 + (scale_pad & 8)) if op == "matmul_q" else x
            run_product(op, v, padded(q, code_pad, scale_pad), y, None, ws)
            assert np.array_equal(f64(y), want), (n, k, code_pad, scale_pad)


@pytest.mark.parametrize("op", ["matmul", "matmul_q", "grad"])
def test_longest_sums(op):
    """One row of 2^26 elements, the first length the tiles leave, against one that they take."""
    for red in (1 << 26, (1 << 26) - 256):
        rows, cols = (red, 32) if op == "grad" else (1, red)
        q = dcr.Fp4Tensor(rows, cols, R.MX)
        q.codes.fill_(0x22), q.scales.fill_(127)           # ones
        x = torch.zeros(1, red, dtype=torch.bfloat16, device="cuda")
        x[0, ::1 << 18] = 1.0
        x[0, red - 1] = 3.0
        if op == "matmul_q":
            v = dcr.Fp4Tensor(1, red, R.MX)
            dcr.dcr_fp4_quantize(x, v)
            x = v
        y = torch.full((1, 32 if op == "grad" else 1), 9.0, device="cuda")
        run_product(op, x, q, y, None, dcr.fp4_workspace())
        assert (y == 256 + 3).all()
        del q, x


@pytest.mark.parametrize("op,fmt", OPS)
@pytest.mark.parametrize("k", [8, 1000, 1016, 1048, 1304])
def test_product_sums_of_whole_pieces(op, fmt, k):
    """Sums that end inside a block, rows of x on 16-byte borders all the same."""
    for m, n in [(3, 40), (24, 136), (70, 1000), (280, 264)]:
        check_product(op, fmt, m, n, k, "fp32", "whole")
        check_product(op, fmt, m, k, n, "fp32", "whole", x_pad=-k % 8)


@pytest.mark.parametrize("m", [6, 150])
def test_graph_of_groups(m):
    """Captured products of experts, replayed with other rows and other offsets: the eager bits every time."""
    rng = np.random.default_rng(m)
    ws, ws2 = dcr.fp4_workspace(), dcr.fp4_workspace()
    q, _ = whole_fp4(8 * 320, 448, R.NV, rng)
    qm, _ = whole_fp4(8 * 320, 448, R.MX, rng)
    x, off = torch.empty(m, 448, dtype=torch.bfloat16, device="cuda"), torch.zeros(9, dtype=torch.int32, device="cuda")
    x4 = dcr.Fp4Tensor(m, 448)
    y, dx, y4 = (torch.empty(m, n, device="cuda") for n in (320, 448, 320))

    def step(work):
        dcr.dcr_fp4_matmul(x, q, y, off, work)
        dcr.dcr_fp4_matmul_grad(y.bfloat16(), q, dx, off, work)
        dcr.dcr_fp4_quantize(x, x4)
        dcr.dcr_fp4_matmul_q(x4, qm, y4, off, work)

    def fill(i):
        r = np.random.default_rng(100 * m + i)
        cuts = np.sort(r.integers(0, m + 1, 7)) if i else np.full(7, m)
        off.copy_(up(np.concatenate([[0], cuts, [m]]).astype(np.int32)))
        x.copy_(up(r.standard_normal((m, 448))))
        y.zero_(), dx.zero_(), y4.zero_()

    fill(0)
    step(ws2)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(ws2)
    for i in (1, 0, 2, 3, 1):
        fill(i)
        step(ws)
        want = [t.clone() for t in (y, dx, y4)]
        fill(i)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((y, dx, y4), want)), i
