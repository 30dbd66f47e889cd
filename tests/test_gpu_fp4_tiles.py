"""4-bit products through every tile of their kernels, against the plain 64-bit implementation.

A call's sizes, strides and groups choose its kernel, its tile and the parts of its sum; the sizes here are chosen so
that each tile of each kernel is taken, whole, less than half full at the end, by groups, and with the sum in parts."""
import numpy as np
import pytest
import torch

from bit_exact_xor_amd import dcr
from tests import fp4_ref as R
from tests.test_gpu_fp4 import OPS, TYPES, bound, f64, padded, random_fp4, run_product, up, whole_fp4

pytestmark = pytest.mark.gpu


def cut(m, groups):
    """Offsets of `groups` ranges over most of m rows: an empty one, one of one row, ragged ones; rows outside at both ends."""
    if groups == 1:
        return None
    r = np.random.default_rng(m)
    inner = np.sort(r.integers(3, m - 4, groups - 3))
    return [2, 2, 3, *inner.tolist(), m - 3]


def check(op, fmt, m, n, k, groups=1, x_shift=0, code_pad=None):
    """Whole numbers (exact in any order) as fp32, then normal ones as bf16; equal bits on a second call.
    x_shift: rows of x off their 16-byte borders; code_pad: bytes between rows of codes (None: rows padded to 16)."""
    red, outs = (n, k) if op == "grad" else (k, n)
    off = cut(m, groups)
    o = None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda")
    ws = dcr.fp4_workspace()
    rng = np.random.default_rng(m + 3 * n + 7 * k + groups)
    for data, dtype in (("whole", "fp32"), ("normal", "bf16")):
        q, w = (whole_fp4 if data == "whole" else random_fp4)(n * groups, k, fmt, rng)
        s = 1.0 if fmt == R.MX else float(q.tensor_scale)
        if code_pad is not None:
            q = padded(q, code_pad, 0)
        if op == "matmul_q":
            x, xv = random_fp4(m, k, R.MX, rng, 126, 127) if data == "whole" else random_fp4(m, k, R.MX, rng)
            x = padded(x, 1, 0) if x_shift else x
        else:
            xv = rng.integers(-2, 3, (m, red)) if data == "whole" else rng.standard_normal((m, red))
            stride = x_shift + red + (-red % 8 if not x_shift else 0)
            x = torch.full((m, stride), float("nan"), dtype=torch.bfloat16, device="cuda")[:, x_shift:x_shift + red]
            x.copy_(up(xv))
            xv = f64(x)
        y = torch.full((m, outs), 99.0, dtype=TYPES[dtype], device="cuda")
        run_product(op, x, q, y, o, ws)
        got = f64(y)
        ref, size = R.product(xv, w, off, op == "grad")
        left = np.isnan(ref)
        assert (got[left] == 99.0).all(), "wrote rows of no group"
        g, r, size = got[~left], ref[~left] * s, size[~left] * s
        if data == "whole":
            assert np.array_equal(g, r), f"{(g != r).sum()} of {g.size} differ"
        else:
            assert (np.abs(g - r) <= bound(size, r, red, dtype)).all(), np.abs(g - r).max()
        y2 = torch.full_like(y, 99.0)
        run_product(op, x, q, y2, o, ws)
        assert torch.equal(y, y2), "the same call gave other bits"


# rows, results and length of the sum, with the tile's rows and whether the sum is in parts
TILES = [
    (20, 136, 520), (20, 136, 512), (20, 136, 1536), (130, 64, 1536),       # 32; 32 in parts
    (4100, 136, 520), (4100, 136, 256), (700, 136, 4096), (1500, 136, 2048),    # 64; 64 in parts
    (8200, 136, 264), (8200, 136, 512), (4100, 136, 4096),                  # 128; 128 in parts
    (4100, 1000, 136), (4100, 1000, 256), (4100, 1000, 512), (8200, 136, 4096),  # 256; 256 in parts
    (20, 136, 536), (4100, 136, 536), (8200, 136, 280), (4100, 1000, 152),  # NV scales two at a time, 32 to 256
    (1500, 4104, 264),
]
# the gradient's tiles are smaller for a sum as long
GRAD_TILES = [
    (20, 136, 136), (20, 72, 1000),                                         # 32; 32 in parts
    (4100, 136, 136), (700, 136, 2048), (400, 136, 2048),                   # 64; 64 in parts
    (8200, 136, 200), (8200, 136, 328), (2050, 136, 4096), (4100, 64, 4096),    # 128; 128 in parts
    (4100, 1000, 136), (4100, 1000, 328), (1500, 4104, 200), (8200, 136, 4096),  # 256; 256 in parts
    (3000, 136, 2048), (1030, 136, 2048),
]
CASES = [(op, fmt, m, outs, red) for op, fmt in OPS for m, outs, red in (GRAD_TILES if op == "grad" else TILES)]


MODEST = [c for c in CASES if c[2] * c[3] * c[4] < 2e9]


def sizes(op, outs, red):
    return (red, outs) if op == "grad" else (outs, red)


@pytest.mark.parametrize("op,fmt,m,outs,red", CASES)
def test_tiles(op, fmt, m, outs, red):
    check(op, fmt, m, *sizes(op, outs, red))


@pytest.mark.parametrize("op,fmt,m,outs,red", CASES)
def test_tiles_of_groups(op, fmt, m, outs, red):
    check(op, fmt, m, *sizes(op, outs, red), groups=8)


@pytest.mark.parametrize("op,fmt,m,outs,red", MODEST)
def test_tiles_of_rows_anywhere(op, fmt, m, outs, red):
    check(op, fmt, m, *sizes(op, outs, red + 1), groups=4 if m == 4100 else 1, x_shift=1)


@pytest.mark.parametrize("op,fmt,m,outs,red", MODEST)
def test_tiles_of_codes_anywhere(op, fmt, m, outs, red):
    n, k = sizes(op, outs, red)
    check(op, fmt, m, n, k, groups=5 if m > 1000 else 1, code_pad=1 if (k + 1) // 2 % 16 != 15 else 2)


# ------------------------------------------------------------- the general kernel

@pytest.mark.parametrize("op,fmt", [("matmul", R.MX), ("matmul", R.NV), ("grad", R.MX), ("grad", R.NV)])
@pytest.mark.parametrize("red", [1, 2, 5, 7])
@pytest.mark.parametrize("groups", [1, 6])
def test_short_sums(op, fmt, red, groups):
    """Sums below eight: several row and column tiles of the kernel that takes what the others do not, with and
    without groups (empty ones and one of a single row among them)."""
    for m, outs in ((200, 200), (65, 129), (1, 300)):
        if groups > 1 and m < 10:
            continue
        check(op, fmt, m, *sizes(op, outs, red), groups=groups)


@pytest.mark.parametrize("op,fmt", OPS)
@pytest.mark.parametrize("groups", [1, 5])
def test_far_rows(op, fmt, groups):
    """Row strides that the tiles do not take, several tiles each way, sums of several steps."""
    m, n, k = 150, 135, 200
    rng = np.random.default_rng(groups)
    q, w = whole_fp4(n * groups, k, fmt, rng)
    red, outs = (n, k) if op == "grad" else (k, n)
    if op == "matmul_q":
        stride = 1 << 22
        x, xv = random_fp4(m, k, R.MX, rng, 126, 127)
        codes = torch.empty((m - 1) * stride + 112, dtype=torch.uint8, device="cuda").as_strided((m, 112), (stride, 1))
        codes.copy_(x.codes)
        x = dcr.Fp4Tensor(m, k, R.MX, codes=codes, scales=x.scales)
    else:
        stride = 1 << 21
        xv = rng.integers(-2, 3, (m, red)).astype(np.float64)
        x = torch.empty((m - 1) * stride + red, dtype=torch.bfloat16, device="cuda").as_strided((m, red), (stride, 1))
        x.copy_(up(xv))
    off = cut(m, groups)
    o = None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda")
    ref = R.product(xv, w, off, op == "grad")[0]
    left = np.isnan(ref)
    for dtype in TYPES.values():
        y = torch.full((m, outs), 99.0, dtype=dtype, device="cuda")
        run_product(op, x, q, y, o, dcr.fp4_workspace())
        got, want = f64(y), ref if dtype == torch.float32 else R.to_bf16(ref)
        assert (got[left] == 99.0).all()
        assert np.array_equal(got[~left], want[~left])


def test_general_kernel_walks_its_grid():
    """More 64 x 64 tiles than the grid has workgroups (2^20): every one is computed."""
    m, n = 65600, 66000
    rng = np.random.default_rng(0)
    q, w = whole_fp4(n, 1, R.MX, rng)
    x = up(rng.integers(-2, 3, (m, 1))).bfloat16()
    y = torch.full((m, n), 99.0, dtype=torch.bfloat16, device="cuda")
    dcr.dcr_fp4_matmul(x, q, y, None, dcr.fp4_workspace())
    wv = up(w[:, 0]).float()
    for i in range(0, m, 8200):
        assert torch.equal(y[i:i + 8200], (x[i:i + 8200].float() * wv).bfloat16()), i
