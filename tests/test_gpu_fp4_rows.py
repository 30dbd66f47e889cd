"""4-bit calls on rows at unusual distances and with unusual neighbours, and of the wrong kind."""
import numpy as np
import pytest
import torch

from bit_exact_xor_amd import dcr
from tests import fp4_ref as R
from tests.test_gpu_fp4 import bound, f64, padded, random_fp4, run_product, up

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [R.MX, R.NV])
def test_one_row_at_any_stride(fmt):
    """A single row has no next one: its strides are not looked at."""
    k = 96
    far = lambda t: t.as_strided((1, t.shape[1]), (1 << 41, 1))     # noqa: E731
    q = dcr.Fp4Tensor(1, k, fmt, codes=far(torch.zeros(1, 48, dtype=torch.uint8, device="cuda")),
                      scales=far(torch.zeros(1, 6, dtype=torch.uint8, device="cuda")),
                      tensor_scale=torch.tensor([0.01], device="cuda"))
    x = far(up(np.random.default_rng(1).standard_normal((1, k))).bfloat16())
    dcr.dcr_fp4_quantize(x, q)
    c, b = R.quantize(f64(x), fmt, 0.01)
    assert np.array_equal(q.codes.cpu().numpy(), c) and np.array_equal(q.scales.cpu().numpy()[:, :b.shape[1]], b)
    y = far(torch.empty(1, k, device="cuda"))
    dcr.dcr_fp4_dequantize(q, y)
    v = R.unit_values(c, b, k, fmt)
    s = np.float32(0.01) if fmt == R.NV else np.float32(1)
    assert np.array_equal(f64(y), (v.astype(np.float32) * s).astype(np.float64))
    r = far(torch.empty(1, 1, device="cuda"))
    dcr.dcr_fp4_matmul(x, q, r, None, dcr.fp4_workspace())
    ref, size = R.product(f64(x), v)
    assert (np.abs(f64(r) - ref * s) <= bound(size * s, ref * s, k, "fp32")).all()


# ------------------------------------------------------------- what lies behind a row

@pytest.mark.parametrize("op", ["matmul", "matmul_q", "grad"])
@pytest.mark.parametrize("byte", [253, 254])
@pytest.mark.parametrize("m,n,k", [(3, 136, 40), (3, 96, 77), (20, 136, 2088), (70, 300, 1000), (70, 300, 1001), (4100, 136, 40),
                                   (4100, 136, 335), (8200, 136, 104), (8200, 136, 105), (4100, 1000, 40), (4100, 1000, 296)])
def test_codes_behind_a_row(op, byte, m, n, k):
    """Sums that end inside a block of the largest scales: the codes between rows, which such a scale takes past
    bf16's range, do not matter.  (Codes up to 1.5 in the rows themselves: times 2^127 still finite.)"""
    rng = np.random.default_rng(byte + m + k)
    w = (k + 1) // 2
    pick = np.array([0, 1, 2, 3, 8, 9, 10, 11], dtype=np.uint8)
    codes = pick[rng.integers(0, 8, (n, w))] | pick[rng.integers(0, 8, (n, w))] << 4
    scales = np.full((n, dcr.fp4_blocks(k, R.MX)), byte, dtype=np.uint8)
    values = R.unit_values(codes, scales, k, R.MX)
    q = padded(dcr.Fp4Tensor(n, k, R.MX, codes=up(codes), scales=up(scales)), -w % 16, -scales.shape[1] % 8 + 8)
    red, outs = (n, k) if op == "grad" else (k, n)
    if op == "matmul_q":
        x, xv = random_fp4(m, k, R.MX, rng, 27, 27)
    else:
        xv = rng.integers(-2, 3, (m, red)) * 2.0 ** -100
        x = up(xv).bfloat16()
    y = torch.empty(m, outs, device="cuda")
    run_product(op, x, q, y, None, dcr.fp4_workspace())
    assert np.array_equal(f64(y), R.product(xv, values, None, op == "grad")[0])


@pytest.mark.parametrize("op", ["matmul", "matmul_q", "grad"])
@pytest.mark.parametrize("m", [2, 70, 300])
@pytest.mark.parametrize("byte,code", [(252, 7), (253, 5), (253, 6), (254, 3), (254, 4), (254, 7),
                                       (0, 1), (0, 3), (0, 7), (1, 1), (1, 2), (2, 1)])
def test_weights_at_the_ends_of_the_range(op, m, byte, code):
    """Scale bytes 253 and 254: values from 2^128 on are infinities to the products that take weights as bf16, as they
    are when read back; the product of two 4-bit operands scales exactly.  Bytes 0 to 2: values below the normal
    numbers, down to 2^-128, are kept."""
    n = k = 96
    codes = np.zeros((n, k // 2), dtype=np.uint8)
    codes[np.arange(n), np.arange(n) // 2] = code << 4 * (np.arange(n) % 2)      # one in each row and column
    scales = np.full((n, 3), byte, dtype=np.uint8)
    q = dcr.Fp4Tensor(n, k, R.MX, codes=up(codes), scales=up(scales))
    back = torch.empty(n, k, dtype=torch.bfloat16, device="cuda")
    dcr.dcr_fp4_dequantize(q, back)
    v, e = R.GRID[code] * 2.0 ** (byte - 127), -100 if byte > 127 else 100
    assert (f64(back).diagonal() == (v if v < 2.0 ** 128 else np.inf)).all()
    if op == "matmul_q":
        ones = np.full((m, k // 2), 0x22, dtype=np.uint8)
        x = dcr.Fp4Tensor(m, k, R.MX, codes=up(ones), scales=up(np.full((m, 3), 127 + e, dtype=np.uint8)))
        want = v * 2.0 ** e
    else:
        x = torch.full((m, k), 2.0 ** e, dtype=torch.bfloat16, device="cuda")
        want = v * 2.0 ** e if v < 2.0 ** 128 else np.inf
    y = torch.empty(m, n, device="cuda")
    run_product(op, x, q, y, None, dcr.fp4_workspace())
    assert (f64(y) == want).all()


def test_calls_of_the_wrong_kind():
    """4-bit rows for a call that takes bf16 ones, matrices of other dimensions, workspaces with gaps: refused."""
    q, ws = dcr.Fp4Tensor(64, 96), dcr.fp4_workspace()
    x = dcr.Fp4Tensor(8, 96)
    with pytest.raises(ValueError):
        dcr.dcr_fp4_matmul(x, q, torch.empty(8, 64, device="cuda"), None, ws)
    with pytest.raises(ValueError):
        dcr.dcr_fp4_matmul_grad(dcr.Fp4Tensor(8, 64), q, torch.empty(8, 96, device="cuda"), None, ws)
    for bad in (torch.zeros((), dtype=torch.bfloat16, device="cuda"), torch.zeros(96, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(2, 8, 96, dtype=torch.bfloat16, device="cuda")):
        with pytest.raises(ValueError):
            dcr.dcr_fp4_matmul(bad, q, torch.empty(8, 64, device="cuda"), None, ws)
    gaps = torch.empty(2 * dcr.FP4_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")[::2]
    with pytest.raises(ValueError):
        dcr.dcr_fp4_matmul(torch.zeros(8, 96, dtype=torch.bfloat16, device="cuda"), q, torch.empty(8, 64, device="cuda"), None, gaps)
    with pytest.raises(ValueError):
        dcr.dcr_fp4_quantize(torch.zeros(8, 96, device="cuda"), dcr.Fp4Tensor(8, 96, R.NV), dcr.FP4_CALIBRATE, gaps)
