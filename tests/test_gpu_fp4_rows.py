"""4-bit calls on rows at unusual distances and with unusual neighbours, and of the wrong kind."""
import numpy as np
import pytest
import torch

from bit_exact_xor_amd import dcr
from tests import fp4_ref as R
from tests.test_gpu_fp4 import bound, f64, up

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
