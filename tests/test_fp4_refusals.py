"""Refusals of the 4-bit weight calls (no GPU: they are made before any launch)."""
import ctypes
import os
import re

import pytest
import torch

from bit_exact_xor_amd import dcr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
AT = 1 << 20            # an aligned address that is never read
WS = dcr.FP4_WORKSPACE_BYTES


def desc(rows=64, cols=64, fmt=0, codes=AT, scales=AT, ts=AT, cs=32, ss=4, reserved=0):
    return dcr.Fp4Desc(codes, scales, ts, rows, cols, cs, ss, fmt, reserved)


def ref(d):
    return None if d is None else ctypes.addressof(d)


def quantize(d=desc(), x=AT, ty=0, stride=64, opt=0, ws=None, n=0):
    return dcr.load_library().dcr_fp4_quantize(x, ty, stride, ref(d), opt, ws, n, None)


def dequantize(d=desc(), y=AT, ty=0, stride=64):
    return dcr.load_library().dcr_fp4_dequantize(ref(d), y, ty, stride, None)


def matmul(d=desc(), x=AT, m=4, xs=64, off=None, g=1, y=AT, ty=0, ys=64, ws=AT, n=WS, grad=False):
    lib = dcr.load_library()
    return (lib.dcr_fp4_matmul_grad if grad else lib.dcr_fp4_matmul)(x, m, xs, ref(d), off, g, y, ty, ys, ws, n, None)


def matmul_q(x=desc(), d=desc(), off=None, g=1, y=AT, ty=0, ys=64, ws=AT, n=WS):
    return dcr.load_library().dcr_fp4_matmul_q(ref(x), ref(d), off, g, y, ty, ys, ws, n, None)


BAD_TENSORS = [None, desc(fmt=2), desc(reserved=1), desc(codes=None), desc(scales=None), desc(codes=AT + 8),
               desc(scales=AT + 1), desc(cs=31), desc(ss=1), desc(fmt=1, ss=3), desc(fmt=1, ts=None),
               desc(fmt=1, ts=AT + 2), desc(cols=1 << 31), desc(rows=1 << 40), desc(cs=1 << 32), desc(ss=1 << 32)]


@pytest.mark.parametrize("i", range(len(BAD_TENSORS)))
def test_bad_tensors(i):
    d = BAD_TENSORS[i]
    for rc in (quantize(d), dequantize(d), matmul(d), matmul(d, grad=True), matmul_q(desc(), d), matmul_q(d, desc())):
        assert rc == dcr.DCR_E_INVAL
        assert dcr.load_library().dcr_last_error()


def test_bad_quantize_arguments():
    nv = desc(fmt=1)
    for kw in (dict(x=None), dict(x=AT + 2), dict(x=AT + 1, ty=1), dict(ty=2), dict(stride=63), dict(stride=1 << 40),
               dict(opt=2), dict(opt=1), dict(d=nv, opt=1), dict(d=nv, opt=1, ws=AT + 8, n=4096)):
        assert quantize(**kw) == dcr.DCR_E_INVAL, kw
    assert quantize(nv, opt=1, ws=AT, n=4095) == dcr.DCR_E_CAPACITY
    for kw in (dict(y=None), dict(y=AT + 2), dict(ty=7), dict(stride=10)):
        assert dequantize(**kw) == dcr.DCR_E_INVAL, kw


@pytest.mark.parametrize("grad", [False, True])
def test_bad_product_arguments(grad):
    for kw in (dict(x=None), dict(x=AT + 1), dict(xs=63), dict(g=0), dict(g=3, off=AT), dict(g=2), dict(g=2, off=AT + 2),
               dict(y=None), dict(y=AT + 2), dict(ty=2), dict(ys=63), dict(ws=None), dict(ws=AT + 4), dict(m=1 << 31),
               dict(d=desc(rows=1 << 31)), dict(d=desc(rows=1 << 20), g=1 << 18, off=AT)):
        assert matmul(grad=grad, **kw) == dcr.DCR_E_INVAL, kw
    assert matmul(grad=grad, n=WS - 1) == dcr.DCR_E_CAPACITY


def test_bad_product_of_two():
    assert matmul_q(d=desc(fmt=1)) == dcr.DCR_E_INVAL
    assert matmul_q(x=desc(fmt=1)) == dcr.DCR_E_INVAL
    assert matmul_q(x=desc(cols=32)) == dcr.DCR_E_INVAL
    assert matmul_q(n=0) == dcr.DCR_E_CAPACITY


@pytest.mark.parametrize("ts", [None, AT + 2])
def test_bad_scale_of_empty_sums(ts):
    """Weights without columns (the gradient: without rows) still give results, zeros, and the kernels read the tensor
    scale for them; with no results nothing is read."""
    for kw in (dict(d=desc(cols=0, fmt=1, ts=ts)), dict(d=desc(rows=0, fmt=1, ts=ts), grad=True),
               dict(d=desc(rows=0, fmt=1, ts=ts), grad=True, g=4, off=AT)):
        assert matmul(**kw) == dcr.DCR_E_INVAL, kw
        assert b"tensor scale" in dcr.load_library().dcr_last_error()
        assert matmul(m=0, **kw) == dcr.DCR_OK, kw
    assert matmul(desc(rows=0, fmt=1, ts=ts)) == dcr.DCR_OK
    assert matmul(desc(cols=0, fmt=1, ts=ts), grad=True) == dcr.DCR_OK
    assert quantize(desc(rows=0, fmt=1, ts=ts)) == dcr.DCR_OK and dequantize(desc(cols=0, fmt=1, ts=ts)) == dcr.DCR_OK


def test_strides_of_one_row():
    """A single row's strides are not looked at; those of two are."""
    for kw in (dict(cs=1 << 32), dict(ss=1 << 40), dict(cs=0, ss=0)):
        assert matmul(desc(rows=1, **kw), m=0) == dcr.DCR_OK, kw
        assert matmul(desc(rows=2, **kw), m=0) == dcr.DCR_E_INVAL, kw


def test_binding_refuses():
    """Python-side checks: host tensors, shapes and types, before the library is called."""
    with pytest.raises(ValueError):
        dcr.Fp4Tensor(4, 64, device="cpu")
    with pytest.raises(ValueError):
        dcr.Fp4Tensor(4, 64, 5, device="cpu")
    with pytest.raises(ValueError):
        dcr.Fp4Tensor(4, 64, codes=torch.zeros(4, 31, dtype=torch.uint8), scales=torch.zeros(4, 2, dtype=torch.uint8))
    with pytest.raises(ValueError):
        dcr.Fp4Tensor(4, 64, codes=torch.zeros(4, 32), scales=torch.zeros(4, 2, dtype=torch.uint8))
    for bad in (torch.zeros(4, 64, dtype=torch.float16), torch.zeros(4, 63), torch.zeros(5, 64), torch.zeros(64, 4).t(),
                torch.zeros(1, 64).expand(4, 64)):
        with pytest.raises(ValueError):
            dcr._wide(bad, 4, 64, "x")
    assert dcr._wide(torch.zeros(4, 64), 4, 64, "x")[1:] == (dcr.F32, 64)


def test_header_exports():
    """Every 4-bit call of the header is exported, and the constants agree."""
    text = open(os.path.join(ROOT, "include", "dcr.h")).read()
    names = set(re.findall(r"\b(dcr_fp4_[a-z_]+)\(const", text))
    assert names == {"dcr_fp4_quantize", "dcr_fp4_dequantize", "dcr_fp4_matmul", "dcr_fp4_matmul_q",
                     "dcr_fp4_matmul_grad"}
    for n in names:
        assert hasattr(dcr.load_library(), n) and hasattr(dcr, n)
    assert "#define DCR_FP4_WORKSPACE_BYTES (64u << 20)" in text and dcr.FP4_WORKSPACE_BYTES == 64 << 20
    assert ctypes.sizeof(dcr.Fp4Desc) == 64
    assert dcr.fp4_blocks(33, dcr.FP4_MX) == 2 and dcr.fp4_blocks(33, dcr.FP4_NV) == 3
