"""Refusals of a training turn's calls, made before any launch, and what of them runs on the host (no GPU)."""
import ctypes
import os

import numpy as np
import pytest
import torch

from bit_exact_xor_amd import dcr
from tests import step_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
AT = 1 << 20            # an aligned address that is never read
WS = dcr.STEP_WORKSPACE_BYTES
INF = float("inf")


def call(name, defaults, **kw):
    return getattr(dcr.load_library(), name)(*{**defaults, **kw}.values(), None)


SELECT = dict(x=AT, ty=0, xs=64, rows=4, e=64, bias=AT, score=0, groups=8, top=4, opt=1, scale=1.0, k=8, ids=AT, w=AT)
SELECT_GRAD = dict(x=AT, ty=0, xs=64, rows=4, e=64, ids=AT, dw=AT, k=8, score=1, opt=0, scale=1.0, d=AT, ds=64)
ORDER = dict(ids=AT, n=32, e=64, off=AT, slots=AT, ws=AT, size=WS)
DISPATCH = dict(x=AT, xt=1, xs=64, tokens=4, width=64, slots=AT, k=8, y=AT, yt=1, ys=64, n=32)
COMBINE = dict(x=AT, xt=1, xs=64, n=32, slots=AT, w=AT, tokens=4, width=64, k=8, y=AT, yt=0, ys=64)
COMBINE_GRAD = dict(dy=AT, dt=0, ds=64, tokens=4, width=64, x=AT, xt=1, xs=64, n=32, slots=AT, w=AT, k=8, dx=AT, gt=1, gs=64, dw=AT)
LOGPROBS = dict(x=AT, ty=1, xs=100, rows=4, v=100, t=AT, tb=8, scale=1.0, logp=AT, lse=AT, ent=AT, top=5, ids=AT, vals=AT, ws=AT,
                size=WS)
LOGPROBS_GRAD = dict(x=AT, ty=1, xs=100, rows=4, v=100, t=AT, tb=4, scale=1.0, lse=AT, dlogp=AT, ent=AT, dent=AT, d=AT, ds=100)

BAD = [
    ("dcr_experts_select", SELECT, [dict(x=None), dict(x=AT + 2), dict(ty=2), dict(xs=63), dict(xs=1 << 32), dict(rows=1 << 31),
                                    dict(rows=1 << 28), dict(e=0), dict(e=1025, xs=2000), dict(score=2), dict(groups=0),
                                    dict(groups=3), dict(groups=65), dict(top=0), dict(top=9), dict(opt=2), dict(scale=INF),
                                    dict(scale=float("nan")), dict(k=0), dict(k=65), dict(e=4, groups=1, top=1), dict(bias=AT + 1),
                                    dict(ids=None), dict(ids=AT + 2), dict(w=None), dict(w=AT + 3)]),
    ("dcr_experts_select_grad", SELECT_GRAD, [dict(x=None), dict(ty=7), dict(xs=1), dict(e=0), dict(k=0), dict(k=65), dict(score=3),
                                              dict(opt=4), dict(scale=-INF), dict(ids=None), dict(dw=None), dict(dw=AT + 1),
                                              dict(d=None), dict(d=AT + 1), dict(ds=63)]),
    ("dcr_experts_order", ORDER, [dict(ids=None), dict(ids=AT + 1), dict(n=1 << 31), dict(e=0), dict(e=1025), dict(off=None),
                                  dict(off=AT + 2), dict(slots=None), dict(slots=AT + 2), dict(ws=None), dict(ws=AT + 8)]),
    ("dcr_experts_dispatch", DISPATCH, [dict(x=None), dict(x=AT + 1), dict(xt=2), dict(xs=63), dict(tokens=1 << 31), dict(slots=None),
                                        dict(slots=AT + 1), dict(k=0), dict(k=65), dict(y=None), dict(y=AT + 1), dict(yt=5),
                                        dict(ys=63), dict(ys=1 << 32), dict(n=1 << 31), dict(width=1 << 31)]),
    ("dcr_experts_combine", COMBINE, [dict(x=None), dict(xt=2), dict(xs=63), dict(n=1 << 31), dict(slots=None), dict(w=AT + 2),
                                      dict(tokens=1 << 31), dict(k=0), dict(k=65), dict(y=None), dict(y=AT + 2), dict(yt=9),
                                      dict(ys=0)]),
    ("dcr_experts_combine_grad", COMBINE_GRAD, [dict(dy=None), dict(dy=AT + 2), dict(dt=3), dict(ds=63), dict(x=None), dict(xt=2),
                                                dict(xs=8), dict(slots=None), dict(w=None), dict(k=0), dict(dx=None), dict(gt=2),
                                                dict(gs=63), dict(dw=None), dict(dw=AT + 2), dict(n=1 << 31)]),
    ("dcr_logprobs", LOGPROBS, [dict(x=None), dict(x=AT + 1), dict(ty=2), dict(xs=99), dict(rows=1 << 31), dict(v=0),
                                dict(v=1 << 31, xs=1 << 31), dict(t=None), dict(t=AT + 4), dict(tb=2), dict(scale=0.0),
                                dict(scale=-1.0), dict(scale=INF), dict(scale=float("nan")), dict(logp=AT + 1), dict(lse=AT + 2),
                                dict(ent=AT + 2), dict(top=65), dict(top=64, v=63), dict(ids=None), dict(vals=None), dict(ws=None),
                                dict(ws=AT + 4)]),
    ("dcr_logprobs_grad", LOGPROBS_GRAD, [dict(x=None), dict(ty=2), dict(xs=99), dict(v=0), dict(t=None), dict(t=AT + 2), dict(tb=3),
                                          dict(scale=0.0), dict(lse=None), dict(dlogp=None), dict(ent=None), dict(dent=AT + 2),
                                          dict(d=None), dict(d=AT + 1), dict(ds=99)]),
]


@pytest.mark.parametrize("name,defaults,bad", BAD, ids=[b[0] for b in BAD])
def test_bad_arguments(name, defaults, bad):
    for kw in bad:
        assert call(name, defaults, **kw) == dcr.DCR_E_INVAL, kw
        assert dcr.load_library().dcr_last_error(), kw


def test_small_workspaces():
    for name, defaults in (("dcr_experts_order", ORDER), ("dcr_logprobs", LOGPROBS)):
        assert call(name, defaults, size=WS - 1) == dcr.DCR_E_CAPACITY


def test_nothing_to_do():
    """Empty calls return without a launch and look at no buffer."""
    assert call("dcr_experts_select", SELECT, rows=0, x=None, ids=None, w=None) == dcr.DCR_OK
    assert call("dcr_experts_select_grad", SELECT_GRAD, rows=0, x=None, d=None, ids=None, dw=None) == dcr.DCR_OK
    for kw in (dict(tokens=0, x=None, slots=None), dict(width=0, x=None, y=None, slots=None), dict(n=0, y=None)):
        assert call("dcr_experts_dispatch", DISPATCH, **kw) == dcr.DCR_OK
    for kw in (dict(tokens=0, y=None, slots=None, w=None), dict(width=0, x=None, y=None, slots=None, w=None)):
        assert call("dcr_experts_combine", COMBINE, **kw) == dcr.DCR_OK
    assert call("dcr_experts_combine_grad", COMBINE_GRAD, tokens=0, dy=None, slots=None, w=None, dw=None) == dcr.DCR_OK
    assert call("dcr_logprobs", LOGPROBS, rows=0, x=None, t=None, logp=None) == dcr.DCR_OK
    assert call("dcr_logprobs_grad", LOGPROBS_GRAD, rows=0, x=None, d=None) == dcr.DCR_OK


def adam(numel=64, param=1, grad=2, m=3, v=4, ms=None, vs=None, copy=None, pt=0, gt=0, bits=32, flags=0, first=0):
    at = lambda i: None if i is None else int(AT * i)  # noqa: E731
    return dcr.AdamWDesc(at(param), at(grad), at(m), at(v), at(ms), at(vs), at(copy), numel, first, pt, gt, bits, flags)


def build(*descs):
    handle = ctypes.c_void_p()
    arr = (dcr.AdamWDesc * max(1, len(descs)))(*descs)
    rc = dcr.load_library().dcr_adamw_plan_build(ctypes.addressof(arr), len(descs), ctypes.byref(handle))
    return rc, handle.value


def test_adamw_plans():
    lib = dcr.load_library()
    for d in (adam(param=None), adam(grad=None), adam(m=None), adam(v=None), adam(param=1 + 2 ** -18), adam(grad=2 + 2 ** -17),
              adam(pt=2), adam(gt=2), adam(bits=16), adam(flags=2), adam(bits=8), adam(bits=8, ms=5), adam(pt=1, copy=5),
              adam(numel=1 << 41), adam(copy=5 + 2 ** -17), adam(numel=1 << 37)):   # (2^-18 and 2^-17 of AT: 4 and 8 bytes)
        rc, handle = build(d)
        assert rc == dcr.DCR_E_INVAL and handle is None
        assert lib.dcr_last_error()
    # memory that is written and read or written through another tensor as well
    for pair in ((adam(), adam()), (adam(), adam(param=11, grad=12, m=13, v=1)), (adam(), adam(param=11, grad=1, m=13, v=14)),
                 (adam(copy=2),), (adam(m=4),), (adam(numel=AT // 4 + 1),), (adam(bits=8, ms=5, vs=5),)):
        rc, handle = build(*pair)
        assert rc == dcr.DCR_E_INVAL and b"overlap" in lib.dcr_last_error()
    # one gradient of two tensors is read only; tensors without elements name nothing
    for good in ((), (adam(),), (adam(), adam(param=11, m=13, v=14)), (adam(numel=0, param=None, grad=None, m=None, v=None),),
                 (adam(bits=8, ms=5, vs=6, copy=7, gt=1),), (adam(numel=AT // 4),)):
        rc, handle = build(*good)
        assert rc == dcr.DCR_OK and handle
        size = ctypes.c_uint64()
        assert lib.dcr_adamw_plan_bytes(handle, ctypes.byref(size)) == dcr.DCR_OK and size.value > 0
        assert lib.dcr_adamw_plan_bytes(handle, None) == dcr.DCR_E_INVAL
        assert lib.dcr_adamw_plan_upload(handle, AT, size.value - 1, None) == dcr.DCR_E_CAPACITY
        assert lib.dcr_adamw_plan_upload(handle, AT + 8, size.value, None) == dcr.DCR_E_INVAL
        assert lib.dcr_adamw_plan_upload(handle, None, size.value, None) == dcr.DCR_E_INVAL
        args = dcr.AdamWArgs(1e-3, .9, .99, 1e-8, 0, 1, 1, None, 0, 0)
        assert lib.dcr_adamw_step(handle, ctypes.addressof(args), None) == dcr.DCR_E_INVAL
        assert b"not uploaded" in lib.dcr_last_error()
        lib.dcr_adamw_plan_destroy(handle)
    assert build()[0] == dcr.DCR_OK and lib.dcr_adamw_plan_build(None, 1, ctypes.byref(ctypes.c_void_p())) == dcr.DCR_E_INVAL
    assert lib.dcr_adamw_plan_build(None, 0, None) == dcr.DCR_E_INVAL
    lib.dcr_adamw_plan_destroy(None)


def test_binding_refuses():
    """Python-side checks: types, shapes, strides, host tensors."""
    f, i32, u8 = torch.float32, torch.int32, torch.uint8
    z = lambda *s, dtype=f: torch.zeros(s, dtype=dtype)  # noqa: E731
    ids, slots, w = z(4, 2, dtype=i32), z(4, 2, dtype=i32), z(4, 2)
    for bad in (lambda: dcr.dcr_experts_select(z(4, 8), ids, w),                                  # host tensors
                lambda: dcr.dcr_experts_select(z(5, 8), ids, w),
                lambda: dcr.dcr_experts_select(z(4, 8, dtype=torch.float16), ids, w),
                lambda: dcr.dcr_experts_select(z(4, 8), ids.long(), w),
                lambda: dcr.dcr_experts_select(z(4, 8), ids, z(4, 3)),
                lambda: dcr.dcr_experts_select(z(4, 8), ids, z(2, 4).t()),
                lambda: dcr.dcr_experts_select(z(4, 8), ids, w, bias=z(7)),
                lambda: dcr.dcr_experts_select_grad(z(4, 8), ids, w, z(4, 8, dtype=torch.bfloat16)),
                lambda: dcr.dcr_experts_order(ids, z(9, dtype=i32), slots, None),
                lambda: dcr.dcr_experts_order(ids, z(1, dtype=i32), slots, z(WS, dtype=u8)),
                lambda: dcr.dcr_experts_order(ids, z(9, dtype=i32), z(8, dtype=i32), z(WS, dtype=u8)),
                lambda: dcr.dcr_experts_dispatch(z(4, 8), slots, z(8, 7)),
                lambda: dcr.dcr_experts_dispatch(z(3, 8), slots, z(8, 8)),
                lambda: dcr.dcr_experts_combine(z(8, 8), slots, w.double(), z(4, 8)),
                lambda: dcr.dcr_experts_combine_grad(z(4, 8), z(8, 8), slots, None, z(8, 8), w),
                lambda: dcr.dcr_experts_combine_grad(z(4, 8), z(8, 8), slots, w, z(7, 8), w),
                lambda: dcr.dcr_logprobs(z(4, 8), None, z(4), workspace=z(WS, dtype=u8)),
                lambda: dcr.dcr_logprobs(z(4, 8), z(4), z(4), workspace=z(WS, dtype=u8)),
                lambda: dcr.dcr_logprobs(z(4, 8), z(4, dtype=i32), z(4)),
                lambda: dcr.dcr_logprobs(z(4, 8), z(4, dtype=i32), z(4), top_ids=ids, workspace=z(WS, dtype=u8)),
                lambda: dcr.dcr_logprobs(z(8, 4).t(), z(4, dtype=i32), z(4), workspace=z(WS, dtype=u8)),
                lambda: dcr.dcr_logprobs_grad(z(4, 8), z(4, dtype=i32), z(4), z(4), z(4, 8), dentropy=z(4)),
                lambda: dcr.dcr_logprobs_grad(z(4, 8), z(5, dtype=i32), z(4), z(4), z(4, 8)),
                lambda: dcr.AdamWTensors([], []),
                lambda: dcr.AdamWTensors([z(4)], [z(4)]),
                lambda: dcr.AdamWTensors([z(4)], [z(4)], bits=16),
                lambda: dcr.dcr_adamw_step(None, 0),
                lambda: dcr.dcr_adamw_step(None, 1, dither=1 << 32)):
        with pytest.raises(ValueError):
            bad()


def test_header_and_binding_agree():
    text = open(os.path.join(ROOT, "include", "dcr.h")).read()
    assert "#define DCR_STEP_WORKSPACE_BYTES (4u << 20)" in text and WS == 4 << 20
    assert "#define DCR_ADAMW_BLOCK 32" in text and dcr.ADAMW_BLOCK == 32
    assert ctypes.sizeof(dcr.AdamWDesc) == 88 and ctypes.sizeof(dcr.AdamWArgs) == 72
    for n in ("dcr_experts_select", "dcr_experts_select_grad", "dcr_experts_order", "dcr_experts_dispatch", "dcr_experts_combine",
              "dcr_experts_combine_grad", "dcr_logprobs", "dcr_logprobs_grad", "dcr_adamw_step"):
        assert n + "(" in text and hasattr(dcr, n) and hasattr(dcr.load_library(), n)


def test_dither_is_even():
    """The dither's numbers are spread evenly over elements, steps and seeds, and the two of an element are independent:
    the mean of n of them is within five of its standard deviations, (12 n)^-1/2, of a half; sixteen bins within five of theirs."""
    n = 1 << 18
    at = np.arange(n, dtype=np.uint64)
    for base, seed, step in ((0, 1, 1), (0, 1, 2), (0, 7, 1000), ((1 << 32) - n // 2, 1, 5), (1 << 40, 99, 123456)):
        a, b = R.dither(at + np.uint64(base), seed, step)
        assert abs(a.mean() - .5) < 5 / np.sqrt(12 * n) and abs(b.mean() - .5) < 5 / np.sqrt(12 * n)
        for x in (a, b, (a + b) % 1.0, (a[1:] - a[:-1]) % 1.0, (b[32:] - b[:-32]) % 1.0):
            count = np.histogram(x, 16, (0, 1))[0]
            assert np.abs(count - len(x) / 16).max() < 5 * np.sqrt(len(x) / 16), (base, seed, step)


def test_adamw_tables_are_small():
    """An entry of 80 bytes for 4096 elements, and at most eight for what is left of a tensor."""
    lib = dcr.load_library()
    far = lambda i: 1 << 44 | i << 40  # noqa: E731
    for n in (1, 511, 4096, 1 << 30, (1 << 30) + 4095, (1 << 33) + 1):
        for bits in (8, 32):
            rc, handle = build(dcr.AdamWDesc(far(0), far(1), far(2), far(3), far(4), far(5), far(6), n, 0, 0, 1, bits, 0))
            assert rc == dcr.DCR_OK
            size = ctypes.c_uint64()
            assert lib.dcr_adamw_plan_bytes(handle, ctypes.byref(size)) == dcr.DCR_OK
            assert size.value <= 80 * (n // 4096 + 8) + 64, n
            lib.dcr_adamw_plan_destroy(handle)
