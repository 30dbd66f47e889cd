"""The choice of experts, the order of pairs and their rows on the GPU against a plain 64-bit implementation."""
import numpy as np
import pytest
import torch

from bit_exact_xor_amd import dcr
from tests import step_ref as R

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}       # half a step of a rounding, relative to the value
SOFTMAX, SIGMOID = dcr.SCORE_SOFTMAX, dcr.SCORE_SIGMOID


def up(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


def logits_of(kind, rows, e, rng):
    x = rng.standard_normal((rows, e)) * 2
    if kind == "ties":               # few values: equal logits side by side, zeros of both signs
        x = rng.integers(-2, 3, (rows, e)) * rng.choice([-1.0, 1.0], (rows, e))
    elif kind == "masked":           # shut experts, rows with few and with no open ones
        x[rng.random((rows, e)) < 0.4] = -np.inf
        x[::3] = -np.inf
        x[1::6, : max(1, e // 7)] = 0.25
    elif kind == "lowest":           # masks of the lowest finite number
        x[rng.random((rows, e)) < 0.5] = np.finfo(np.float32).min if e % 2 else -3.3895e38
        x[:1] = -3.3895e38
    elif kind == "far":              # scores far below the largest, and sigmoids at 1
        x = np.exp(rng.uniform(0, 6, (rows, e))) * rng.choice([-1.0, 1.0], (rows, e))
    return x


KINDS = ["normal", "ties", "masked", "lowest", "far"]


def run_select(x, k, bias=None, score=SOFTMAX, groups=1, top_groups=1, renormalize=False, scale=1.0):
    ids = torch.full((x.shape[0], k), 77, dtype=torch.int32, device="cuda")
    w = torch.full((x.shape[0], k), float("nan"), device="cuda")
    dcr.dcr_experts_select(x, ids, w, bias=bias, score=score, groups=groups, top_groups=top_groups, renormalize=renormalize,
                           scale=scale)
    return ids, w


# (rows, experts, k): one token to many, odd numbers of experts, every layout of a row in lanes
SIZES = [(1, 1, 1), (1, 128, 8), (3, 7, 7), (33, 60, 6), (65, 64, 1), (5, 65, 64), (130, 128, 8), (17, 160, 12), (9, 255, 3),
         (12, 384, 8), (7, 513, 10), (4, 1024, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", KINDS)
def test_select(kind, dtype):
    """Ids are the reference's; a weight is rounded once (64-bit scores, off by about 1e-14 of themselves where the argument
    of an exponential is rounded: up to 710 * 2^-53)."""
    rng = np.random.default_rng(KINDS.index(kind))
    for n, (rows, e, k) in enumerate(SIZES):
        x = up(logits_of(kind, rows, e, rng).astype(np.float32)).to(TYPES[dtype])
        host = f64(x)
        for score in (SOFTMAX, SIGMOID):
            for bias in (None, (0.2 * rng.standard_normal(e)).astype(np.float32)):
                renorm, scale = bool((n + score) % 2), (1.0, 2.5)[n % 2]
                ids, w = run_select(x, k, None if bias is None else up(bias), score, renormalize=renorm, scale=scale)
                want_ids, want = R.select(host, bias, k, score == SIGMOID, renormalize=renorm, scale=scale)
                assert np.array_equal(ids.cpu().numpy(), want_ids), (rows, e, k, score, bias is None)
                assert (np.abs(f64(w) - want) <= np.abs(want) * (2.0 ** -24 + 1e-12) + 2.0 ** -149).all(), (rows, e, k)


@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("groups,top_groups", [(2, 1), (4, 2), (8, 4), (8, 7), (16, 3), (64, 5)])
def test_select_groups(score, groups, top_groups):
    rng = np.random.default_rng(groups)
    for rows, size, k in ((1, 1, 1), (19, 5, 3), (40, 16, 4), (6, 128 // groups * 2, 2)):
        e = groups * size
        if e > 1024:
            continue
        k = min(k, e)
        for kind in ("normal", "ties", "masked"):
            x = up(logits_of(kind, rows, e, rng).astype(np.float32))
            for bias in (None, (0.1 * rng.standard_normal(e)).astype(np.float32)):
                ids, w = run_select(x, k, None if bias is None else up(bias), score, groups, top_groups, renormalize=True)
                want_ids, want = R.select(f64(x), bias, k, score == SIGMOID, groups, top_groups, True)
                assert np.array_equal(ids.cpu().numpy(), want_ids), (rows, e, k, kind, bias is None)
                assert (np.abs(f64(w) - want) <= np.abs(want) * (2.0 ** -24 + 1e-12) + 2.0 ** -149).all()


@pytest.mark.parametrize("rows,e,k,groups,top_groups", [(50, 456, 10, 8, 3), (33, 322, 7, 2, 1), (9, 1000, 20, 40, 7),
                                                        (7, 210, 30, 30, 4), (5, 99, 24, 33, 11), (6, 24, 5, 12, 5),
                                                        (40, 1023, 64, 31, 9), (600, 100, 24, 1, 1), (9000, 100, 24, 4, 2),
                                                        (2100, 57, 13, 3, 2)])
def test_select_groups_of_any_size(rows, e, k, groups, top_groups):
    """Groups that lie across lanes, more groups than lanes, more experts to take than lanes hold a row."""
    rng = np.random.default_rng(e)
    for score, kind in ((SOFTMAX, "ties"), (SIGMOID, "normal"), (SIGMOID, "masked")):
        x = logits_of(kind, rows, e, rng).astype(np.float32)
        bias = (0.1 * rng.standard_normal(e)).astype(np.float32)
        ids, w = run_select(up(x), k, up(bias), score, groups, top_groups)
        want_ids, want = R.select(x, bias, k, score == SIGMOID, groups, top_groups)
        assert np.array_equal(ids.cpu().numpy(), want_ids), kind
        assert (np.abs(f64(w) - want) <= np.abs(want) * (2.0 ** -24 + 1e-12) + 2.0 ** -149).all()


def test_select_close_to_a_border():
    """Sums of score and bias that 32 bits cannot tell apart: the bias undoes the scores' differences but for 2^-30."""
    rng = np.random.default_rng(8)
    for score in (SOFTMAX, SIGMOID):
        x = rng.standard_normal((1, 96)).astype(np.float32)
        s = R.scores(x.astype(np.float64), score == SIGMOID)[0]
        bias = (0.5 - s + rng.integers(-3, 4, 96) * 2.0 ** -30).astype(np.float32)
        for groups, top_groups in ((1, 1), (8, 3)):
            ids, _w = run_select(up(x), 16, up(bias), score, groups, top_groups)
            want, _ = R.select(x, bias, 16, score == SIGMOID, groups, top_groups)
            assert np.array_equal(ids.cpu().numpy(), want)


def test_select_groups_of_far_biases():
    """Groups whose two best have biases that cancel: what is left decides, 2^-20 of them."""
    rng = np.random.default_rng(15)
    for groups, size in ((8, 16), (16, 8), (5, 7)):
        e = groups * size
        for score in (SOFTMAX, SIGMOID):
            x = rng.standard_normal((30, e)).astype(np.float32)
            bias = np.full((groups, size), -2.0 ** 20, dtype=np.float32)
            bias[np.arange(groups), rng.integers(0, size, groups)] = 2.0 ** 20
            bias[:, 0] += (rng.integers(-2, 3, groups) / 16).astype(np.float32)
            for top_groups in (1, 3):
                ids, w = run_select(up(x), 3, up(bias.reshape(-1)), score, groups, top_groups)
                want_ids, want = R.select(x, bias.reshape(-1), 3, score == SIGMOID, groups, top_groups)
                assert np.array_equal(ids.cpu().numpy(), want_ids), (groups, score, top_groups)
                assert (np.abs(f64(w) - want) <= np.abs(want) * (2.0 ** -24 + 1e-12)).all()


def test_select_infinite_biases():
    """Experts that a bias puts in front of all or behind all: in the order of their indices there."""
    rng = np.random.default_rng(12)
    for e, k, first, last in ((40, 8, 3, 10), (200, 8, 12, 100), (128, 20, 8, 110), (20, 20, 5, 10)):
        x = rng.standard_normal((9, e)).astype(np.float32)
        bias = (0.1 * rng.standard_normal(e)).astype(np.float32)
        at = rng.permutation(e)
        bias[at[:first]], bias[at[first:first + last]] = np.inf, -np.inf
        for score in (SOFTMAX, SIGMOID):
            ids, w = run_select(up(x), k, up(bias), score)
            want_ids, want = R.select(x, bias, k, score == SIGMOID)
            assert np.array_equal(ids.cpu().numpy(), want_ids), (e, k, score)
            assert (np.abs(f64(w) - want) <= np.abs(want) * (2.0 ** -24 + 1e-12)).all()


def test_select_nan_is_seen():
    """A NaN counts as the largest and its weight is NaN; other rows do not change."""
    rng = np.random.default_rng(4)
    x = rng.standard_normal((6, 40)).astype(np.float32)
    good, _ = R.select(x, None, 4, True)
    x[2, 33] = np.nan
    for groups in ((1, 1), (4, 2)):
        ids, w = run_select(up(x), 4, None, SIGMOID, *groups)
        assert int(ids[2, 0]) == 33 and torch.isnan(w[2, 0]) and not torch.isnan(w[[0, 1, 3, 4, 5]]).any()
    assert np.array_equal(np.delete(run_select(up(x), 4, None, SIGMOID)[0].cpu().numpy(), 2, 0), np.delete(good, 2, 0))
    _ids, w = run_select(up(x), 4)
    assert torch.isnan(w[2]).all() and not torch.isnan(w[[0, 1, 3, 4, 5]]).any()


def test_select_strided_logits():
    rng = np.random.default_rng(2)
    big = up(rng.standard_normal((20, 300)).astype(np.float32))
    for dtype in (torch.float32, torch.bfloat16):
        b = big.to(dtype)
        for view in (b[:, 3:131], b[::2, 8:136], b[1:2, 5:], b[:, 1:8]):
            ids, _ = run_select(view, 5)
            assert np.array_equal(ids.cpu().numpy(), R.select(f64(view), None, 5, False)[0])
            d = torch.full((20, 400), 5.0, dtype=dtype, device="cuda")
            out = d[: view.shape[0], 7: 7 + view.shape[1]]
            dw = torch.ones(view.shape[0], 5, device="cuda") * torch.arange(5, device="cuda")
            dcr.dcr_experts_select_grad(view, ids, dw, out)
            assert (d[:, :7] == 5).all() and (d[:, 7 + view.shape[1]:] == 5).all() and (d[view.shape[0]:] == 5).all()
            want, most = R.select_grad(f64(view), ids.cpu().numpy(), f64(dw), False, False)
            assert (np.abs(f64(out) - want) <= most * 2.0 ** -18 + np.abs(want) * 2.0 ** -8).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("renormalize", [False, True])
def test_select_grad(dtype, score, renormalize):
    """Scores in 32 bits are off by the rounding of the exponential's argument (below 32 here: 2^-19) and some roundings
    of 2^-24: 2^-18 of the sum of the terms' magnitudes, then the rounding of the result."""
    rng = np.random.default_rng(3)
    for rows, e, k in SIZES:
        for kind in ("normal", "masked"):
            x = up(logits_of(kind, rows, e, rng).astype(np.float32)).to(TYPES[dtype])
            ids, _ = run_select(x, k, score=score)
            dw = up(rng.standard_normal((rows, k)).astype(np.float32))
            d = torch.full(x.shape, float("nan"), dtype=x.dtype, device="cuda")
            dcr.dcr_experts_select_grad(x, ids, dw, d, score=score, renormalize=renormalize, scale=1.5)
            want, most = R.select_grad(f64(x), ids.cpu().numpy(), f64(dw), score == SIGMOID, renormalize, 1.5)
            err = np.abs(f64(d) - want)
            assert (err <= most * 2.0 ** -18 + np.abs(want) * HALF[dtype] + 2.0 ** -140).all(), (rows, e, k, kind, err.max())
            if k == 1 and renormalize:
                assert (d == 0).all()                  # a single weight is 1 whatever the logits are
            dcr.dcr_experts_select_grad(x, ids, dw, x, score=score, renormalize=renormalize, scale=1.5)   # in place
            assert torch.equal(x, d)


def test_select_grad_against_differences():
    """The reference's gradient is the limit of its weights' differences, in 64 bits: central differences at h = 1e-5 are
    off by h^2 times third derivatives (below 2 here) and 2^-52 / h."""
    rng = np.random.default_rng(6)
    x = rng.standard_normal((3, 9))
    for sigmoid in (False, True):
        for renorm in (False, True):
            ids, _ = R.select(x, None, 4, sigmoid)
            dw = rng.standard_normal((3, 4))

            def value(y):
                s = np.take_along_axis(R.scores(y, sigmoid), ids.astype(np.int64), 1)
                return (dw * (s / s.sum(1, keepdims=True) if renorm else s) * 0.7).sum()
            want, _ = R.select_grad(x, ids, dw, sigmoid, renorm, 0.7)
            for r in range(3):
                for c in range(9):
                    y, z = x.copy(), x.copy()
                    y[r, c] += 1e-5
                    z[r, c] -= 1e-5
                    assert abs((value(y) - value(z)) / 2e-5 - want[r, c]) < 1e-9


def test_select_grad_of_odd_ids():
    """Ids out of range have no part, one that is there twice counts twice."""
    rng = np.random.default_rng(5)
    x = rng.standard_normal((4, 20)).astype(np.float32)
    ids = np.array([[3, -1, 5, 20], [7, 7, 2, 2], [-5, 1 << 30, -(1 << 31), 19], [-1, -1, -1, -1]], np.int32)
    dw = rng.standard_normal((4, 4)).astype(np.float32)
    for renorm in (False, True):
        for score in (SOFTMAX, SIGMOID):
            d = torch.empty(4, 20, device="cuda")
            dcr.dcr_experts_select_grad(up(x), up(ids), up(dw), d, score=score, renormalize=renorm)
            want, most = R.select_grad(x, ids, dw, score == SIGMOID, renorm)
            assert (np.abs(f64(d) - want) <= most * 2.0 ** -18 + np.abs(want) * 2.0 ** -24).all()
            assert (d[3] == 0).all()


# ------------------------------------------------------------------- order

def run_order(ids, experts, slots=None):
    offsets = torch.full((experts + 1,), 99, dtype=torch.int32, device="cuda")
    slots = torch.full(ids.shape, 99, dtype=torch.int32, device="cuda") if slots is None else slots
    dcr.dcr_experts_order(ids, offsets, slots, dcr.step_workspace())
    return offsets, slots


@pytest.mark.parametrize("n,experts", [(0, 4), (1, 1), (8, 128), (63, 3), (64, 64), (65, 1000), (2048, 7), (2049, 128), (4096, 256),
                                       (12345, 60), (100003, 513), (131072, 128), (300001, 1024)])
def test_order(n, experts):
    rng = np.random.default_rng(n)
    for kind in ("even", "skewed", "holes", "one"):
        ids = rng.integers(0, experts, n)
        if kind == "skewed":
            ids = (experts * rng.random(n) ** 4).astype(np.int64)
        elif kind == "holes":
            bad = rng.random(n) < 0.3
            ids[bad] = rng.choice([-1, -7, experts, 1 << 30, -(1 << 31)], bad.sum())
        elif kind == "one":
            ids[:] = experts - 1
        ids = ids.astype(np.int32)
        offsets, slots = run_order(up(ids), experts)
        want_offsets, want = R.order(ids, experts)
        assert np.array_equal(offsets.cpu().numpy(), want_offsets), kind
        assert np.array_equal(slots.cpu().numpy(), want), kind
        t = up(ids)
        offsets, slots = run_order(t, experts, t)                    # in place
        assert np.array_equal(offsets.cpu().numpy(), want_offsets) and np.array_equal(slots.cpu().numpy(), want), kind


# -------------------------------------------------------------------- rows

def some_slots(tokens, k, experts, rng, holes=0.1):
    ids = np.argsort(rng.random((tokens, max(k, experts))), 1)[:, :k].astype(np.int32)
    ids[rng.random((tokens, k)) < holes] = -1
    ids[: tokens // 5] = -1                                          # padding
    return R.order(ids, max(k, experts))[1]


ROWS = [(1, 1, 1, 4), (3, 7, 2, 4), (5, 8, 1, 3), (24, 2048, 8, 128), (33, 100, 6, 16), (70, 768, 8, 60), (9, 4096, 4, 8),
        (6, 8192, 12, 16), (130, 24, 3, 7), (11, 2055, 5, 9), (4, 16390, 64, 70)]


@pytest.mark.parametrize("xt", ["bf16", "fp32"])
@pytest.mark.parametrize("yt", ["bf16", "fp32"])
def test_rows(xt, yt):
    """Dispatched rows are copies (or one conversion); a combined value is k + 1 roundings of 2^-24 of the sum of magnitudes
    off and rounded once; rows without a pair stay as they were."""
    rng = np.random.default_rng(7)
    for tokens, width, k, e in ROWS:
        slots = some_slots(tokens, k, e, rng)
        n = tokens * k + 3
        for gap, shift in ((0, 0), (5, 1), (16, 8)):
            x = up(rng.standard_normal((tokens, width + gap + shift)).astype(np.float32)).to(TYPES[xt])[:, shift: shift + width]
            y = torch.full((n, width + gap), 3.0, dtype=TYPES[yt], device="cuda")
            dcr.dcr_experts_dispatch(x, up(slots), y[:, :width])
            want = torch.full_like(y, 3.0)
            at, has = up(slots.reshape(-1)).long(), up(slots.reshape(-1) >= 0)
            want[:, :width][at[has]] = x.repeat_interleave(k, 0)[has].to(y.dtype)
            assert torch.equal(y, want), (tokens, width, gap)
            w = up(rng.standard_normal((tokens, k)).astype(np.float32))
            z = up(rng.standard_normal((n, width + gap + shift)).astype(np.float32)).to(TYPES[xt])[:, shift: shift + width]
            for weights in (w, None):
                out = torch.full((tokens, width + gap), 3.0, dtype=TYPES[yt], device="cuda")
                dcr.dcr_experts_combine(z, up(slots), weights, out[:, :width])
                zz = f64(z)[np.maximum(slots, 0)] * (slots >= 0)[..., None]
                ww = np.ones((tokens, k)) if weights is None else f64(w)
                exact, most = (zz * ww[..., None]).sum(1), (np.abs(zz) * np.abs(ww)[..., None]).sum(1)
                err = np.abs(f64(out[:, :width]) - exact)
                assert (err <= (k + 1) * 2.0 ** -24 * most + HALF[yt] * (np.abs(exact) + (k + 1) * 2.0 ** -24 * most)).all()
                assert (out[:, width:] == 3).all()


@pytest.mark.parametrize("dt,xt,gt", [("bf16", "bf16", "bf16"), ("fp32", "bf16", "bf16"), ("bf16", "fp32", "bf16"),
                                      ("fp32", "fp32", "fp32"), ("bf16", "bf16", "fp32"), ("fp32", "bf16", "fp32"),
                                      ("bf16", "fp32", "fp32"), ("fp32", "fp32", "bf16")])
def test_combine_grad(dt, xt, gt):
    """dx is one product, rounded to 32 bits and to its type; a lane of dw adds up an eighth of its eighths of a row at
    most (width / 64 + 8 terms), 64 lanes by six more sums: (width / 64 + 16) 2^-24 of the sum of magnitudes."""
    rng = np.random.default_rng(9)
    for tokens, width, k, e in ROWS:
        slots = some_slots(tokens, k, e, rng)
        n = tokens * k + 2
        for gap, shift in ((0, 0), (3, 1)):
            def some(rows, t):
                return up(rng.standard_normal((rows, width + gap + shift)).astype(np.float32)).to(TYPES[t])[:, shift: shift + width]
            dy, x, w = some(tokens, dt), some(n, xt), up(rng.standard_normal((tokens, k)).astype(np.float32))
            dx = torch.full((n, width + gap), 3.0, dtype=TYPES[gt], device="cuda")
            dw = torch.full((tokens, k), float("nan"), device="cuda")
            dcr.dcr_experts_combine_grad(dy, x, up(slots), w, dx[:, :width], dw)
            want = np.full((n, width), 3.0)
            has = slots >= 0
            each = f64(w)[..., None] * f64(dy)[:, None, :]
            want[slots[has]] = each[has]
            got = f64(dx)
            assert (np.abs(got[:, :width] - want) <= np.abs(want) * (HALF[gt] + 2.0 ** -23)).all()
            untouched = np.ones(n, bool)
            untouched[slots[has]] = False
            assert (got[untouched] == 3).all() and (got[:, width:] == 3).all()
            terms = f64(dy)[:, None, :] * f64(x)[np.maximum(slots, 0)] * has[..., None]
            assert (np.abs(f64(dw) - terms.sum(2)) <= (width / 64 + 16) * 2.0 ** -24 * np.abs(terms).sum(2)).all()
            assert (f64(dw)[~has] == 0).all()


def test_rows_of_foreign_slots():
    """Slots out of range are left out, one that is named twice gets one of its rows."""
    x = torch.arange(1, 4, device="cuda", dtype=torch.float32)[:, None].expand(3, 40).contiguous()
    slots = up(np.array([[0, 5], [-3, 1 << 30], [2, 2]], np.int32))
    y = torch.zeros(5, 40, device="cuda")
    dcr.dcr_experts_dispatch(x, slots, y)
    assert torch.equal(y[:, 0].cpu(), torch.tensor([1., 0, 3, 0, 0])) and (y == y[:, :1]).all()
    out = torch.full((3, 40), 9.0, device="cuda")
    dcr.dcr_experts_combine(y, slots, torch.full((3, 2), 2.0, device="cuda"), out)
    assert torch.equal(out[:, 0].cpu(), torch.tensor([2., 0, 12])) and (out == out[:, :1]).all()
    dw, dx = torch.full((3, 2), 9.0, device="cuda"), torch.zeros(5, 40, device="cuda")
    dcr.dcr_experts_combine_grad(x, y, slots, torch.full((3, 2), 2.0, device="cuda"), dx, dw)
    assert torch.equal(dw.cpu(), torch.tensor([[40., 0], [0, 0], [360, 360]]))
    empty = torch.zeros(0, 40, device="cuda")
    dcr.dcr_experts_dispatch(x, slots, empty)
    dcr.dcr_experts_combine(empty, slots, None, out)
    assert (out == 0).all()
    dcr.dcr_experts_combine_grad(x, empty, slots, torch.ones(3, 2, device="cuda"), empty, dw)
    assert (dw == 0).all()


def test_offsets_past_32_bits():
    """Rows that begin more than 2^32 elements into their matrix (strides, so that little memory is needed)."""
    pool = torch.zeros((1 << 32) + (1 << 12), dtype=torch.bfloat16, device="cuda")
    stride = 1 << 31
    x = torch.as_strided(pool, (3, 64), (stride, 1))
    x.copy_(torch.arange(1, 4, device="cuda")[:, None].expand(3, 64))
    slots = up(np.array([[2, 0], [1, 2]], np.int32))
    y = torch.empty(2, 64, device="cuda")
    dcr.dcr_experts_combine(x, slots, None, y)
    assert torch.equal(y[:, 0].cpu(), torch.tensor([4., 5.])) and (y == y[:, :1]).all()
    dcr.dcr_experts_dispatch(y[:1] * 2, up(np.array([[2]], np.int32)), x)
    assert (x[2] == 8).all() and (x[1] == 2).all()
    ids, w = run_select(x, 3)
    assert torch.equal(ids.cpu(), torch.tensor([[0, 1, 2]] * 3, dtype=torch.int32)) and (w == 1 / 64).all()


@pytest.mark.parametrize("tokens,width,k", [(2100, 520, 2), (2048, 4096, 18), (2047, 513, 3), (4096, 512, 2), (3000, 24, 5),
                                            (2500, 198, 10), (2500, 51, 11), (2100, 1031, 3), (100, 9, 4)])
def test_rows_of_many_tokens(tokens, width, k):
    """The forms for many tokens (a wave a token, narrow rows, results past the caches) against 32-bit torch on the GPU:
    copies are equal; sums of k products within (k + 2) 2^-24, of `width` within (width / 64 + 16) 2^-24 of the sums of
    magnitudes on both sides, bf16 results within half a step more."""
    g = torch.Generator(device="cuda")
    g.manual_seed(tokens)
    n = tokens * k
    slots = torch.randperm(n, device="cuda", generator=g).int().view(tokens, k)
    slots[::50] = -1
    has = slots >= 0
    at = slots.clamp(min=0).long()
    x = torch.randn(tokens, width, device="cuda", generator=g).bfloat16()
    sent = torch.full((n, width), 3.0, dtype=torch.bfloat16, device="cuda")
    dcr.dcr_experts_dispatch(x, slots, sent)
    for j in range(k):
        assert torch.equal(sent[at[has[:, j], j]], x[has[:, j]])
    untouched = torch.ones(n, dtype=torch.bool, device="cuda")
    untouched[at[has]] = False
    assert (sent[untouched] == 3).all()
    z = torch.randn(n, width, device="cuda", generator=g).bfloat16()
    w = torch.randn(tokens, k, device="cuda", generator=g)
    y = torch.empty_like(x)
    dcr.dcr_experts_combine(z, slots, w, y)
    want, most = torch.zeros(tokens, width, device="cuda"), torch.zeros(tokens, width, device="cuda")
    for j in range(k):
        term = torch.where(has[:, j, None], w[:, j, None] * z[at[:, j]].float(), 0.0)
        want += term
        most += term.abs()
    tol = 2 * (k + 2) * 2.0 ** -24 * most
    assert ((y.float() - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol)).all()
    dy = torch.randn(tokens, width, device="cuda", generator=g).bfloat16()
    dz, dw = torch.full_like(z, 3.0), torch.full((tokens, k), 77.0, device="cuda")
    dcr.dcr_experts_combine_grad(dy, z, slots, w, dz, dw)
    assert (dz[untouched] == 3).all()
    for j in range(k):
        h = has[:, j]
        a, b = at[h, j], dy[h].float()
        assert torch.equal(dz[a], (w[h, j, None] * b).bfloat16())
        terms = b * z[a].float()
        assert ((dw[h, j].double() - terms.double().sum(1)).abs() <= (width / 64 + 17) * 2.0 ** -24 * terms.abs().sum(1)).all()
        assert (dw[~h, j] == 0).all()


def by_definition(x, bias, k, sigmoid, groups=1, top_groups=1, renormalize=False):
    """As step_ref.select, of rows with infinities and NaN: a NaN counts as the largest of what is compared, the lowest index
    of equals first, a group's value is the sum of its two largest above -infinity, ids of -1 have weight 0."""
    first = lambda v, i: (not np.isnan(v), -(0.0 if np.isnan(v) else v), i)  # noqa: E731
    x = x.astype(np.float64)
    with np.errstate(invalid="ignore"):
        s = R.scores(x, sigmoid)
        value = s + (0 if bias is None else bias.astype(np.float64))
    rows, e = x.shape
    size = e // groups
    ids, w = np.full((rows, k), -1), np.zeros((rows, k))
    for r in range(rows):
        taken = range(groups)
        if top_groups < groups:
            of = []
            for g in range(groups):
                best = sorted((first(value[r, i], i) for i in range(g * size, (g + 1) * size)
                               if not np.isneginf(x[r, i]) and not np.isneginf(value[r, i])))[:2]
                of.append(sum(value[r, i] for _n, _v, i in best) if best else -np.inf)
            taken = sorted(range(groups), key=lambda g: first(of[g], g))[:top_groups]
        rank = x[r] if bias is None else value[r]
        best = sorted((first(rank[i], i) for i in range(e) if not np.isneginf(x[r, i]) and i // size in set(taken)))[:k]
        ids[r, :len(best)] = [i for _n, _v, i in best]
        w[r, :len(best)] = s[r, ids[r, :len(best)]]
        if renormalize and w[r].sum() != 0:
            w[r, :len(best)] /= w[r].sum()
    return ids, w


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("e,k,groups,top_groups", [(40, 6, 1, 1), (64, 8, 8, 3), (200, 12, 1, 1), (456, 10, 8, 3), (1000, 20, 40, 7)])
def test_select_of_infinite_and_nan_logits(e, k, groups, top_groups, dtype):
    """A softmax of a row with +infinity or NaN has no numbers: all weights of its chosen experts are NaN, and where scores
    are compared (a bias, groups) all are equal.  A sigmoid of +infinity is 1.  (A weight is rounded once, as above.)"""
    rng = np.random.default_rng(e)
    x = rng.standard_normal((12, e)) * 2
    x[1, 5] = np.inf
    x[2, [7, e - 1]] = np.inf
    x[3, e // 2] = np.nan
    x[4, 3], x[4, e - 2] = np.nan, np.inf
    x[5, : e - 3], x[5, e - 2] = -np.inf, np.inf           # fewer open than are asked for
    x[6, ::2], x[6, 1] = -np.inf, np.inf
    x[7] = np.inf
    logits = up(x.astype(np.float32)).to(TYPES[dtype])
    host = f64(logits)
    for score in (SOFTMAX, SIGMOID):
        for bias in (None, (0.1 * rng.standard_normal(e)).astype(np.float32), np.zeros(e, np.float32)):
            for renorm in (False, True):
                ids, w = run_select(logits, k, None if bias is None else up(bias), score, groups, top_groups, renorm)
                want_ids, want = by_definition(host, bias, k, score == SIGMOID, groups, top_groups, renorm)
                what = (score, None if bias is None else float(np.abs(bias).max()), renorm)
                assert np.array_equal(ids.cpu().numpy(), want_ids), what
                got = f64(w)
                assert np.array_equal(np.isnan(got), np.isnan(want)), what
                good = ~np.isnan(want)
                assert (np.abs(got - want)[good] <= np.abs(want[good]) * (2.0 ** -24 + 1e-12) + 2.0 ** -149).all(), what


def test_select_groups_do_not_depend_on_other_rows():
    """Rows in which fewer groups than are taken have a value (the others are behind all by their bias): the rest is taken by
    index, whether or not a row beside them has to be decided in 64 bits (two equal groups at the border)."""
    e, groups, k = 64, 8, 12
    rng = np.random.default_rng(21)
    bias = np.zeros(e, np.float32)
    bias[:16] = -np.inf                                    # groups 0 and 1
    for score in (SOFTMAX, SIGMOID):
        x = rng.standard_normal((16, e)).astype(np.float32)
        x[1::2, 16:56] = -np.inf                           # only group 7 has a value
        alone, _ = run_select(up(x[1::2]), k, up(bias), score, groups, 4)
        x[0::2, 16:] = np.tile(x[0::2, 16:24], (1, 6))     # six equal groups
        ids, _ = run_select(up(x), k, up(bias), score, groups, 4)
        want, _ = by_definition(x, bias, k, score == SIGMOID, groups, 4)
        assert np.array_equal(alone.cpu().numpy(), want[1::2]), score
        assert np.array_equal(ids.cpu().numpy(), want), score


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
def test_select_grad_of_small_scores(score, dtype):
    """Renormalised weights have derivatives of their own size whatever the chosen scores are: logits near where a score
    leaves the normal numbers of 32 bits, far below it, and chosen ones far below the row's largest.  An exponential's
    argument is a difference d rounded once (2^-24 |d| of the term, d as far as the chosen ones lie apart, and what is that
    far down is as small itself: |d| e^-|d| < 0.37), some 2^-22 more for its own rounding and the sums: 2^-18 of the sum of
    the terms' magnitudes as above."""
    rng = np.random.default_rng(31)
    for e, k in ((60, 6), (128, 8), (384, 12), (1000, 64)):
        for base in (-60, -86, -87.5, -88, -88.6, -89, -100, -103.5, -110, -300, -600):
            x = (base + rng.standard_normal((20, e))).astype(np.float32)
            bias = None
            if score == SOFTMAX:                           # the bias chooses among experts far below the largest
                x[:, 0] = 0.5
                bias = np.zeros(e, np.float32)
                bias[1::2] = 2.0
            logits = up(x).to(TYPES[dtype])
            ids, w = run_select(logits, k, None if bias is None else up(bias), score, renormalize=True)
            dw = up(rng.standard_normal((20, k)).astype(np.float32))
            d = torch.full(logits.shape, float("nan"), dtype=logits.dtype, device="cuda")
            dcr.dcr_experts_select_grad(logits, ids, dw, d, score=score, renormalize=True, scale=1.5)
            want, most = R.select_grad(f64(logits), ids.cpu().numpy(), f64(dw), score == SIGMOID, True, 1.5)
            assert np.abs(want).max() > 0.01
            err = np.abs(f64(d) - want)
            assert (err <= most * 2.0 ** -18 + np.abs(want) * HALF[dtype] + 2.0 ** -126).all(), (e, k, base, err.max())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
def test_select_grad_of_far_logits(score, renormalize, dtype):
    """The kinds that the choice is tested with: masks of the lowest finite number, logits up to some hundreds.  Where weights
    are not renormalised a score's exponent is rounded as its distance |d| from the largest (or from 0) has it, 2^-23 |d| of
    the score; the others as above."""
    rng = np.random.default_rng(32)
    for rows, e, k in SIZES:
        for kind in ("lowest", "far", "ties"):
            x = up(logits_of(kind, rows, e, rng).astype(np.float32)).to(TYPES[dtype])
            ids, _ = run_select(x, k, score=score)
            dw = up(rng.standard_normal((rows, k)).astype(np.float32))
            d = torch.full(x.shape, float("nan"), dtype=x.dtype, device="cuda")
            dcr.dcr_experts_select_grad(x, ids, dw, d, score=score, renormalize=renormalize, scale=1.5)
            host = f64(x)
            with np.errstate(over="ignore"):
                want, most = R.select_grad(host, ids.cpu().numpy(), f64(dw), score == SIGMOID, renormalize, 1.5)
                far = np.abs(host if score == SIGMOID else host - host.max(1, keepdims=True))
            err = np.abs(f64(d) - want)
            tol = most * (2.0 ** -18 + 2.0 ** -23 * np.minimum(far, 1e3))
            assert (err <= tol + np.abs(want) * HALF[dtype] + 2.0 ** -126).all(), (rows, e, k, kind, err.max())


def test_select_near_a_border_of_many_experts():
    """More than 512 experts (16 a lane), whose softmax scores a bias undoes but for a few 2^-20 of the largest: the choice is
    that of 64 bits however the sum of 32 bits is rounded."""
    rng = np.random.default_rng(41)
    for e in (513, 700, 1024):
        for kind in range(3):
            x = rng.standard_normal((1, e)).astype(np.float32)
            if kind:
                x = np.sort(x)[:, ::-1] if kind == 1 else np.full((1, e), 0.3, np.float32) + rng.standard_normal((1, e)).astype(np.float32) * 2.0 ** -10
            s = R.scores(x.astype(np.float64), False)[0]
            bias = (1.0 - s + rng.integers(-4, 5, e) * (2.0 ** -20 * s.max())).astype(np.float32)
            for k in (1, 7, 64):
                for groups, top_groups in ((1, 1), (e // (e // 9 if e == 513 else e // 4), 2)):
                    ids, _w = run_select(up(x), k, up(bias), SOFTMAX, groups, top_groups)
                    want, _ = R.select(x, bias, k, False, groups, top_groups)
                    assert np.array_equal(ids.cpu().numpy(), want), (e, kind, k, groups)
