"""Log probabilities and their gradient on the GPU against a plain 64-bit implementation."""
import numpy as np
import pytest
import torch

from bit_exact_xor_amd import dcr
from tests import step_ref as R

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
INF = float("inf")


def up(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


def logits_of(kind, rows, vocab, dtype, rng, gap=0, shift=0):
    x = rng.standard_normal((rows, vocab)) * 3
    if kind == "peaked":
        x[np.arange(rows), rng.integers(0, vocab, rows)] = 25
    elif kind == "masked":
        x[rng.random((rows, vocab)) < 0.5] = -np.inf
        x[::3] = -np.inf
        x[1::6, vocab // 2] = -2.0
    elif kind == "lowest":
        x[rng.random((rows, vocab)) < 0.5] = -3.3895e38
        x[::3] = -3.3895e38
    elif kind == "ties":
        x = rng.integers(-1, 2, (rows, vocab)) * rng.choice([-1.0, 1.0], (rows, vocab))
    elif kind == "rising":
        x = np.sort(x, 1)
    elif kind == "shifted":
        x += 1000
    t = torch.empty(rows, vocab + gap + shift, dtype=TYPES[dtype], device="cuda")[:, shift: shift + vocab]
    return t.copy_(up(x.astype(np.float32)))


KINDS = ["normal", "peaked", "masked", "lowest", "ties", "rising", "shifted"]
SIZES = [(1, 1), (2, 3), (5, 64), (3, 1000), (2, 4096), (1, 4097), (9, 50257), (2, 151936), (520, 300), (513, 5001)]


def order_of(x):
    """Indices by value, the lowest of equals first."""
    return np.lexsort((np.arange(x.shape[1])[None].repeat(len(x), 0), -(x + 0.0)), axis=1)


def close(got, want, tol):
    both = np.isneginf(want)
    assert (np.isneginf(got) == both).all()
    with np.errstate(invalid="ignore"):
        err = np.abs(np.where(both, 0, got - np.where(both, 0, want)))
    assert (err <= tol).all(), (err.max(), np.max(err - tol))


def tolerances(x, scale):
    """(of lse, of log p without its own difference, of the entropy).  An exponential 2^d takes a difference rounded
    twice (2^-23 |d|, d up to 160 before it vanishes: but p |d| is below 0.54) and is 2^-23 off: 2^-21 of S in all.  A
    thread adds at most vocab / 256 + 16 terms and its sums are rescaled as often as it takes 16 terms, then 20 joins:
    (vocab / 256 + 40) 2^-24 of S and, with |T| / S for the entropy, of T.  log S below 2^5: 2^-20 with its own rounding."""
    rows, vocab = x.shape
    lp, lse, ent, p = R.logprobs(x, scale)
    grow = (vocab / 256 + 40) * 2.0 ** -24 + 2.0 ** -21
    with np.errstate(invalid="ignore"):
        d = np.where(p > 0, (x - x.max(1, keepdims=True)) * scale, 0)
    t = -(p * d).sum(1)
    big = np.abs(np.where(np.isneginf(lse), 0, lse))
    return grow + 2.0 ** -20 + 2.0 ** -23 * big, grow + 2.0 ** -20, 2 * grow * (1 + t) + 2.0 ** -20


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", KINDS)
def test_logprobs(kind, dtype):
    rng = np.random.default_rng(KINDS.index(kind))
    ws = dcr.step_workspace()
    ws.fill_(0xFF)
    for n, (rows, vocab) in enumerate(SIZES):
        gap, shift = ((0, 0), (5, 1), (8, 8))[n % 3]
        scale = float(np.float32((1.0, 0.7, 1.0)[n % 3]))
        logits = logits_of(kind, rows, vocab, dtype, rng, gap, shift)
        x = f64(logits)
        targets = rng.integers(0, vocab, rows)
        targets[1::4] = -1
        t = up(targets.astype(np.int64 if n % 2 else np.int32))
        lp, lse, ent, p = R.logprobs(x, scale)
        at_lse, at_lp, at_ent = tolerances(x, scale)
        order = order_of(x)
        for top in sorted({0, 1, min(5, vocab), min(20, vocab), min(64, vocab)}):
            out = [torch.full((rows,), 77.0, device="cuda") for _ in range(3)]
            ids = torch.full((rows, top), -5, dtype=torch.int32, device="cuda") if top else None
            vals = torch.full((rows, top), 77.0, device="cuda") if top else None
            dcr.dcr_logprobs(logits, t, *out, ids, vals, scale=scale, workspace=ws)
            at = np.maximum(targets, 0)
            mine = np.take_along_axis(lp, at[:, None], 1)[:, 0]
            with np.errstate(invalid="ignore"):
                far = 2.0 ** -22 * np.abs(np.nan_to_num((x[np.arange(rows), at] - x.max(1)) * scale, nan=0, posinf=0, neginf=0))
            close(f64(out[0]), np.where(targets < 0, 0, mine), at_lp + far)
            close(f64(out[1]), lse, at_lse)
            close(f64(out[2]), ent, at_ent)
            if top:
                assert np.array_equal(ids.cpu().numpy(), order[:, :top]), (rows, vocab, top)
                best = np.take_along_axis(lp, order[:, :top], 1)
                with np.errstate(invalid="ignore"):
                    d = np.nan_to_num((np.take_along_axis(x, order[:, :top], 1) - x.max(1, keepdims=True)) * scale, nan=0, neginf=0)
                close(f64(vals), best, at_lp + 2.0 ** -22 * np.abs(d))


def test_logprobs_of_odd_targets():
    """None, the ends, past the vocabulary; outputs that are not asked for."""
    x = torch.randn(6, 1003, device="cuda")
    ws = dcr.step_workspace()
    t = torch.tensor([-100, 0, 1002, 1003, 1 << 40, -(1 << 40)], device="cuda")
    lp = torch.empty(6, device="cuda")
    dcr.dcr_logprobs(x, t, lp, workspace=ws)
    want = torch.log_softmax(x.double(), 1)
    assert lp[0] == 0 and lp[5] == 0 and torch.isnan(lp[3:5]).all()
    assert abs(float(lp[1] - want[1, 0])) < 1e-5 and abs(float(lp[2] - want[2, 1002])) < 1e-5
    lse = torch.empty(6, device="cuda")
    dcr.dcr_logprobs(x, None, lse=lse, workspace=ws)
    assert torch.allclose(lse.double(), torch.logsumexp(x.double(), 1), atol=1e-5)
    dcr.dcr_logprobs(x[:0], t[:0], lp[:0], workspace=ws)


@pytest.mark.parametrize("rows", [3, 600])
def test_nan_and_infinity_stay_in_their_row(rows):
    x = torch.randn(rows, 5000, device="cuda")
    x[1, 4321], x[2, 17] = float("nan"), INF
    out = [torch.empty(rows, device="cuda") for _ in range(3)]
    ids, vals = torch.empty(rows, 4, dtype=torch.int32, device="cuda"), torch.empty(rows, 4, device="cuda")
    dcr.dcr_logprobs(x, torch.zeros(rows, dtype=torch.int32, device="cuda"), *out, ids, vals, workspace=dcr.step_workspace())
    for v in (*out, vals[:, 0]):
        assert torch.isnan(v[1:3]).all() and not torch.isnan(v[0]) and not torch.isnan(v[3:]).any()
    assert ids[2, 0] == 17 and (ids[1] >= 0).all() and len(set(ids[1].tolist())) == 4


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["normal", "peaked", "masked", "ties"])
def test_logprobs_grad(kind, dtype):
    """With l = log p rounded once and multiplied (|l| 2^-22 in the exponent) and an exponential 2^-23 off, a term's factors
    are off by (3 |l| + 8) 2^-23 of themselves; the one-hot term is one rounding; then the result's."""
    rng = np.random.default_rng(11)
    for n, (rows, vocab) in enumerate(SIZES):
        gap, shift = ((0, 0), (5, 1), (8, 8))[n % 3]
        scale = float(np.float32((1.0, 0.7, 1.3)[n % 3]))       # the call takes the scale in 32 bits
        logits = logits_of(kind, rows, vocab, dtype, rng, gap, shift)
        x = f64(logits)
        targets = rng.integers(0, vocab, rows)
        targets[2::4] = -1
        t = up(targets.astype(np.int32 if n % 2 else np.int64))
        _lp, lse, ent, _p = R.logprobs(x, scale)
        lse, ent = up(lse.astype(np.float32)), up(ent.astype(np.float32))
        dlogp, dent = up(rng.standard_normal(rows).astype(np.float32)), up(rng.standard_normal(rows).astype(np.float32))
        for b in (None, dent):
            d = torch.full((rows, vocab + 3), 9.0, dtype=TYPES[dtype], device="cuda")
            dcr.dcr_logprobs_grad(logits, t, lse, dlogp, d[:, :vocab], entropy=ent if b is not None else None, dentropy=b,
                                  scale=scale)
            a = np.where(targets < 0, 0, f64(dlogp))[:, None]
            be, h = (np.zeros((rows, 1)), 0) if b is None else (f64(b)[:, None], f64(ent)[:, None])
            low = f64(lse)[:, None]
            empty = np.isneginf(low)
            with np.errstate(invalid="ignore"):
                l = np.where(empty, -np.inf, x * scale - low)
            p = np.exp(l)
            ll = np.where(p > 0, l, 0)
            hot = np.zeros_like(x)
            hot[np.arange(rows), np.maximum(targets, 0)] = 1
            want = scale * (a * (hot - p) - be * p * (ll + h)) * ~empty
            most = scale * p * (np.abs(a) + np.abs(be) * (np.abs(ll) + np.abs(h)))
            tol = most * (3 * np.abs(ll) + 8) * 2.0 ** -23 + 2.0 ** -23 * scale * hot * np.abs(a)
            err = np.abs(f64(d[:, :vocab]) - want)
            assert (err <= tol + HALF[dtype] * (np.abs(want) + tol) + 2.0 ** -126).all(), (rows, vocab, (err - tol).max())
            assert (d[:, vocab:] == 9).all()
        copy = logits.clone()
        dcr.dcr_logprobs_grad(copy, t, lse, dlogp, copy, entropy=ent, dentropy=dent, scale=scale)     # in place
        assert torch.equal(copy, d[:, :vocab])


def test_grad_against_differences():
    """logp and entropy as the calls give them, their derivative along a direction against central differences of the
    64-bit reference (h = 1e-4: off by h^2 and 2^-52 / h; the gradient itself by 2^-20 of its terms)."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((4, 50)) * 2
    t = np.array([3, -1, 49, 0])
    a, b = rng.standard_normal(4), rng.standard_normal(4)
    scale = float(np.float32(0.8))
    logits = up(x.astype(np.float32))
    x = f64(logits)
    lse, ent = torch.empty(4, device="cuda"), torch.empty(4, device="cuda")
    targets = up(t)
    dcr.dcr_logprobs(logits, targets, None, lse, ent, scale=scale, workspace=dcr.step_workspace())
    d = torch.empty_like(logits)
    dcr.dcr_logprobs_grad(logits, targets, lse, up(a.astype(np.float32)), d, entropy=ent, dentropy=up(b.astype(np.float32)),
                          scale=scale)

    def value(y):
        lp, _lse, h, _p = R.logprobs(y, scale)
        return sum(a[r] * lp[r, t[r]] for r in range(4) if t[r] >= 0) + (b * h).sum()
    for _ in range(20):
        u = rng.standard_normal(x.shape)
        got = (f64(d) * u).sum()
        want = (value(x + 1e-4 * u) - value(x - 1e-4 * u)) / 2e-4
        assert abs(got - want) < 2e-5 * max(1, np.abs(f64(d) * u).sum())


def test_grad_of_odd_targets():
    x = torch.randn(4, 100, device="cuda")
    lse = torch.logsumexp(x, 1)
    d = torch.empty_like(x)
    one = torch.ones(4, device="cuda")
    dcr.dcr_logprobs_grad(x, torch.tensor([-1, 100, 1 << 35, 5], device="cuda"), lse, one, d)
    assert (d[0] == 0).all() and torch.isnan(d[1:3]).all() and not torch.isnan(d[3]).any()
    lse[0], lse[3] = -INF, float("nan")
    dcr.dcr_logprobs_grad(x, torch.tensor([7, 7, 7, 5], device="cuda"), lse, one, d)
    assert (d[0] == 0).all() and torch.isnan(d[3]).all() and not torch.isnan(d[1:3]).any()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,vocab", [(4, 700), (300, 5000), (5000, 1100)])
def test_top_of_rows_with_nan(rows, vocab, dtype):
    """Numbers first, -infinity behind them, then NaN by their indices; rows of all NaN, of nearly nothing else, with equals
    at the end of what is asked for."""
    rng = np.random.default_rng(vocab)
    x = np.round(rng.standard_normal((rows, vocab)) * 4) / 4
    x[0] = np.nan
    x[1] = np.where(rng.random(vocab) < 0.98, np.nan, x[1])
    x[2, : vocab - 30] = np.nan
    x[3, 30:] = -np.inf
    x[3, 40: vocab // 2] = np.nan
    logits = up(x.astype(np.float32)).to(TYPES[dtype])
    order = np.lexsort((np.arange(vocab)[None].repeat(rows, 0), -(np.nan_to_num(x, nan=-np.inf) + 0.0), np.isnan(x)), axis=1)
    for top in (1, 20, 33, 64):
        ids, vals = torch.empty(rows, top, dtype=torch.int32, device="cuda"), torch.empty(rows, top, device="cuda")
        dcr.dcr_logprobs(logits, None, top_ids=ids, top_values=vals, workspace=dcr.step_workspace())
        assert np.array_equal(ids.cpu().numpy(), order[:, :top])
        nan = torch.isnan(vals)
        assert nan[:4][[0, 1, 2, 3]].all() and not nan[4:].any()


def test_rows_past_32_bits():
    """A row that begins more than 2^32 elements into its matrix."""
    pool = torch.zeros((1 << 32) + (1 << 13), dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(pool, (3, 4100), (1 << 31, 1))
    x[2, 4099] = 3.0
    lp = torch.empty(3, device="cuda")
    ids, vals = torch.empty(3, 2, dtype=torch.int32, device="cuda"), torch.empty(3, 2, device="cuda")
    lse = torch.empty(3, device="cuda")
    t = torch.tensor([5, 5, 4099], device="cuda")
    dcr.dcr_logprobs(x, t, lp, lse, top_ids=ids, top_values=vals, workspace=dcr.step_workspace())
    assert ids.tolist() == [[0, 1], [0, 1], [4099, 0]]
    want = torch.log_softmax(x.double(), 1)
    assert torch.allclose(lp.double(), want[torch.arange(3), t.cpu()], atol=1e-5)
    one = torch.ones(3, device="cuda")
    dcr.dcr_logprobs_grad(x, t, lse, one, x)
    got = 1 - torch.exp(want[2, 4099])
    assert abs(float(x[2, 4099]) - float(got)) < 2.0 ** -8 and float(x[2, 0]) < 0


# rows and vocabulary so that a row goes to one wave, to several, to one workgroup, to several
SPLITS = [(4100, 1500), (4097, 66000), (1100, 65600), (2048, 65536), (2100, 65544), (4095, 65537), (1500, 9001), (1023, 70000),
          (256, 40001), (341, 33333), (700, 2047), (1024, 1025), (1025, 20000)]


@pytest.mark.parametrize("rows,vocab", SPLITS)
def test_every_split(rows, vocab):
    """Against 64-bit arithmetic on the GPU, with the workspace at the end of a larger buffer: nothing is written behind it.
    (Tolerances as above, with log p and the entropy below 2^5.)"""
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    x = torch.empty(rows, vocab + 8, dtype=torch.bfloat16, device="cuda")[:, :vocab]
    for part in x.split(512):
        part.copy_(torch.randn(part.shape, device="cuda", generator=g) * 3)
    x[3] = -INF
    x[5, : vocab // 2] = -INF
    x[7] = x[7].sort().values                     # rising
    x[9] = 1.0                                    # all alike
    t = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
    buffer = torch.full((dcr.STEP_WORKSPACE_BYTES + (1 << 20),), 0xAB, dtype=torch.uint8, device="cuda")
    ws = buffer[: dcr.STEP_WORKSPACE_BYTES]
    for top in (0, 20, 64):
        out = [torch.full((rows,), 77.0, device="cuda") for _ in range(3)]
        ids = torch.full((rows, top), -5, dtype=torch.int32, device="cuda") if top else None
        vals = torch.full((rows, top), 77.0, device="cuda") if top else None
        dcr.dcr_logprobs(x, t, *out, ids, vals, workspace=ws)
        assert (buffer[dcr.STEP_WORKSPACE_BYTES:] == 0xAB).all()
        for i in range(0, rows, 256):
            y = x[i:i + 256].double()
            lse = torch.logsumexp(y, 1)
            lp = torch.where(torch.isneginf(lse)[:, None], -INF, y - lse[:, None])
            ent = -(lp.exp() * torch.where(lp.exp() > 0, lp, 0.0)).sum(1)
            tol = (vocab / 256 + 40) * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -21
            mine = lp.gather(1, t[i:i + 256, None])[:, 0]
            for got, want, wide in ((out[0], mine, 2.0 ** -17), (out[1], lse, 2.0 ** -18), (out[2], ent, 64 * tol)):
                got = got[i:i + 256].double()
                none = torch.isneginf(want)
                assert torch.equal(torch.isneginf(got), none)
                assert ((got - want)[~none].abs() <= tol + wide).all()
            if top:
                # logits first, then indices: the lowest of equals (both exact in 64 bits)
                key = torch.where(torch.isneginf(y), -1e9, y * 2.0 ** 24) * 2.0 ** 20 - torch.arange(vocab, device="cuda", dtype=torch.float64)
                best = key.topk(top, 1).indices
                assert torch.equal(ids[i:i + 256].long(), best), (i, top)
                want = lp.gather(1, best)
                none = torch.isneginf(want)
                got = vals[i:i + 256].double()
                assert torch.equal(torch.isneginf(got), none) and ((got - want)[~none].abs() <= tol + 2.0 ** -17).all()


# (rows, vocabulary): a wave a row, a workgroup a row, parts of both kinds
FORMS = [(10, 300), (10, 5001), (10, 70000), (1100, 65600), (4100, 1500), (1030, 9001), (300, 30001)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("mask", [-1e4, -1e9, -1e10, -1e12, -1e20, -1e25, -1e30, -2.0 ** 100, -2e30, -3.3895e38])
def test_finite_masks_are_numbers(mask, dtype):
    """Masks by finite numbers of any size, at any scale: of whole rows (uniform then), of a tail and of every second half of
    what a thread, a wave or a part sees, of all but one token, with both largest in turn.  Against 64 bits on the GPU; the
    largest's product with the scale is rounded in lse, and a difference twice in log p: 2^-22 of themselves; the sums as
    in tolerances()."""
    for n, (rows, vocab) in enumerate(FORMS):
        g = torch.Generator(device="cuda")
        g.manual_seed(n)
        scale = float(np.float32((1.0, 0.7, 2.5, 0.01)[n % 4]))
        x = torch.empty(rows, vocab, dtype=TYPES[dtype], device="cuda")
        for part in x.split(256):
            part.copy_(torch.randn(part.shape, device="cuda", generator=g) * 3)
        j = torch.arange(vocab, device="cuda")
        x[0] = mask
        x[1, vocab // 3:] = mask                           # a padded vocabulary
        x[2, 1:] = mask                                    # one open token, at the front and at the end
        x[7, :-1] = mask
        for r, width in enumerate((8, 128, 1024, 2048)):   # stretches
            x[r + 3, (j // width) % 2 == 0] = mask
        x[rows - 1, ::2], x[rows - 1, 1::2] = mask, 2 * mask if abs(mask) < 1e38 else mask
        t = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
        top = min(7, vocab)
        ws = dcr.step_workspace()
        for some in (0, top):
            out = [torch.full((rows,), 77.0, device="cuda") for _ in range(3)]
            ids = torch.full((rows, top), -5, dtype=torch.int32, device="cuda") if some else None
            vals = torch.full((rows, top), 77.0, device="cuda") if some else None
            dcr.dcr_logprobs(x, t, *out, ids, vals, scale=scale, workspace=ws)
            grow = (vocab / 256 + 40) * 2.0 ** -24 + 2.0 ** -21
            for i in range(0, rows, 256):
                y = x[i:i + 256].double() * scale
                most = y.amax(1, keepdim=True)
                d = y - most
                log_s = d.exp().sum(1, keepdim=True).log()
                lp = d - log_s
                ent = -(lp.exp() * lp.clamp(min=-800)).sum(1)
                mine = lp.gather(1, t[i:i + 256, None])[:, 0]
                want = [mine, (most + log_s)[:, 0], ent]
                tol = [grow + 2.0 ** -20 + 2.0 ** -22 * mine.abs(), grow + 2.0 ** -20 + 2.0 ** -23 * want[1].abs(),
                       2 * grow * (1 + ent) + 2.0 ** -20]
                for name, a, b, c in zip(("logp", "lse", "entropy"), out, want, tol):
                    a = a[i:i + 256].double()
                    low = b < -3.4028e38                   # (beyond the numbers of 32 bits)
                    assert torch.isfinite(a[~low]).all() and (a[low] <= -3.4028e38).all(), (rows, vocab, some, name)
                    assert ((a - b).abs() <= c)[~low].all(), (rows, vocab, some, name, (a - b).abs()[~low].max())
                if some:
                    best = lp.gather(1, ids[i:i + 256].long())
                    got = vals[i:i + 256].double()
                    low = best < -3.4028e38
                    assert ((got - best).abs() <= grow + 2.0 ** -20 + 2.0 ** -22 * best.abs())[~low].all(), (rows, vocab)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_peaked_rows_have_no_positive_log_probabilities(dtype):
    """One token far above the others: its log probability is at most 0 and the entropy at least 0, and where all others
    together weigh less than 2^-26 the sum is 1 and log p is 0 to within their weight.  (The largest term is 1 itself, so no
    sum is below it, and what is added to 1 is rounded to 1 below 2^-24.)"""
    rng = np.random.default_rng(51)
    ws = dcr.step_workspace()
    for rows, vocab in ((3000, 2000), (700, 900), (64, 20000), (1100, 65600), (4100, 1500)):
        g = torch.Generator(device="cuda")
        g.manual_seed(vocab)
        x = torch.empty(rows, vocab, dtype=TYPES[dtype], device="cuda")
        for part in x.split(256):
            part.copy_(torch.randn(part.shape, device="cuda", generator=g))
        at = torch.randint(0, vocab, (rows, 1), device="cuda", generator=g)
        x.scatter_(1, at, (25 + 20 * torch.rand(rows, 1, device="cuda", generator=g)).to(x.dtype))
        for scale in (1.0, float(np.float32(0.7)), float(np.float32(1.3))):
            lp, lse, ent = (torch.full((rows,), 77.0, device="cuda") for _ in range(3))
            ids, vals = torch.empty(rows, 2, dtype=torch.int32, device="cuda"), torch.empty(rows, 2, device="cuda")
            dcr.dcr_logprobs(x, at[:, 0], lp, lse, ent, ids, vals, scale=scale, workspace=ws)
            assert torch.equal(ids[:, :1].long(), at) and torch.equal(vals[:, 0], lp)
            assert (lp <= 0).all() and (ent >= 0).all(), (rows, vocab, scale, float(lp.max()), float(ent.min()))
            for i in range(0, rows, 256):
                y = x[i:i + 256].double() * scale
                y -= y.amax(1, keepdim=True)
                rest = y.exp().sum(1) - 1
                sharp = rest < 2.0 ** -26
                assert (lp[i:i + 256].double() + rest)[sharp].abs().max() <= 2.0 ** -26 if sharp.any() else True


GRAD_FORMS = [(6, 300), (300, 77), (5, 2047), (5, 5001), (3, 70000), (700, 2500), (40, 32000)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["lowest", "all lowest", "1e10", "1e30", "shifted", "far shifted", "rising", "padded"])
def test_grad_is_that_of_the_log_probabilities(kind, dtype):
    """Against the gradient in 64 bits from the logits themselves, with the lse that the forward call gives.  A term p is off
    by the rounding of log p (3 |log p| + 8) 2^-23, by half a step of lse where that is below 64 (2^-19), else by its own
    sum's (vocab / 256 + 40) 2^-24 and 2^-20.  A row's terms add up to what the rounding of p leaves of |dlogp|."""
    rng = np.random.default_rng(61)
    ws = dcr.step_workspace()
    for n, (rows, vocab) in enumerate(GRAD_FORMS):
        gap, shift = ((0, 0), (5, 1), (8, 8))[n % 3]
        scale = float(np.float32((1.0, 0.7, 1.4)[n % 3]))
        x = rng.standard_normal((rows, vocab)) * 3
        some = rng.random((rows, vocab)) < 0.5
        if kind in ("lowest", "1e10", "1e30"):
            x[some] = {"lowest": -3.3895e38, "1e10": -1e10, "1e30": -1e30}[kind]
            x[::3] = {"lowest": -3.3895e38, "1e10": -1e10, "1e30": -1e30}[kind]
        elif kind == "all lowest":
            x[:] = -3.3895e38
        elif kind == "shifted":
            x += np.where(np.arange(rows) % 2, 1000, -70)[:, None]
        elif kind == "far shifted":
            x = np.round(x) * 4096 + 1e5
        elif kind == "rising":
            x = np.sort(x, 1) * 8
        elif kind == "padded":
            x = x - 90
            x[:, vocab * 2 // 3:] = -np.inf
            x[::5] = -np.inf
        logits = torch.empty(rows, vocab + gap + shift, dtype=TYPES[dtype], device="cuda")[:, shift: shift + vocab]
        logits.copy_(up(x.astype(np.float32)))
        x = f64(logits)
        targets = rng.integers(0, vocab, rows)
        targets[2::4] = -1
        t = up(targets)
        lse = torch.empty(rows, device="cuda")
        dcr.dcr_logprobs(logits, t, lse=lse, scale=scale, workspace=ws)
        lp, lse64, ent64, p = R.logprobs(x, scale)
        ent = up(ent64.astype(np.float32))
        dlogp, dent = up(rng.standard_normal(rows).astype(np.float32)), up(rng.standard_normal(rows).astype(np.float32))
        hot = np.zeros_like(x)
        hot[np.arange(rows), np.maximum(targets, 0)] = 1
        open_rows = ~np.isneginf(lse64)[:, None]
        grow = (vocab / 256 + 40) * 2.0 ** -24 + 2.0 ** -20
        for b in (None, dent):
            d = torch.full((rows, vocab + 3), 9.0, dtype=TYPES[dtype], device="cuda")
            dcr.dcr_logprobs_grad(logits, t, lse, dlogp, d[:, :vocab], entropy=ent if b is not None else None, dentropy=b, scale=scale)
            a = np.where(targets < 0, 0, f64(dlogp))[:, None]
            be, h = (np.zeros((rows, 1)), 0) if b is None else (f64(b)[:, None], f64(ent)[:, None])
            ll = np.where(p > 0, lp, 0)
            want = scale * (a * (hot - p) - be * p * (ll + h)) * open_rows
            off = (3 * np.abs(ll) + 8) * 2.0 ** -23 + 2.0 ** -19 + grow
            # (p off by `off` of itself, and log p by the same where the entropy's part multiplies it)
            most = scale * p * ((np.abs(a) + np.abs(be) * (np.abs(ll) + np.abs(h))) * off + np.abs(be) * off)
            tol = most + 2.0 ** -23 * scale * hot * np.abs(a)
            # (an exponential below 2^-126 is 0: p is off by as much, times what it is multiplied with)
            tol = tol + 2.0 ** -126 * scale * (np.abs(a) + np.abs(be) * (np.abs(ll) + np.abs(h)))
            err = np.abs(f64(d[:, :vocab]) - want)
            assert (err <= tol + HALF[dtype] * (np.abs(want) + tol) + 2.0 ** -126).all(), (rows, vocab, b is None, np.max(err - tol))
            assert (d[:, vocab:] == 9).all()
            if dtype == "fp32":
                total = np.abs(f64(d[:, :vocab]).sum(1))
                assert (total <= (tol + 2.0 ** -24 * np.abs(want)).sum(1) + 2.0 ** -40).all(), (rows, vocab)
        copy = torch.empty(rows, vocab + gap + shift, dtype=TYPES[dtype], device="cuda")[:, shift: shift + vocab].copy_(logits)
        dcr.dcr_logprobs_grad(copy, t, lse, dlogp, copy, entropy=ent, dentropy=dent, scale=scale)     # in place
        assert torch.equal(copy, d[:, :vocab])


def test_grad_with_a_foreign_lse():
    """An lse that is not these logits' own (of a vocabulary that several GPUs share, say) is taken as it is given, near 0 and
    far from it: p = exp(scale x - lse), rounded as |lse| has it."""
    rng = np.random.default_rng(62)
    for rows, vocab in ((9, 300), (9, 6000)):
        for base in (0.0, 90.0, -500.0):
            x = (base + rng.standard_normal((rows, vocab))).astype(np.float32)
            lse = (R.logprobs(x, 1.0)[1] + np.linspace(0.01, 3, rows)).astype(np.float32)
            d = torch.empty(rows, vocab, device="cuda")
            one = torch.ones(rows, device="cuda")
            dcr.dcr_logprobs_grad(up(x), torch.full((rows,), 3, device="cuda"), up(lse), one, d)
            l = x.astype(np.float64) - lse.astype(np.float64)[:, None]
            want = -np.exp(l)
            want[:, 3] += 1
            tol = np.exp(l) * ((3 * np.abs(l) + 8) * 2.0 ** -23)
            assert (np.abs(f64(d) - want) <= tol + 2.0 ** -23).all(), (rows, base)


@pytest.mark.parametrize("rows,vocab", [(9, 700), (9, 5001), (5, 70000)])
def test_scales_up_to_the_largest_number(rows, vocab):
    """A temperature near 0: the largest logit (the equal ones in equal parts) has all of the probability, no sum is lost to
    a scale that leaves the numbers of 32 bits in another base; and a scale near 0 makes all alike."""
    rng = np.random.default_rng(vocab)
    x = rng.integers(-50, 50, (rows, vocab)).astype(np.float32)
    x[:, :3] = -60
    x[1] = 7
    x[2, :vocab // 2] = -np.inf
    t = x.argmax(1)
    most = x.max(1)
    equal = (x == most[:, None]).sum(1)
    for scale in (3.4e38, 2.0 ** 127, 2.4e38, 1e30):
        lp, lse, ent = (torch.full((rows,), 77.0, device="cuda") for _ in range(3))
        logits = up(x)
        dcr.dcr_logprobs(logits, up(t), lp, lse, ent, scale=scale, workspace=dcr.step_workspace())
        for got, want in ((lp, -np.log(equal)), (ent, np.log(equal))):
            assert (np.abs(f64(got) - want) <= 2.0 ** -20 + (vocab / 256 + 40) * 2.0 ** -24).all(), scale
        assert torch.isfinite(lse).all()
        d, one = torch.empty_like(logits), torch.ones(rows, device="cuda")
        dcr.dcr_logprobs_grad(logits, torch.full((rows,), -1, device="cuda"), lse, one, d, entropy=ent, dentropy=one * 0, scale=scale)
        assert (d == 0).all()                              # (no target, no weight of the entropy)
    lp, lse, ent = (torch.full((rows,), 77.0, device="cuda") for _ in range(3))
    dcr.dcr_logprobs(up(x), up(t), lp, lse, ent, scale=2.0 ** -140, workspace=dcr.step_workspace())
    n = np.isfinite(x).sum(1)
    assert (np.abs(f64(lp) + np.log(n)) <= 2.0 ** -19 + (vocab / 256 + 40) * 2.0 ** -24).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("vocab", [1, 5, 8, 9, 30, 95, 96, 97, 104, 511])
def test_grad_of_short_rows_with_a_far_lse(vocab, dtype):
    """Rows of a thread's and of a wave's, near and far ones side by side, as given and in place.  (Off as above, and what
    an exponential below 2^-126 leaves.)"""
    rng = np.random.default_rng(vocab)
    rows = 137
    x = rng.standard_normal((rows, vocab)) * 2 + rng.choice([0, 0, 50, -90, 3000, -1e5, 1e20], (rows, 1))
    x[::9] = -np.inf
    x[4::9, vocab // 2:] = -np.inf
    logits = torch.empty(rows, vocab + 3, dtype=TYPES[dtype], device="cuda")[:, 1:vocab + 1].copy_(up(x.astype(np.float32)))
    x = f64(logits)
    t = rng.integers(-1, vocab, rows)
    lse = torch.empty(rows, device="cuda")
    dcr.dcr_logprobs(logits, None, lse=lse, workspace=dcr.step_workspace())
    lp, lse64, ent64, p = R.logprobs(x, 1.0)
    a, b = up(rng.standard_normal(rows).astype(np.float32)), up(rng.standard_normal(rows).astype(np.float32))
    ent = up(ent64.astype(np.float32))
    out = torch.full((rows, vocab + 3), 9.0, dtype=TYPES[dtype], device="cuda")
    dcr.dcr_logprobs_grad(logits, up(t), lse, a, out[:, :vocab], entropy=ent, dentropy=b)
    hot = np.zeros_like(x)
    hot[np.arange(rows), np.maximum(t, 0)] = 1
    aa, be, h = np.where(t < 0, 0, f64(a))[:, None], f64(b)[:, None], f64(ent)[:, None]
    ll = np.where(p > 0, lp, 0)
    want = (aa * (hot - p) - be * p * (ll + h)) * ~np.isneginf(lse64)[:, None]
    off = (3 * np.abs(ll) + 8) * 2.0 ** -23 + 2.0 ** -19 + (vocab / 256 + 40) * 2.0 ** -24 + 2.0 ** -20
    size = np.abs(aa) + np.abs(be) * (np.abs(ll) + np.abs(h))
    tol = p * (size + np.abs(be)) * off + 2.0 ** -23 * hot * np.abs(aa) + 2.0 ** -126 * (size + 1)
    assert (np.abs(f64(out[:, :vocab]) - want) <= tol + HALF[dtype] * (np.abs(want) + tol)).all()
    assert (out[:, vocab:] == 9).all()
    dcr.dcr_logprobs_grad(logits, up(t), lse, a, logits, entropy=ent, dentropy=b)
    assert torch.equal(logits, out[:, :vocab])
