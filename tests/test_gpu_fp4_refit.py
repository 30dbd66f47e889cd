"""Refits of 4-bit weights that go wrong, that share a GPU with products on other streams, and products of groups."""
import numpy as np
import pytest
import torch

from bit_exact_xor_amd import dcr, pipeline
from tests import fp4_ref as R
from tests.test_gpu_fp4 import bound, f64, up

pytestmark = pytest.mark.gpu
SHAPES = [(768, 2048), (130, 96), (33, 70)]


def weights(seed, shapes=SHAPES):
    rng = np.random.default_rng(seed)
    return [up((0.02 * rng.standard_normal(s)).astype(np.float32)) for s in shapes]


def check_held(link, fmt, w):
    """The receiver holds the bytes of w, under the tensor scale that the sender took."""
    for t, q, sent in zip(w, link.held, link.sent):
        s = float(q.tensor_scale) if fmt == R.NV else 1.0
        assert fmt == R.MX or s == float(sent.tensor_scale)
        c, b = R.quantize(t.cpu().numpy(), fmt, s)
        assert np.array_equal(q.codes.cpu().numpy()[:, :c.shape[1]], c)
        assert np.array_equal(q.scales.cpu().numpy(), b)


@pytest.mark.parametrize("fmt", [R.MX, R.NV])
@pytest.mark.parametrize("where", ["send", "apply", "refused"])
@pytest.mark.parametrize("then", ["same", "other", "recover"])
def test_refit_after_a_failure(fmt, where, then, monkeypatch):
    """A refit that fails before, within or after its applies leaves weights that no product takes; the next refit, or
    recover(), ends at the bytes it should have given."""
    link = pipeline.Fp4Refit(SHAPES, fmt)
    w0, w1, w2 = weights(0), weights(1), weights(2)
    link.refit(w0)
    x = torch.ones(3, 2048, dtype=torch.bfloat16, device="cuda")
    real = dcr.dcr_apply

    def broken_apply(plan, canon, header, dirs, payload, flags, first, n, *rest, **kw):
        real(plan, canon, header, dirs, payload, flags, first, max(1, n // 2), *rest, **kw)
        raise RuntimeError("planted")

    def broken_wait(*_args):
        raise RuntimeError("planted")

    def refusing_result(t):
        r = np.zeros(1, dcr.APPLY_RESULT)
        r["n_invalid"] = 1
        return r[0]

    with monkeypatch.context() as mp:
        if where == "apply":
            mp.setattr(dcr, "dcr_apply", broken_apply)
        elif where == "send":
            mp.setattr(dcr, "dcr_ready_wait", broken_wait)
        else:
            mp.setattr(dcr, "apply_result", refusing_result)
        with pytest.raises(RuntimeError):
            link.refit(w1)
        assert link.version == 1
    with pytest.raises(dcr.DcrError):
        link.matmul(0, x)
    if then == "recover":
        link.recover()
        assert link.version == 2
        check_held(link, fmt, w1)
        link.matmul(0, x)
    w = w2 if then == "other" else w1
    link.refit(w)
    assert link.version == 3
    check_held(link, fmt, w)
    assert link.refit(w) == 0
    y = torch.empty(3, 768, device="cuda")
    dcr.dcr_fp4_matmul(x, link.sent[0], y, None, link.fp4_workspace)
    assert torch.equal(link.matmul(0, x, torch.float32), y)


def test_refit_refused_before_it_sends():
    """Weights of a wrong shape are refused before anything travels: products and the next refit are as if not called."""
    link = pipeline.Fp4Refit(SHAPES, R.NV)
    w0 = weights(0)
    link.refit(w0)
    w1 = weights(1)
    with pytest.raises(ValueError):
        link.refit([w1[0], w1[1], w1[2][:, 1:]])
    link.matmul(1, torch.ones(3, 96, dtype=torch.bfloat16, device="cuda"))
    check_held(link, R.NV, w0)
    link.refit(w1)
    assert link.version == 2
    check_held(link, R.NV, w1)
    link.recover()
    assert link.version == 2


def test_refit_waits_for_products_on_other_streams():
    """A product enqueued on a side stream before a refit reads the weights from before it."""
    link = pipeline.Fp4Refit(SHAPES, R.MX)
    link.refit(weights(0))
    x = up(np.random.default_rng(5).standard_normal((40, 2048))).bfloat16()
    old = link.matmul(0, x, torch.float32)
    busy, sides = torch.zeros(1 << 26, device="cuda"), [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for side in sides:
        with torch.cuda.stream(side):
            for _ in range(500):          # keeps the stream from its product for some time
                busy.add_(1)
            got.append(link.matmul(0, x, torch.float32))
    assert not any(s.query() for s in sides)
    link.refit(weights(1))
    new = link.matmul(0, x, torch.float32)
    torch.cuda.synchronize()
    assert all(torch.equal(y, old) for y in got)
    assert not torch.equal(new, old)


def test_products_on_two_streams_at_once():
    """Products that split their sums, on two streams together with a refit that takes tensor scales: the results of
    one after the other."""
    shape = (136, 4096)
    link = pipeline.Fp4Refit([shape], R.NV)
    w = weights(0, [shape])
    link.refit(w)
    rng = np.random.default_rng(6)
    xs = [up(rng.standard_normal((700, 4096))).bfloat16() for _ in range(2)]
    want = [link.matmul(0, x, torch.float32) for x in xs]
    sides = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(40):
        for i, side in enumerate(sides):
            with torch.cuda.stream(side):
                got[i].append(link.matmul(0, xs[i], torch.float32))
    link.refit(w, calibrate=True)
    torch.cuda.synchronize()
    for ys, t in zip(got, want):
        assert all(torch.equal(y, t) for y in ys)
    check_held(link, R.NV, w)


def test_captured_product():
    """A product captured into a graph, replayed beside eager ones on another stream and after a refit."""
    shape = (136, 4096)
    link = pipeline.Fp4Refit([shape], R.NV)
    rng = np.random.default_rng(7)
    x, z = (up(rng.standard_normal((700, 4096))).bfloat16() for _ in range(2))
    link.refit(weights(0, [shape]))
    want_z = link.matmul(0, z, torch.float32)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = link.matmul(0, x, torch.float32)
    side = torch.cuda.Stream()
    for seed in (0, 1, 2):
        if seed:
            link.refit(weights(seed, [shape]))
            want_z = link.matmul(0, z, torch.float32)
        want = link.matmul(0, x, torch.float32)
        torch.cuda.synchronize()
        for _ in range(3):
            y.zero_()
            with torch.cuda.stream(side):
                others = [link.matmul(0, z, torch.float32) for _ in range(4)]
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want)
            assert all(torch.equal(o, want_z) for o in others)


def late(stream, busy):
    """Work that keeps `stream` busy for some time."""
    with torch.cuda.stream(stream):
        for _ in range(500):
            busy.add_(1)


def test_refused_on_one_stream_refitted_on_another():
    """What a refused refit has enqueued on its stream does not reach the next one's weights."""
    link = pipeline.Fp4Refit(SHAPES, R.MX)
    w0, w1 = weights(0), weights(1)
    link.refit(w0)
    side, busy = torch.cuda.Stream(), torch.zeros(1 << 26, device="cuda")
    torch.cuda.synchronize()
    late(side, busy)
    with torch.cuda.stream(side), pytest.raises(ValueError):
        link.refit([w0[0] + 1, w0[1] + 1, w0[2][:, 1:]])
    link.refit(w1)
    torch.cuda.synchronize()
    check_held(link, R.MX, w1)
    assert all(torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales) for a, b in zip(link.held, link.sent))
    assert link.refit(w1) == 0


def test_made_on_one_stream_used_on_another():
    """The first refit on another stream than the object was made on: its buffers hold what they should by then."""
    side, busy = torch.cuda.Stream(), torch.zeros(1 << 26, device="cuda")
    torch.cuda.synchronize()
    late(side, busy)
    with torch.cuda.stream(side):
        link = pipeline.Fp4Refit(SHAPES, R.NV)
    w = weights(0)
    link.refit(w)
    torch.cuda.synchronize()
    check_held(link, R.NV, w)
    assert link.refit(w) == 0


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two GPUs")
def test_weights_on_another_gpu():
    """Refit, recovery and product with the weights on a GPU that is not the current one."""
    link = pipeline.Fp4Refit(SHAPES, R.NV, device="cuda:1")
    for seed in (0, 1):
        w = [t.to("cuda:1") for t in weights(seed)]
        link.refit(w)
        check_held(link, R.NV, w)
    link.interrupted = True
    link.recover()
    y = link.matmul(0, torch.ones(3, 2048, dtype=torch.bfloat16, device="cuda:1"), torch.float32)
    v = R.unit_values(link.held[0].codes.cpu().numpy(), link.held[0].scales.cpu().numpy(), 2048, R.NV)
    s = float(link.held[0].tensor_scale)
    ref, size = R.product(np.ones((3, 2048)), v)
    assert torch.cuda.current_device() == 0 and (np.abs(f64(y) - ref * s) <= bound(size * s, ref * s, 2048, "fp32")).all()


def test_device_is_the_one_it_was_made_on():
    assert pipeline.Fp4Refit([(4, 32)], R.MX).device == torch.device("cuda", torch.cuda.current_device())
    with pytest.raises(ValueError):
        pipeline.Fp4Refit([(4, 32)], R.MX, device="cpu")


@pytest.mark.parametrize("dtype", [torch.float32, None])
def test_product_rows_of_no_group_are_zeros(dtype):
    """Rows in front of the first group and behind the last one (a padded batch) come back as zeros."""
    link = pipeline.Fp4Refit([(4 * 48, 64)], R.MX)
    w = weights(3, [(4 * 48, 64)])
    link.refit(w)
    x = up(np.random.default_rng(8).integers(-2, 3, (64, 64))).bfloat16()
    off = [5, 20, 20, 41, 50]
    torch.full((64, 48), 99.0, dtype=dtype or torch.bfloat16, device="cuda")    # (freed: what new memory holds)
    y = f64(link.matmul(0, x, dtype, torch.tensor(off, dtype=torch.int32, device="cuda")))
    c, b = R.quantize(w[0].cpu().numpy(), R.MX)
    ref, size = R.product(f64(x), R.unit_values(c, b, 64, R.MX), off)
    rows = np.isnan(ref).all(1)
    assert rows.sum() == 19 and (y[rows] == 0).all()
    assert (np.abs(y - ref) <= bound(size, ref, 64, "fp32" if dtype else "bf16"))[~rows].all()


def test_product_into_a_tensor():
    """Results in the caller's tensor: rows of no group as they were."""
    link = pipeline.Fp4Refit([(4 * 48, 64)], R.MX)
    link.refit(weights(3, [(4 * 48, 64)]))
    x = up(np.random.default_rng(8).integers(-2, 3, (64, 64))).bfloat16()
    off = torch.tensor([5, 20, 20, 41, 50], dtype=torch.int32, device="cuda")
    want = link.matmul(0, x, torch.float32, off)
    y = torch.full((64, 48), 99.0, device="cuda")
    assert link.matmul(0, x, offsets=off, y=y) is y
    assert torch.equal(y[5:50], want[5:50]) and (y[:5] == 99.0).all() and (y[50:] == 99.0).all()
    with pytest.raises(ValueError):
        link.matmul(0, x, offsets=off, y=y[:, 1:])


def test_product_refuses_offsets():
    link = pipeline.Fp4Refit([(4 * 48, 64)], R.MX)
    x = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    for off in (torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda"),
                torch.zeros(5, device="cuda"), torch.zeros(6, dtype=torch.int32, device="cuda")):
        with pytest.raises(ValueError):
            link.matmul(0, x, offsets=off)


@pytest.mark.parametrize("fmt", [R.MX, R.NV])
def test_recovery_with_nothing_to_send(fmt, monkeypatch):
    """A refit of unchanged weights that is interrupted: recover() has no records to apply."""
    link = pipeline.Fp4Refit(SHAPES, fmt)
    w = weights(0)
    link.refit(w)

    def broken_wait(*_args):
        raise RuntimeError("planted")

    for _ in range(2):
        with monkeypatch.context() as mp:
            mp.setattr(dcr, "dcr_ready_wait", broken_wait)
            with pytest.raises(RuntimeError):
                link.refit(w)
        link.recover()
    assert link.version == 3 and link.refit(w) == 0
    check_held(link, fmt, w)


@pytest.mark.parametrize("fmt", [R.MX, R.NV])
def test_first_refit_interrupted(fmt, monkeypatch):
    """The first refit, which takes the NV tensor scales, finished by the second."""
    link = pipeline.Fp4Refit(SHAPES, fmt)
    real = dcr.dcr_apply

    def broken_apply(plan, canon, header, dirs, payload, flags, first, n, *rest, **kw):
        real(plan, canon, header, dirs, payload, flags, first, max(1, n // 2), *rest, **kw)
        raise RuntimeError("planted")

    with monkeypatch.context() as mp:
        mp.setattr(dcr, "dcr_apply", broken_apply)
        with pytest.raises(RuntimeError):
            link.refit(weights(0))
    w = weights(1)
    link.refit(w)
    assert link.version == 2
    check_held(link, fmt, w)
