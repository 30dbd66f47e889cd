"""AdamW steps on the GPU against a plain 64-bit implementation."""
import numpy as np
import pytest
import torch

from bit_exact_xor_amd import dcr
from tests import step_ref as R

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
E = 2.0 ** -24
SIZES = [0, 1, 3, 31, 32, 33, 64, 255, 1000, 4095, 4096, 4097, 20001]


def up(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


def formula(p, g, m, v, t, lr, b1, b2, eps, wd, gs):
    g = g * gs
    m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    den = np.sqrt(v / (1 - b2 ** t)) + eps
    return p * (1 - lr * wd) - lr / (1 - b1 ** t) * m / den, m, v, den


def tolerances(p, g, m, v, t, lr, b1, b2, eps, wd, gs):
    """m: both products' factors and themselves are rounded (4 roundings); v: a square more; p: the decayed weight's two,
    the update's from m's error and about 8 of its own."""
    g = g * gs
    tm = 4 * E * (np.abs(b1 * m) + np.abs((1 - b1) * g))
    tv = 7 * E * (b2 * v + (1 - b2) * g * g)
    p1, m1, v1, den = formula(p, g / gs, m, v, t, lr, b1, b2, eps, wd, gs)
    rate = lr / (1 - b1 ** t)
    return 3 * E * np.abs(p) + rate / den * (tm + 12 * E * np.abs(m1)) + 2.0 ** -140, tm + 2.0 ** -149, tv + 2.0 ** -140


HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, grad_scale=0.37)


def tensors_of(sizes, pt, gt, bits, rng, copy=False, **kw):
    params = [up(rng.standard_normal(n).astype(np.float32)).to(TYPES[pt]) for n in sizes]
    grads = [up((rng.standard_normal(n) * 10.0 ** rng.integers(-6, 2, n)).astype(np.float32)).to(TYPES[gt]) for n in sizes]
    for g in grads:
        g[::7] = 0
    copies = [torch.full((n,), 7.0, dtype=torch.bfloat16, device="cuda") for n in sizes] if copy else None
    return dcr.AdamWTensors(params, grads, bits=bits, copies=copies, **kw)


@pytest.mark.parametrize("pt,gt", [("fp32", "fp32"), ("fp32", "bf16"), ("bf16", "bf16"), ("bf16", "fp32")])
def test_wide_states(pt, gt):
    """Three steps, each from the state that the one before left; tensors of all sizes in one call."""
    rng = np.random.default_rng(1)
    decay = [i % 3 != 1 for i in range(len(SIZES))]
    T = tensors_of(SIZES, pt, gt, 32, rng, copy=pt == "fp32", decay=decay)
    for t in (1, 2, 50):
        before = [[f64(x) for x in row] for row in zip(T.params, T.grads, T.m, T.v)]
        dcr.dcr_adamw_step(T, t, **HYPER)
        for i, (p, g, m, v) in enumerate(before):
            h = [HYPER["lr"], 0.9, 0.95, 1e-8, 0.1 if decay[i] else 0.0, 0.37]
            want = formula(p, g, m, v, t, *h)
            tp, tm, tv = tolerances(p, g, m, v, t, *h)
            assert (np.abs(f64(T.params[i]) - want[0]) <= tp + HALF[pt] * (np.abs(want[0]) + tp)).all()
            assert (np.abs(f64(T.m[i]) - want[1]) <= tm).all() and (np.abs(f64(T.v[i]) - want[2]) <= tv).all()
            if pt == "fp32":
                assert torch.equal(T.copies[i], T.params[i].bfloat16())


@pytest.mark.parametrize("pt,gt", [("fp32", "bf16"), ("bf16", "fp32")])
@pytest.mark.parametrize("seed", [0, 77])
def test_narrow_states(pt, gt, seed):
    """Codes and scales in 8 bits: with betas that are sums of few powers of two, and gradients and moments of few bits,
    every product is exact in 32 bits, so a moment is the exact one rounded once and its codes are the reference's; the
    parameters take the moments before they are rounded."""
    rng = np.random.default_rng(2)
    T = tensors_of(SIZES, pt, gt, 8, rng)
    h = dict(lr=1e-2, beta1=0.5, beta2=0.75, eps=1e-6, weight_decay=0.0, grad_scale=2.0)
    for i, n in enumerate(SIZES):
        # gradients: 1 or 3 times a power of two; moments: few codes under any scale
        T.grads[i].copy_(up((rng.choice([0.0, 1.0, -1.0, 3.0], n) * 2.0 ** rng.integers(-9, 9, n)).astype(np.float32)))
        T.m[i].copy_(up(rng.choice([0.0, 1.0, -1.5, 2.0, 448.0, 2.0 ** -9], n).astype(np.float32)).to(torch.float8_e4m3fn))
        T.v[i].copy_(up(rng.choice([0.0, 1.0, 2.0, 256.0], n).astype(np.float32)).to(torch.float8_e4m3fn))
        T.m_scales[i].copy_(up(rng.integers(120, 134, -(-n // 32)).astype(np.uint8)))
        T.v_scales[i].copy_(up(rng.integers(120, 134, -(-n // 32)).astype(np.uint8)))
    at = 0
    first = []
    for n in SIZES:
        first.append(at)
        at += -(-n // 32) * 32
    before = [(f64(p), f64(g), R.from8(m.view(torch.uint8).cpu().numpy(), ms.cpu().numpy()),
               R.from8(v.view(torch.uint8).cpu().numpy(), vs.cpu().numpy()) ** 2)
              for p, g, m, v, ms, vs in zip(T.params, T.grads, T.m, T.v, T.m_scales, T.v_scales)]
    dcr.dcr_adamw_step(T, 9, dither=seed, **h)
    for i, (p, g, m, v) in enumerate(before):
        want = formula(p, g, m, v, 9, *h.values())
        tp, _tm, _tv = tolerances(p, g, m, v, 9, *h.values())
        assert (np.abs(f64(T.params[i]) - want[0]) <= tp + HALF[pt] * (np.abs(want[0]) + tp)).all()
        m32 = want[1].astype(np.float32).astype(np.float64)
        u = np.sqrt(want[2].astype(np.float32)).astype(np.float64)        # (correctly rounded on both sides)
        rm, rv = R.dither(np.arange(SIZES[i], dtype=np.uint64) + np.uint64(first[i]), seed, 9) if seed else (0.5, 0.5)
        for name, x, r, keep in (("m", m32, rm, False), ("v", u, rv, True)):
            codes, byte = R.to8(x, r, keep)
            got = getattr(T, name)[i].view(torch.uint8).cpu().numpy()
            assert np.array_equal(getattr(T, name + "_scales")[i].cpu().numpy(), byte), (SIZES[i], name)
            assert np.array_equal(got, codes), (SIZES[i], name, np.nonzero(got != codes)[0][:5])


def test_narrow_states_follow():
    """With the dither the held moments follow small changes: over many steps with one gradient the second moment's root
    comes near |g| although a step changes it by less than half a code (a standard deviation of the mean of 4096
    elements' codes, each within an eighth: 2^-3 / 64 / sqrt(3) of the value, five of them and the moment's own
    1 - 0.99^400 = 0.982)."""
    n = 4096
    T = dcr.AdamWTensors([torch.zeros(n, device="cuda")], [torch.full((n,), 0.37, device="cuda")], bits=8)
    for t in range(1, 401):
        dcr.dcr_adamw_step(T, t, lr=0.0, beta1=0.99, beta2=0.99, dither=5)
    for codes, scales, want in ((T.m[0], T.m_scales[0], 0.37 * (1 - .99 ** 400)), (T.v[0], T.v_scales[0], 0.37 * (1 - .99 ** 400) ** .5)):
        held = R.from8(codes.view(torch.uint8).cpu().numpy(), scales.cpu().numpy())
        assert abs(held.mean() / want - 1) < 0.03, held.mean() / want


@pytest.mark.parametrize("bits", [8, 32])
def test_extremes(bits):
    """Zero, tiny and huge gradients, infinities and NaN: only the element (8 bits: its block's states) is touched by them,
    nothing else becomes other than finite, and a second moment that is not zero stays so."""
    n = 320
    g = torch.zeros(n, device="cuda")
    g[0], g[33], g[70], g[100], g[130], g[200] = 1e-30, 1e18, float("nan"), float("inf"), -3e38, 1e-3
    T = dcr.AdamWTensors([torch.ones(n, device="cuda")], [g], bits=bits)
    for t in (1, 2):
        dcr.dcr_adamw_step(T, t, lr=1e-3)
    p = T.params[0]
    bad = ~torch.isfinite(p)
    allowed = torch.zeros(n, dtype=torch.bool, device="cuda")
    for i in (70, 100, 130):                    # (the square of 3e38 is infinite)
        block = slice(i, i + 1) if bits == 32 else slice(i // 32 * 32, i // 32 * 32 + 32)
        allowed[block] = True
    assert not (bad & ~allowed).any() and bad[70]
    assert (p[1:32] == 1).all() and p[33] < 1 and p[200] < 1
    if bits == 8:
        assert T.m_scales[0][70 // 32] == 255 and T.v_scales[0][100 // 32] == 255 and T.v_scales[0][130 // 32] == 255
        v = T.v[0].view(torch.uint8)
        assert v[200] > 0 and v[33] > 0 and (v[1:32] == 0).all()
        codes = T.m[0].view(torch.uint8)
        assert (codes[64:96] == 0).all()


def test_smallest_second_moment_stays():
    """A second moment far below its block's largest keeps the smallest code, not zero."""
    g = torch.full((32,), 1e-8, device="cuda")
    g[3] = 1.0
    for seed in (0, 1, 2, 3):
        T = dcr.AdamWTensors([torch.zeros(32, device="cuda")], [g], bits=8)
        dcr.dcr_adamw_step(T, 1, dither=seed)
        assert (T.v[0].view(torch.uint8) >= 1).all()


@pytest.mark.parametrize("spread", [0, 14])
def test_dither_past_32_bits(spread):
    """Elements whose index passes 32 bits inside a workgroup's, from an odd one on; codes that are all above the smallest
    normal one (spread 0) and of all sizes.  Moments are exact in 32 bits but for a last rounding, as above."""
    rng = np.random.default_rng(spread)
    n, first = 2053, (1 << 32) - 713
    h = dict(lr=2.0 ** -6, beta1=0.75, beta2=0.875, eps=2.0 ** -20, weight_decay=0.0, grad_scale=1.0)
    g = rng.choice([1.0, -1.0, 3.0], n) * 2.0 ** rng.integers(-spread, 1, n)
    T = dcr.AdamWTensors([up(np.ones(n, np.float32))], [up(g.astype(np.float32))], bits=8, first=[first])
    T.m[0].copy_(up(rng.choice([1.0, -1.5, 2.0], n).astype(np.float32)).to(torch.float8_e4m3fn))
    T.v[0].copy_(up(rng.choice([1.0, 2.0, 3.0], n).astype(np.float32)).to(torch.float8_e4m3fn))
    T.m_scales[0].fill_(127 - spread), T.v_scales[0].fill_(127 - spread)
    m, v = (R.from8(x.view(torch.uint8).cpu().numpy(), y.cpu().numpy())
            for x, y in ((T.m[0], T.m_scales[0]), (T.v[0], T.v_scales[0])))
    dcr.dcr_adamw_step(T, 9, dither=5, **h)
    _p, m, v, _den = formula(np.ones(n), g, m, v * v, 9, *h.values())
    rm, rv = R.dither(np.arange(n, dtype=np.uint64) + np.uint64(first), 5, 9)
    for x, r, keep, codes, scales in ((m.astype(np.float32), rm, False, T.m[0], T.m_scales[0]),
                                      (np.sqrt(v.astype(np.float32)), rv, True, T.v[0], T.v_scales[0])):
        want, byte = R.to8(x.astype(np.float64), r, keep)
        assert np.array_equal(scales.cpu().numpy(), byte)
        assert np.array_equal(codes.view(torch.uint8).cpu().numpy(), want)


@pytest.mark.parametrize("bits", [8, 32])
def test_shards_are_rounded_as_the_whole(bits):
    """A tensor in three shards, with `first`, gives the bits of the whole tensor."""
    rng = np.random.default_rng(3)
    n = 3 * 1024 + 512
    p, g = rng.standard_normal(n).astype(np.float32), rng.standard_normal(n).astype(np.float32)
    base = (1 << 32) - 1024                        # the index passes 32 bits on the way
    whole = dcr.AdamWTensors([up(p)], [up(g)], bits=bits, first=[base])
    cuts = [0, 1024, 2080, n]
    parts = dcr.AdamWTensors([up(p[a:b]) for a, b in zip(cuts, cuts[1:])], [up(g[a:b]) for a, b in zip(cuts, cuts[1:])], bits=bits,
                             first=[base + a for a in cuts[:-1]])
    for t in (1, 2, 3):
        dcr.dcr_adamw_step(whole, t, dither=11)
        dcr.dcr_adamw_step(parts, t, dither=11)
    assert torch.equal(whole.params[0], torch.cat(parts.params))
    for a, b in ((whole.m, parts.m), (whole.v, parts.v)):
        assert torch.equal(a[0].view(torch.uint8), torch.cat([x.view(torch.uint8) for x in b]))


def test_live_arguments_and_graphs():
    """A captured step reads its number, rate and scale from device memory: replays give the bits of eager steps, with
    eager work in between."""
    rng = np.random.default_rng(4)
    for bits in (8, 32):
        mk = lambda: tensors_of([1000, 5000], "fp32", "bf16", bits, np.random.default_rng(4), copy=True)  # noqa: E731
        A, B = mk(), mk()
        live = torch.tensor([1.0, 1e-3, 0.5], dtype=torch.float64, device="cuda")
        s = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=s):
            dcr.dcr_adamw_step(A, 1, live=live, beta2=0.95, weight_decay=0.01, dither=3)
            live[0] += 1
        for t in range(1, 6):
            lr = 1e-3 / t
            live[1] = lr
            graph.replay()
            dcr.dcr_adamw_step(B, t, lr=lr, beta2=0.95, weight_decay=0.01, grad_scale=0.5, dither=3)
            for g, h in zip(A.grads, B.grads):
                new = up(rng.standard_normal(g.numel()).astype(np.float32)).bfloat16()
                torch.cuda.synchronize()
                for x, y in ((A, B),):
                    for a, b in zip(x.params + x.m + x.v + x.copies, y.params + y.m + y.v + y.copies):
                        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), (bits, t)
                g.copy_(new)
                h.copy_(new)


def test_streams_and_lifetime():
    """Steps on a stream of the caller's; a plan that goes away leaves its tensors."""
    rng = np.random.default_rng(5)
    T = tensors_of([3000], "fp32", "fp32", 32, rng)
    U = tensors_of([3000], "fp32", "fp32", 32, np.random.default_rng(5))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for t in (1, 2, 3):
        dcr.dcr_adamw_step(T, t, stream=s)
        dcr.dcr_adamw_step(U, t)
    torch.cuda.synchronize()
    assert torch.equal(T.params[0], U.params[0])
    p = T.params[0]
    del T
    assert torch.equal(p, U.params[0])


def test_refusals_of_tensors():
    z = lambda n, **k: torch.zeros(n, device="cuda", **k)  # noqa: E731
    a = z(64)
    for bad in (lambda: dcr.AdamWTensors([a], [z(63)]), lambda: dcr.AdamWTensors([a], [z(64, dtype=torch.float16)]),
                lambda: dcr.AdamWTensors([a], [torch.zeros(64)]), lambda: dcr.AdamWTensors([a], [z(64)], m=[z(64, dtype=torch.bfloat16)]),
                lambda: dcr.AdamWTensors([a], [z(64)], bits=8, m_scales=[z(3, dtype=torch.uint8)]),
                lambda: dcr.AdamWTensors([a], [z(64)], copies=[z(64)]), lambda: dcr.AdamWTensors([a], [z(64), z(64)]),
                lambda: dcr.AdamWTensors([z(128)[::2]], [z(64)]), lambda: dcr.AdamWTensors([a], [z(64)], decay=[])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: dcr.AdamWTensors([a], [a]), lambda: dcr.AdamWTensors([a, a], [z(64), z(64)]),
                lambda: dcr.AdamWTensors([z(65)[1:]], [z(64)]),
                lambda: dcr.AdamWTensors([z(64, dtype=torch.bfloat16)], [z(64)], copies=[z(64, dtype=torch.bfloat16)])):
        with pytest.raises(dcr.DcrError):
            bad()
    T = dcr.AdamWTensors([a], [z(64)])
    for kw in (dict(beta1=1.0), dict(beta2=-0.1), dict(eps=0.0), dict(eps=float("nan")), dict(lr=float("inf")),
               dict(weight_decay=float("nan")), dict(grad_scale=float("nan")), dict(beta1=float("nan"))):
        with pytest.raises(dcr.DcrError):
            dcr.dcr_adamw_step(T, 1, **kw)
    for kw in (dict(live=torch.zeros(3, dtype=torch.float64)), dict(live=z(3)), dict(live=z(2, dtype=torch.float64))):
        with pytest.raises(ValueError):
            dcr.dcr_adamw_step(T, 1, **kw)
    assert (a == 0).all()


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("pt,gt", [("fp32", "bf16"), ("bf16", "fp32")])
def test_many_elements(bits, pt, gt):
    """More elements than the caches hold, and more than take short steps: the bits that slices of them by themselves give."""
    n = 12_000_031 if bits == 32 else 24_000_031
    g = torch.Generator(device="cuda")
    g.manual_seed(bits)
    p = torch.randn(n, device="cuda", generator=g).to(TYPES[pt])
    grad = (torch.randn(n, device="cuda", generator=g) * 1e-2).to(TYPES[gt])
    copy = lambda m: [torch.empty(m, dtype=torch.bfloat16, device="cuda")] if pt == "fp32" else None  # noqa: E731
    cuts = [(0, 5000), (4096 * 1000, 4096 * 1000 + 70000), (n // 32 * 32 - 32000, n)]
    big = dcr.AdamWTensors([p.clone()], [grad], bits=bits, copies=copy(n))
    small = [dcr.AdamWTensors([p[a:b].clone()], [grad[a:b].clone()], bits=bits, copies=copy(b - a), first=[a]) for a, b in cuts]
    for t in (1, 2):
        dcr.dcr_adamw_step(big, t, dither=9, weight_decay=0.1)
        for s in small:
            dcr.dcr_adamw_step(s, t, dither=9, weight_decay=0.1)
    for s, (a, b) in zip(small, cuts):
        # (8 bits: a block that a slice cuts has its scale from other elements; whole blocks are compared)
        whole = bits == 32 or b == n
        b = b if whole else a + (b - a) // 32 * 32
        assert torch.equal(big.params[0][a:b], s.params[0][:b - a])
        if pt == "fp32":
            assert torch.equal(big.copies[0][a:b], s.copies[0][:b - a])
        for x, y in ((big.m, s.m), (big.v, s.v)):
            assert torch.equal(x[0][a:b].view(torch.uint8), y[0][:b - a].view(torch.uint8))
        if bits == 8:
            assert torch.equal(big.m_scales[0][a // 32: -(-b // 32)], s.m_scales[0][: -(-(b - a) // 32)])


def test_updates_are_divided():
    """Zero parameters, so that the result is the update itself, of numbers whose sums and products are exact (no averages,
    powers of two as rate, scale and eps, squares of up to twelve bits): it is the quotient rounded once."""
    rng = np.random.default_rng(71)
    n = 20000
    g = (rng.integers(1, 4096, n) * rng.choice([-1.0, 1.0], n)).astype(np.float32)
    T = dcr.AdamWTensors([torch.zeros(n, device="cuda")], [up(g)])
    dcr.dcr_adamw_step(T, 1, lr=2.0 ** -7, beta1=0.0, beta2=0.0, eps=3 * 2.0 ** -3)
    den = np.abs(g).astype(np.float64) + 0.375              # 12 bits and three behind the point
    want = -(2.0 ** -7 * g.astype(np.float64) / den)
    assert np.array_equal(f64(T.params[0]), want.astype(np.float32).astype(np.float64))


@pytest.mark.parametrize("bits", [8, 32])
def test_small_decays(bits):
    """A decay far below a step of 1 is taken off what it is of, not rounded as a factor: without gradients the parameter is
    p (1 - lr decay) within its own rounding and 2^-23 of the decay."""
    rng = np.random.default_rng(72)
    n = 20000
    p = rng.standard_normal(n).astype(np.float32)
    for lr, decay in ((1e-6, 0.1), (3e-7, 0.1), (1e-6, 0.3), (2e-5, 0.01)):
        T = dcr.AdamWTensors([up(p)], [torch.zeros(n, device="cuda")], bits=bits)
        dcr.dcr_adamw_step(T, 1, lr=lr, weight_decay=decay)
        want = p.astype(np.float64) * (1 - lr * decay)
        half = np.spacing(np.abs(want).astype(np.float32)).astype(np.float64) / 2
        assert (np.abs(f64(T.params[0]) - want) <= half * (1 + 2.0 ** -20) + np.abs(p) * lr * decay * 2.0 ** -22).all(), (lr, decay)


def test_live_arguments_of_several_graphs_stay():
    """What a captured step reads stays with the tensors, of every graph."""
    import gc
    import weakref
    T = tensors_of([1000], "fp32", "fp32", 32, np.random.default_rng(6))
    seen = []
    for _ in range(2):
        live = torch.tensor([1.0, 1e-3, 0.5], dtype=torch.float64, device="cuda")
        seen.append(weakref.ref(live))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            dcr.dcr_adamw_step(T, 1, live=live)
        del live
    gc.collect()
    assert all(r() is not None for r in seen)
    # an eager step's is the caller's: nothing grows from step to step
    live = torch.tensor([1.0, 1e-3, 0.5], dtype=torch.float64, device="cuda")
    r = weakref.ref(live)
    dcr.dcr_adamw_step(T, 1, live=live)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (s, s.cuda_stream, torch.cuda.default_stream(), 0):
        dcr.dcr_adamw_step(T, 1, live=live, stream=stream)
        torch.cuda.synchronize()
    del live
    gc.collect()
    assert r() is None
    del T
    gc.collect()
    assert all(r() is None for r in seen)


@pytest.mark.parametrize("bits", [8, 32])
def test_tensors_of_every_length_round_a_table_entry(bits):
    """Lengths on both sides of what an entry of the table and a workgroup have, in one plan, against each by itself."""
    sizes = [1, 511, 512, 513, 4095, 4096, 4097, 4608, 8192, 8193, 0, 12287, 12289, 36864, 40000]
    one = lambda n, s: up(np.random.default_rng(s).standard_normal(n).astype(np.float32))  # noqa: E731
    first = [1 << 20 | i << 16 for i in range(len(sizes))]
    decay = [i % 2 == 0 for i in range(len(sizes))]
    copies = lambda ns: [torch.full((n,), 7.0, dtype=torch.bfloat16, device="cuda") for n in ns]  # noqa: E731
    A = dcr.AdamWTensors([one(n, i) for i, n in enumerate(sizes)], [one(n, 100 + i) for i, n in enumerate(sizes)], bits=bits,
                         copies=copies(sizes), first=first, decay=decay)
    B = [dcr.AdamWTensors([one(n, i)], [one(n, 100 + i)], bits=bits, copies=copies([n]), first=[first[i]], decay=[decay[i]])
         for i, n in enumerate(sizes)]
    for t in (1, 2):
        for x in (A, *B):
            dcr.dcr_adamw_step(x, t, dither=9, weight_decay=0.1, lr=3e-3)
    for i, b in enumerate(B):
        for x, y in ((A.params, b.params), (A.m, b.m), (A.v, b.v), (A.copies, b.copies)):
            raw = torch.int32 if x[i].element_size() == 4 else torch.int16 if x[i].element_size() == 2 else torch.uint8
            assert torch.equal(x[i].view(raw), y[0].view(raw)), sizes[i]
        if bits == 8:
            assert torch.equal(A.m_scales[i], b.m_scales[0]) and torch.equal(A.v_scales[i], b.v_scales[0])


def test_live_arguments_are_those_passed():
    """The bias corrections and rates that the GPU makes of `live` are the host's, bit by bit, for many step numbers."""
    rng = np.random.default_rng(75)
    n = 256
    p, g = rng.standard_normal(n).astype(np.float32), rng.standard_normal(n).astype(np.float32)
    T = dcr.AdamWTensors([up(p)], [up(g)])
    steps = sorted({int(x) for x in np.exp(rng.uniform(0, np.log(1e6), 120))}) + [1 << 53]
    for beta1, beta2 in ((0.9, 0.999), (0.93, 0.9501), (0.5, 0.99999)):
        for t in steps:
            lr, scale = float(rng.uniform(1e-6, 1e-2)), float(rng.uniform(0.1, 2))
            got = []
            for live in (None, torch.tensor([t, lr, scale], dtype=torch.float64, device="cuda")):
                T.params[0].copy_(up(p))
                T.m[0].fill_(0.01), T.v[0].fill_(0.02)
                dcr.dcr_adamw_step(T, t, lr=lr, grad_scale=scale, beta1=beta1, beta2=beta2, weight_decay=0.1, live=live)
                got.append(T.params[0].clone())
            assert torch.equal(*got), (t, beta1)


def test_types_mixed_in_one_plan():
    """Parameters and gradients of both types, moments and lengths of all kinds in one plan, against each by itself."""
    sizes = [300, 9000, 4096, 70001, 0, 512, 13000, 1, 8192, 5000]
    pt = [TYPES["fp32" if i % 3 else "bf16"] for i in range(len(sizes))]
    gt = [TYPES["bf16" if i % 2 else "fp32"] for i in range(len(sizes))]
    one = lambda i, s: up(np.random.default_rng(s + i).standard_normal(sizes[i]).astype(np.float32))  # noqa: E731
    copy = lambda i: torch.full((sizes[i],), 7.0, dtype=torch.bfloat16, device="cuda") if pt[i] is torch.float32 else None  # noqa: E731
    first = [1 << 20 | i << 17 for i in range(len(sizes))]
    for bits in (8, 32):
        make = lambda at: dcr.AdamWTensors([one(i, 0).to(pt[i]) for i in at], [one(i, 50).to(gt[i]) for i in at], bits=bits,  # noqa: E731
                                           copies=[copy(i) for i in at], first=[first[i] for i in at])
        A, B = make(range(len(sizes))), [make([i]) for i in range(len(sizes))]
        for t in (1, 2):
            for x in (A, *B):
                dcr.dcr_adamw_step(x, t, dither=4, weight_decay=0.1)
        for i, b in enumerate(B):
            assert torch.equal(A.params[i], b.params[0]), (bits, sizes[i])
            assert A.copies[i] is None or torch.equal(A.copies[i], b.copies[0])
            raw = torch.int32 if bits == 32 else torch.uint8
            assert torch.equal(A.m[i].view(raw), b.m[0].view(raw)) and torch.equal(A.v[i].view(raw), b.v[0].view(raw))


@pytest.mark.parametrize("pt", ["fp32", "bf16"])
@pytest.mark.parametrize("bits", [8, 32])
def test_infinite_parameters_stay(bits, pt):
    """p (1 - lr decay) of an infinite parameter, as a mask that is held among others, is what it was; NaN stays NaN."""
    n = 1000
    p = torch.ones(n, device="cuda").to(TYPES[pt])
    p[3], p[500], p[700] = float("-inf"), float("inf"), float("nan")
    for decay in (0.0, 0.1):
        for flag in (True, False):
            g = torch.zeros(n, device="cuda")
            g[4] = 1.0
            T = dcr.AdamWTensors([p.clone()], [g], bits=bits, decay=[flag])
            for t in (1, 2):
                dcr.dcr_adamw_step(T, t, weight_decay=decay)
            q = T.params[0]
            assert q[3] == float("-inf") and q[500] == float("inf") and torch.isnan(q[700])
            assert torch.isfinite(q).sum() == n - 3
            if pt == "fp32":                 # (a step of 1e-3 is less than half of bf16's below 1, 2^-9)
                assert q[4] < q[5]
