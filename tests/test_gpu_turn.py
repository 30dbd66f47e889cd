"""The calls of a training turn together, round a refit: a step of the optimizer, the refit of its weights, the experts'
layer and the head's log probabilities with the refitted weights, and the gradient back through all of it."""
import numpy as np
import pytest
import torch

from bit_exact_xor_amd import dcr, pipeline
from tests import step_ref as R

pytestmark = pytest.mark.gpu
TOKENS, WIDTH, INNER, EXPERTS, K, VOCAB = 40, 128, 96, 12, 3, 517


def f64(t):
    return t.detach().double().cpu()


def relu2(h):
    return torch.relu(h) ** 2


def weights(rng):
    """fp32 masters of the experts' up and down matrices and the head."""
    shapes = [(EXPERTS * INNER, WIDTH), (EXPERTS * WIDTH, INNER), (VOCAB, WIDTH)]
    return shapes, [torch.from_numpy((rng.standard_normal(s) / np.sqrt(s[1])).astype(np.float32)).cuda() for s in shapes]


def held(refit):
    """The receiver's weights in 64 bits."""
    out = []
    for q in refit.held:
        y = torch.empty(q.rows, q.cols, device="cuda")
        dcr.dcr_fp4_dequantize(q, y)
        out.append(f64(y))
    return out


def rounded(x):
    """To bf16 and back, with the gradient of a copy."""
    return x + (x.detach().bfloat16().double() - x.detach())


def layer64(x, logits, up, down, ids):
    """The experts' layer in 64 bits at the choice `ids`, rows rounded to bf16 where the calls round them."""
    s = torch.softmax(logits, 1)
    w = s.gather(1, ids.clamp(min=0)) * (ids >= 0)
    w = w / w.sum(1, keepdim=True)
    y = []
    for t in range(len(x)):
        row = 0
        for j in range(K):
            e = int(ids[t, j])
            h = rounded(up[e * INNER:(e + 1) * INNER] @ x[t])
            z = rounded(down[e * WIDTH:(e + 1) * WIDTH] @ rounded(relu2(h)))
            row = row + w[t, j] * z
        y.append(row)
    return torch.stack(y)


@pytest.mark.parametrize("bits", [8, 32])
def test_turn(bits):
    """Every result within the roundings on its way: each bf16 rounding is 2^-8 of the value, sums of up to 128 such terms
    grow at most with their 2-norm, so a norm is 2^-8 off for each rounding in a row (products of operands rounded alike:
    h, its square twice that, z, y forward; about twice as many backward), 8 and 16 of them at most."""
    rng = np.random.default_rng(bits)
    shapes, masters = weights(rng)
    refit = pipeline.Fp4Refit(shapes, dcr.FP4_NV)
    grads = [torch.zeros_like(w) for w in masters]
    tensors = dcr.AdamWTensors(masters, grads, bits=bits)
    first = refit.refit(masters)
    old = held(refit)
    for g in grads:
        g.copy_(torch.from_numpy(rng.standard_normal(g.shape).astype(np.float32)).cuda())
    sent = refit.step(tensors, 1, lr=2e-2, dither=3)
    assert 0 < sent < first
    up, down, head = held(refit)
    assert not torch.equal(up, old[0])
    for w, q in zip(masters, refit.held):          # what the receiver holds is what the stepped masters quantise to
        mine = dcr.Fp4Tensor(q.rows, q.cols, dcr.FP4_NV, tensor_scale=q.tensor_scale)
        dcr.dcr_fp4_quantize(w, mine)
        assert torch.equal(mine.codes, q.codes) and torch.equal(mine.scales, q.scales)

    x = torch.from_numpy(rng.standard_normal((TOKENS, WIDTH)).astype(np.float32)).cuda().bfloat16()
    router = torch.from_numpy(rng.standard_normal((TOKENS, EXPERTS)).astype(np.float32)).cuda()
    targets = torch.from_numpy(rng.integers(-1, VOCAB, TOKENS)).cuda()
    y = refit.experts(0, 1, x, router, K, relu2)
    logp, entropy, ids, values = refit.logprobs(2, y, targets, scale=0.9, top=4)

    # the same turn with the calls themselves, kept for the gradient
    ws, step_ws = dcr.fp4_workspace(), dcr.step_workspace()
    new = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
    chosen, w = new(TOKENS, K, dtype=torch.int32), new(TOKENS, K, dtype=torch.float32)
    offsets, slots = new(EXPERTS + 1, dtype=torch.int32), new(TOKENS, K, dtype=torch.int32)
    dcr.dcr_experts_select(router, chosen, w, renormalize=True)
    dcr.dcr_experts_order(chosen, offsets, slots, step_ws)
    n = TOKENS * K
    sorted_x, h, z, y2 = new(n, WIDTH), new(n, INNER), new(n, WIDTH), new(TOKENS, WIDTH)
    dcr.dcr_experts_dispatch(x, slots, sorted_x)
    dcr.dcr_fp4_matmul(sorted_x, refit.held[0], h, offsets, ws)
    a = relu2(h)
    dcr.dcr_fp4_matmul(a, refit.held[1], z, offsets, ws)
    dcr.dcr_experts_combine(z, slots, w, y2)
    assert torch.equal(y, y2)
    logits = new(TOKENS, VOCAB, dtype=torch.float32)
    dcr.dcr_fp4_matmul(y2, refit.held[2], logits, None, ws)
    lse, ent, lp = (new(TOKENS, dtype=torch.float32) for _ in range(3))
    dcr.dcr_logprobs(logits, targets, lp, lse, ent, scale=0.9, workspace=step_ws)
    assert torch.equal(lp, logp) and torch.equal(ent, entropy)

    # forward against 64 bits
    X, L = f64(x).requires_grad_(), f64(router).requires_grad_()
    want_ids, _ = R.select(f64(router).numpy(), None, K, False)
    assert np.array_equal(chosen.cpu().numpy(), want_ids)
    Y = layer64(X, L, up, down, torch.from_numpy(want_ids).long())
    assert (f64(y) - Y.detach()).norm() < 8 * 2.0 ** -8 * Y.detach().norm()
    Z = torch.from_numpy(f64(y).numpy()).requires_grad_()
    lp64 = torch.log_softmax(Z @ head.T * 0.9, 1)
    t = targets.cpu()
    mine = torch.where(t < 0, 0.0, lp64.gather(1, t.clamp(min=0)[:, None])[:, 0])
    ent64 = -(lp64.exp() * lp64).sum(1)
    assert (f64(logp) - mine.detach()).abs().max() < 1e-4 and (f64(entropy) - ent64.detach()).abs().max() < 1e-4
    best = lp64.detach().gather(1, ids.cpu().long())
    assert (f64(values) - best).abs().max() < 1e-4
    assert (best - lp64.detach().topk(4, 1).values).abs().max() < 1e-4

    # backward: a policy's loss, sum of advantage * logp + 0.01 entropy
    adv = torch.from_numpy(rng.standard_normal(TOKENS).astype(np.float32)).cuda()
    dent = torch.full((TOKENS,), 0.01, device="cuda")
    dcr.dcr_logprobs_grad(logits, targets, lse, adv, logits, entropy=ent, dentropy=dent, scale=0.9)
    dy = new(TOKENS, WIDTH)
    dcr.dcr_fp4_matmul_grad(logits.bfloat16(), refit.held[2], dy, None, ws)
    dz, dw, da, dh, dsorted, dx = new(n, WIDTH), new(TOKENS, K, dtype=torch.float32), new(n, INNER), None, new(n, WIDTH), new(TOKENS, WIDTH)
    dcr.dcr_experts_combine_grad(dy, z, slots, w, dz, dw)
    dcr.dcr_fp4_matmul_grad(dz, refit.held[1], da, offsets, ws)
    dh = (da.float() * 2 * torch.relu(h.float())).bfloat16()
    dcr.dcr_fp4_matmul_grad(dh, refit.held[0], dsorted, offsets, ws)
    dcr.dcr_experts_combine(dsorted, slots, None, dx)
    drouter = new(TOKENS, EXPERTS, dtype=torch.float32)
    dcr.dcr_experts_select_grad(router, chosen, dw, drouter, renormalize=True)

    ((f64(adv) * mine).sum() + 0.01 * ent64.sum()).backward()
    assert (f64(dy) - Z.grad).norm() < 16 * 2.0 ** -8 * Z.grad.norm()
    Y.backward(f64(dy))
    assert (f64(dx) - X.grad).norm() < 16 * 2.0 ** -8 * X.grad.norm()
    assert (f64(drouter) - L.grad).norm() < 16 * 2.0 ** -8 * L.grad.norm()
    torch.cuda.synchronize()


def test_captured_and_on_streams():
    """The receiver's calls captured into graphs and on two streams at once give the bits of calls by themselves, replay
    after replay, with other inputs and eager work in between."""
    rng = np.random.default_rng(2)
    shapes, masters = weights(rng)
    refit = pipeline.Fp4Refit(shapes, dcr.FP4_NV)
    refit.refit(masters)
    x, router = torch.randn(TOKENS, WIDTH, device="cuda").bfloat16(), torch.randn(TOKENS, EXPERTS, device="cuda")
    targets = torch.randint(-1, VOCAB, (TOKENS,), device="cuda")

    def both(x, router, targets):
        y = refit.experts(0, 1, x, router, K, relu2, score=dcr.SCORE_SIGMOID, groups=4, top_groups=2)
        return [y, *refit.logprobs(2, y, targets, top=5)]
    both(x, router, targets)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = both(x, router, targets)
        graphs.append((g, out))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for r in range(4):
        x.copy_(torch.randn(TOKENS, WIDTH, device="cuda"))
        router.copy_(torch.randn(TOKENS, EXPERTS, device="cuda"))
        router[: r * 3] = -float("inf")                 # padding
        targets.copy_(torch.randint(-1, VOCAB, (TOKENS,), device="cuda"))
        want = [v.clone() for v in both(x, router, targets)]
        torch.cuda.synchronize()
        side = []
        for s, (g, _out) in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
                side.append(both(x, router, targets))
        torch.cuda.synchronize()
        for got in (graphs[0][1], graphs[1][1], *side):
            for a, b in zip(got, want):
                assert torch.equal(a, b)
        assert (want[0][: r * 3] == 0).all()


def test_graph_of_a_training_turn():
    """Choice, rows, log probabilities and their gradients captured with torch's own work, replayed with eager calls of
    the same functions in between."""
    rows, vocab, e, k, width = 300, 6000, 32, 4, 100
    x, router = torch.randn(rows, width, device="cuda"), torch.randn(rows, e, device="cuda")
    logits, t = torch.randn(rows, vocab, device="cuda"), torch.randint(0, vocab, (rows,), device="cuda")

    def turn(ws):
        new = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
        ids, w, off, slots = new(rows, k, dtype=torch.int32), new(rows, k), new(e + 1, dtype=torch.int32), new(rows, k, dtype=torch.int32)
        dcr.dcr_experts_select(router, ids, w)
        dcr.dcr_experts_order(ids, off, slots, ws)
        sent = torch.zeros(rows * k, width, device="cuda")
        dcr.dcr_experts_dispatch(x, slots, sent)
        y, dx, dw, dr = new(rows, width), torch.zeros_like(sent), new(rows, k), new(rows, e)
        dcr.dcr_experts_combine(sent, slots, w, y)
        dcr.dcr_experts_combine_grad(y, sent, slots, w, dx, dw)
        dcr.dcr_experts_select_grad(router, ids, dw, dr)
        lp, lse, ent, d = new(rows), new(rows), new(rows), new(rows, vocab)
        dcr.dcr_logprobs(logits, t, lp, lse, ent, workspace=ws)
        dcr.dcr_logprobs_grad(logits, t, lse, lp, d, entropy=ent, dentropy=lse)
        return [ids, w, off, slots, sent, y, dx, dw, dr, lp, lse, ent, d]
    ws = dcr.step_workspace()
    turn(ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = turn(dcr.step_workspace())
    for _ in range(4):
        for v in (x, router, logits):
            v.copy_(torch.randn_like(v))
        want = turn(ws)
        g.replay()
        again = turn(ws)
        torch.cuda.synchronize()
        for a, b, c in zip(got, want, again):
            assert torch.equal(a, b) and torch.equal(b, c)


def test_interrupted_refits_refuse():
    rng = np.random.default_rng(3)
    shapes, masters = weights(rng)
    refit = pipeline.Fp4Refit(shapes, dcr.FP4_NV)
    refit.refit(masters)
    x, router = torch.randn(4, WIDTH, device="cuda").bfloat16(), torch.randn(4, EXPERTS, device="cuda")
    refit.interrupted = True
    with pytest.raises(dcr.DcrError):
        refit.experts(0, 1, x, router, K, relu2)
    with pytest.raises(dcr.DcrError):
        refit.logprobs(2, x, torch.zeros(4, dtype=torch.int64, device="cuda"))
    refit.interrupted = False
    with pytest.raises(ValueError):
        refit.step(dcr.AdamWTensors(masters[:1], [torch.zeros_like(masters[0])]), 1)


def quantised(masters, refit):
    """Whether the receiver holds what the trainer's weights quantise to."""
    for w, q in zip(masters, refit.held):
        mine = dcr.Fp4Tensor(q.rows, q.cols, dcr.FP4_NV, tensor_scale=q.tensor_scale)
        dcr.dcr_fp4_quantize(w, mine)
        if not (torch.equal(mine.codes, q.codes) and torch.equal(mine.scales, q.scales)):
            return False
    return True


def test_step_on_another_stream():
    """The refit waits for a step that is put on a stream of the caller's, which is busy for a while before it."""
    rng = np.random.default_rng(5)
    shapes, masters = weights(rng)
    refit = pipeline.Fp4Refit(shapes, dcr.FP4_NV)
    refit.refit(masters)
    grads = [torch.from_numpy(rng.standard_normal(w.shape).astype(np.float32)).cuda() for w in masters]
    tensors = dcr.AdamWTensors(masters, grads)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for number, stream in ((1, s), (2, s.cuda_stream)):
        before = [w.clone() for w in masters]
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
        assert refit.step(tensors, number, lr=2e-2, stream=stream) > 0
        torch.cuda.synchronize()
        assert not any(torch.equal(a, b) for a, b in zip(before, masters))
        assert quantised(masters, refit)


def test_step_whose_refit_has_not_begun(monkeypatch):
    """An error before anything is sent: the step has been taken, nothing is interrupted, and refit() sends the weights."""
    rng = np.random.default_rng(6)
    shapes, masters = weights(rng)
    refit = pipeline.Fp4Refit(shapes, dcr.FP4_NV)
    refit.refit(masters)
    tensors = dcr.AdamWTensors(masters, [torch.from_numpy(rng.standard_normal(w.shape).astype(np.float32)).cuda() for w in masters])
    before = [w.clone() for w in masters]

    def fails(*args, **kw):
        raise MemoryError("as if there were none")
    with monkeypatch.context() as m:
        m.setattr(dcr, "dcr_fp4_quantize", fails)
        with pytest.raises(MemoryError):
            refit.step(tensors, 1, lr=2e-2)
    assert not refit.interrupted and refit.version == 1
    assert not any(torch.equal(a, b) for a, b in zip(before, masters))
    refit.recover()
    assert not quantised(masters, refit)
    assert refit.refit(masters) > 0
    assert quantised(masters, refit)
