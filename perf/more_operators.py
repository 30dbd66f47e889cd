"""The operators of one turn of training round a refit, as they are measured:
cases, inputs, a plain form of each in elementary torch operations, and the
calls of the library.

Kinds of a case:

  select         a router's logits to the experts of each token: softmax or
                 sigmoid scores, a bias that only the choice sees, groups of
                 experts, the k best, their weights; then the slot that each
                 (token, expert) pair takes in the rows sorted by expert, and
                 the experts' offsets
  select_grad    the gradient of the weights with respect to the logits
  rows           tokens copied to their slots, and the experts' results added
                 up again, each with its weight
  rows_grad      the gradient of both: of the results, the weights, the tokens
  logprobs       log probabilities of given tokens, with the entropy of their
                 distribution and the most probable tokens
  logprobs_grad  the gradient of log probabilities and entropy with respect to
                 the logits
  adamw          an AdamW step over many tensors, with states in 32 bits or in
                 8 (blocks of 32 e4m3 values under a power of two, the second
                 moment by its square root, rounded up or down by a dither)
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
LR, BETA1, BETA2, EPS, DECAY, GRAD_SCALE = 2e-5, 0.9, 0.95, 1e-8, 0.1, 0.5
SEED = 12345                       # of the dither
BLOCK = 32                         # elements under one scale of an 8-bit state
MOST_LOGITS = 4096 * 151936
MOST_ADAMW = 176_193_536
PAIRS_ROWS = 16384 * 8 * 2048


def listed():
    return [
        # a decode batch of 4 tokens through the router of a 128-expert layer: latency counts
        {"name": "select_decode", "kind": "select", "rows": 4, "experts": 128, "k": 8, "score": "softmax", "bias": False,
         "groups": 1, "top_groups": 1, "renormalize": True, "padding": 0, "dtype": "bf16"},
        # a long prompt, 256 experts in 8 groups of which 4 are taken, sigmoid scores and a bias for balance, some rows padding
        {"name": "select_groups", "kind": "select", "rows": 16384, "experts": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "top_groups": 4, "renormalize": True, "padding": 300, "dtype": "fp32"},
        # backward through the router of a training batch
        {"name": "select_grad", "kind": "select_grad", "rows": 16384, "experts": 128, "k": 8, "score": "softmax", "bias": False,
         "groups": 1, "top_groups": 1, "renormalize": True, "padding": 0, "dtype": "bf16"},
        # 24 tokens of a decode batch to their experts and back
        {"name": "rows_decode", "kind": "rows", "rows": 24, "width": 2048, "k": 8, "experts": 128, "padding": 0, "dtype": "bf16"},
        # a training batch of 16384 tokens, 8 of 128 experts each
        {"name": "rows_batch", "kind": "rows", "rows": 16384, "width": 2048, "k": 8, "experts": 128, "padding": 500, "dtype": "bf16"},
        # its backward
        {"name": "rows_batch_grad", "kind": "rows_grad", "rows": 16384, "width": 2048, "k": 8, "experts": 128, "padding": 500,
         "dtype": "bf16"},
        # sampled tokens of a decode batch with 20 alternatives each
        {"name": "logprobs_decode", "kind": "logprobs", "rows": 8, "vocab": 151936, "top": 20, "scale": 1.25, "masked": 267,
         "gap": 0, "dtype": "bf16"},
        # the answers of a training batch, log probabilities and entropy
        {"name": "logprobs_batch", "kind": "logprobs", "rows": 4096, "vocab": 151936, "top": 0, "scale": 1.0, "masked": 0,
         "gap": 0, "dtype": "bf16"},
        # its backward
        {"name": "logprobs_batch_grad", "kind": "logprobs_grad", "rows": 4096, "vocab": 151936, "top": 0, "scale": 1.0,
         "masked": 0, "gap": 0, "dtype": "bf16"},
        # vectors and small matrices of a small model: latency counts
        {"name": "adamw_small", "kind": "adamw", "count": 4, "rows": 640, "less": 100, "cols": 256, "norms": 5, "bits": 32,
         "param": "fp32", "grad": "fp32"},
        # a TP=4 share of some layers, fp32 masters with the bf16 weights that a refit compares
        {"name": "adamw_layers", "kind": "adamw", "count": 12, "rows": 3584, "less": 0, "cols": 4096, "norms": 8, "bits": 32,
         "param": "fp32", "grad": "bf16"},
        # the matrices of 16 experts in two layers, states in 8 bits
        {"name": "adamw_experts_8bit", "kind": "adamw", "count": 96, "rows": 768, "less": 0, "cols": 2048, "norms": 4, "bits": 8,
         "param": "fp32", "grad": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["select", "select_grad", "rows", "rows_grad", "logprobs", "logprobs_grad", "adamw"])
    dtype = rng.choice(["bf16", "fp32"])
    if kind in ("select", "select_grad"):
        groups = rng.choice([1, 1, 2, 4, 8]) if kind == "select" else 1
        each = _log(rng, 4, 512 // groups)
        k = _log(rng, 1, min(16, each))
        rows = min(_log(rng, 1, 32768), 16384 * 256 // (groups * each))
        top = rng.randint(1, groups)
        return {"kind": kind, "rows": rows, "experts": groups * each, "k": k, "score": rng.choice(["softmax", "sigmoid"]),
                "bias": kind == "select" and rng.random() < 0.5, "groups": groups, "top_groups": top,
                "renormalize": rng.random() < 0.6, "padding": rng.choice([0, rows // 9]), "dtype": dtype}
    if kind in ("rows", "rows_grad"):
        width = _log(rng, 16, 8192)
        if rng.random() < 0.6:
            width = max(16, width // 16 * 16)
        k = _log(rng, 1, 12)
        rows = min(_log(rng, 1, 32768), PAIRS_ROWS // 2 // (width * k))
        return {"kind": kind, "rows": rows, "width": width, "k": k, "experts": max(k, _log(rng, 4, 256)),
                "padding": rng.choice([0, rows // 9]), "dtype": dtype}
    if kind in ("logprobs", "logprobs_grad"):
        vocab = _log(rng, 64, 262144)
        if rng.random() < 0.6:
            vocab = vocab // 16 * 16
        top = rng.choice([0, 1, 5, 20, 32]) if kind == "logprobs" else 0
        rows = min(_log(rng, 1, 16384), MOST_LOGITS // (8 if top else 2) // vocab)
        return {"kind": kind, "rows": rows, "vocab": vocab, "top": top, "scale": rng.choice([1.0, 1.0, 0.5, 1.4]),
                "masked": rng.choice([0, vocab // 50]), "gap": rng.choice([0, 0, 8, 3]), "dtype": dtype}
    count, cols = _log(rng, 1, 48), _log(rng, 8, 8192)
    rows = min(_log(rng, 1, 8192), MOST_ADAMW // 2 // (count * cols))
    return {"kind": "adamw", "count": count, "rows": rows, "less": rng.choice([0, 1, rows // (2 * count)]), "cols": cols,
            "norms": rng.randint(0, 6), "bits": rng.choice([32, 8]), "param": rng.choice(["fp32", "fp32", "bf16"]),
            "grad": dtype}


def work(case):
    kind = case["kind"]
    if kind == "adamw":
        n = sum(_numels(case))
        p, g = (4 if case[t] == "fp32" else 2 for t in ("param", "grad"))
        state = 8 if case["bits"] == 32 else 2 + 2 / BLOCK
        return {"bytes": n * (2 * p + g + 2 * state + (2 if p == 4 else 0)), "flops": 16.0 * n}
    size, rows = (2 if case["dtype"] == "bf16" else 4), case["rows"]
    if kind.startswith("select"):
        e, k = case["experts"], case["k"]
        if kind == "select":
            return {"bytes": rows * (e * size + 12 * k), "flops": 8.0 * rows * e}
        return {"bytes": rows * (2 * e * size + 8 * k), "flops": 8.0 * rows * e}
    if kind.startswith("rows"):
        width, k = case["width"], case["k"]
        pairs = (rows - case["padding"]) * k
        if kind == "rows":       # x once, k copies; k results, y once
            return {"bytes": size * width * (2 * rows + 2 * pairs) + 12 * rows * k, "flops": 2.0 * pairs * width}
        # dy once, k results, k gradients of them; k gradients of copies, dx once
        return {"bytes": size * width * (2 * rows + 3 * pairs) + 16 * rows * k, "flops": 4.0 * pairs * width}
    n = rows * case["vocab"]
    if kind == "logprobs":
        return {"bytes": n * size + rows * (16 + 8 * case["top"]), "flops": 6.0 * n}
    return {"bytes": 2 * n * size + rows * 20, "flops": 6.0 * n}


# ------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _matrix(rows, cols, gap, dtype):
    """An empty [rows, cols] whose rows lie `gap` elements further apart than they are long."""
    return torch.empty(rows, cols + gap, dtype=dtype, device="cuda")[:, :cols]


def prepare(case, seed):
    return _with_handles(_inputs(case, seed))


def _inputs(case, seed):
    g = _generator(seed)
    s = {"case": dict(case)}
    make = {"adamw": _adamw_inputs, "select": _select_inputs, "rows": _rows_inputs, "logprobs": _logprobs_inputs}
    make[case["kind"].replace("_grad", "")](s, case, g)
    return s


def _select_inputs(s, c, g):
    """Logits of a router: experts of different popularity, some experts shut (-inf), the last rows padding (all shut)."""
    rows, e, k = c["rows"], c["experts"], c["k"]
    logits = torch.randn(rows, e, device="cuda", generator=g) * 1.5 + torch.randn(e, device="cuda", generator=g)
    if e >= 8 * k and c["groups"] == 1:
        logits[:, torch.rand(e, device="cuda", generator=g) < 0.02] = -math.inf
    if c["padding"]:
        logits[rows - c["padding"]:] = -math.inf
    s["logits"] = logits.to(TYPES[c["dtype"]])
    s["bias"] = 0.1 * torch.randn(e, device="cuda", generator=g) if c["bias"] else None
    if c["kind"] == "select_grad":
        s["ids"] = _choice(s["logits"].double(), None, c)
        s["dweights"] = torch.randn(rows, k, device="cuda", generator=g)


def _rows_inputs(s, c, g):
    """Tokens, the slots of their pairs in rows sorted by expert, weights, results and gradients."""
    rows, width, k, e = c["rows"], c["width"], c["k"], c["experts"]
    dtype = TYPES[c["dtype"]]
    popular = torch.randn(rows, e, device="cuda", generator=g) + torch.randn(e, device="cuda", generator=g)
    ids = popular.topk(k, dim=1).indices
    ids[rows - c["padding"]:] = -1
    s["slots"] = _slots(ids, e)[1]
    weights = torch.rand(rows, k, device="cuda", generator=g) + 0.05
    s["weights"] = weights / weights.sum(1, keepdim=True)

    def some(m):
        return torch.randn(m, width, device="cuda", generator=g).to(dtype)
    s["results"] = some(rows * k)
    s["sent"] = torch.zeros(rows * k, width, dtype=dtype, device="cuda")   # rows of no pair stay as they are
    if c["kind"] == "rows":
        s["x"] = some(rows)
    else:
        s["dy"], s["dsent"] = some(rows), some(rows * k)


def _logprobs_inputs(s, c, g):
    """Logits of a language model, peaked in most rows, the end of the vocabulary masked; targets likely and not, some
    positions without one (-1)."""
    rows, v = c["rows"], c["vocab"]
    logits = _matrix(rows, v, c["gap"], TYPES[c["dtype"]])
    sharp = 1.0 + 2.0 * torch.rand(rows, 1, device="cuda", generator=g)
    for part, sh in zip(logits.split(512), sharp.split(512)):
        part.copy_(torch.randn(part.shape, device="cuda", generator=g) * sh)
    live = v - c["masked"]
    peak = torch.randint(0, live, (rows,), device="cuda", generator=g)
    at = torch.arange(rows, device="cuda")
    logits[at, peak] = (8 + 6 * torch.rand(rows, device="cuda", generator=g)).to(logits.dtype)
    logits[:, live:] = -math.inf
    other = torch.randint(0, live, (rows,), device="cuda", generator=g)
    u = torch.rand(rows, device="cuda", generator=g)
    s["targets"] = torch.where(u < 0.6, peak, torch.where(u < 0.95, other, -1))
    s["logits"] = logits
    if c["kind"] == "logprobs_grad":
        s["dlogp"] = torch.randn(rows, device="cuda", generator=g)
        s["dentropy"] = 0.01 * torch.randn(rows, device="cuda", generator=g)
        lse, ent = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        for a, b, part in zip(lse.split(256), ent.split(256), logits.split(256)):
            x = part.double() * c["scale"]
            top = x.amax(1)
            ex = torch.exp(x - top[:, None])
            z = ex.sum(1)
            a.copy_(top + z.log())
            b.copy_(z.log() - torch.where(ex > 0, ex * (x - top[:, None]), 0.0).sum(1) / z)
        s["lse"], s["entropy"] = lse, ent


def _numels(c):
    """Elements of each tensor: the matrices, then the vectors (which do not decay)."""
    return [max(1, c["rows"] - i * c["less"]) * c["cols"] for i in range(c["count"])] + [c["cols"]] * c["norms"]


def _starts(c):
    """First element of each tensor in the flat buffers, which hold them on borders of 256, and the end of all."""
    at = [0]
    for n in _numels(c):
        at.append(at[-1] + -(-n // 256) * 256)
    return at


def _adamw_inputs(s, c, g):
    """Weights, gradients (a tenth of the rows without any, as of experts and words not met) and states in flat buffers."""
    at, sizes = _starts(c), _numels(c)
    total = at[-1]
    live = torch.zeros(total, device="cuda")
    for a, n in zip(at, sizes):
        live[a:a + n] = 1.0
    met = (torch.rand(total // 256, 1, device="cuda", generator=g) > 0.1).float()
    size = torch.exp(torch.randn(total // 256, 1, device="cuda", generator=g)) * 1e-3

    def normal():
        return torch.randn(total, device="cuda", generator=g).mul_(live).view(-1, 256)
    s["param"] = normal().mul_(0.02).view(-1).to(TYPES[c["param"]])
    s["grad"] = normal().mul_(size * met).view(-1).to(TYPES[c["grad"]])
    m = normal().mul_(size * 0.3).view(-1)
    u = normal().abs_().add_(0.1).mul_(size).view(-1).mul_(live)
    if c["bits"] == 32:
        s["m"], s["v"] = m, u * u
    else:
        s["m"], s["m_scales"] = _to8(m, 0.5, False)
        s["v"], s["v_scales"] = _to8(u, 0.5, True)
    s["copy"] = s["param"].to(torch.bfloat16) if c["param"] == "fp32" else None
    s["step"] = 10


def _with_handles(s):
    """The results' buffers, workspaces and tables that a program keeps from call to call."""
    if own:
        from bit_exact_xor_amd import dcr
        c = s["case"]
        if c["kind"] in ("select", "logprobs"):
            s["workspace"] = dcr.step_workspace()
        if c["kind"] == "select_grad":
            s["ids"] = s["ids"].int()            # as dcr_experts_select gives them
        if c["kind"] == "adamw":
            at, sizes = _starts(c), _numels(c)

            def views(t, per=1):
                return None if t is None else [t[a // per: a // per + -(-n // per)] for a, n in zip(at, sizes)]
            s["tensors"] = dcr.AdamWTensors(
                views(s["param"]), views(s["grad"]), bits=c["bits"], copies=views(s["copy"]), m=views(s["m"]), v=views(s["v"]),
                m_scales=views(s.get("m_scales"), BLOCK), v_scales=views(s.get("v_scales"), BLOCK),
                decay=[i < c["count"] for i in range(len(sizes))], first=at[:-1])
    return s


def run(state):
    return (_run_own if own else _run_plain)(state, state["case"])


# ------------------------------------------------------------ plain forms

def _run_plain(s, c):
    kind = c["kind"]
    if kind == "select":
        logits = s["logits"].double()            # next to a border of the choice 32 bits decide wrongly
        ids = _choice(logits, s["bias"], c)
        weights = _weights(_scores(logits, c), ids, c).float()
        offsets, slots = _slots(ids, c["experts"])
        return {"ids": ids.int(), "weights": weights, "offsets": offsets, "slots": slots}
    if kind == "select_grad":
        return _plain_select_grad(s, c)
    if kind == "rows":
        return {"sent": _plain_dispatch(s["x"], s["slots"], s["sent"]),
                "y": _plain_combine(s["results"], s["slots"], s["weights"])}
    if kind == "rows_grad":
        return _plain_rows_grad(s)
    if kind == "logprobs":
        return _plain_logprobs(s, c)
    if kind == "logprobs_grad":
        return _plain_logprobs_grad(s, c)
    return _plain_adamw(s, c)


def _scores(logits, c):
    """Softmax or sigmoid; a row that is shut everywhere has scores of zero."""
    if c["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-logits))
    top = logits.amax(1, keepdim=True)
    e = torch.exp(logits - torch.where(top == -math.inf, 0.0, top))
    z = e.sum(1, keepdim=True)
    return e / torch.where(z == 0, 1.0, z)


def _choice(logits, bias, c):
    """The k best experts of each row, the best first, the lowest of equals first; -1 where fewer than k are open."""
    rows, e = logits.shape
    shut = logits == -math.inf
    rank = logits if bias is None else torch.where(shut, -math.inf, _scores(logits, c) + bias.to(logits.dtype))
    groups = c["groups"]
    if c["top_groups"] < groups:
        value = torch.where(shut, -math.inf, _scores(logits, c) if bias is None else rank).view(rows, groups, e // groups)
        best = value.topk(min(2, e // groups), dim=2).values
        one = best[..., 0]
        total = torch.where(best == -math.inf, 0.0, best).sum(2)
        of_group = torch.where(one == -math.inf, -math.inf, total)
        order = torch.sort(of_group, dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        taken = torch.zeros(rows, groups, dtype=torch.bool, device=logits.device).scatter_(1, order, True)
        rank = torch.where(taken[:, :, None], rank.view(rows, groups, -1), -math.inf).view(rows, e)
    value, ids = torch.sort(rank, dim=1, descending=True, stable=True)
    return torch.where(value[:, :c["k"]] == -math.inf, -1, ids[:, :c["k"]])


def _weights(scores, ids, c):
    w = torch.where(ids < 0, 0.0, scores.gather(1, ids.clamp(min=0).long()))
    if c["renormalize"]:
        z = w.sum(1, keepdim=True)
        w = w / torch.where(z == 0, 1.0, z)
    return w


def _slots(ids, experts):
    """(offsets [experts + 1], slots like ids) of the pairs sorted by expert, those of one expert by token."""
    flat = torch.where(ids < 0, experts, ids).reshape(-1)
    order = torch.sort(flat, stable=True).indices
    slots = torch.empty(flat.shape, dtype=torch.int32, device=ids.device)
    slots[order] = torch.arange(flat.numel(), dtype=torch.int32, device=ids.device)
    count = torch.zeros(experts + 1, dtype=torch.int64, device=ids.device)
    count.scatter_add_(0, flat.long(), torch.ones_like(flat, dtype=torch.int64))
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = torch.cumsum(count[:experts], 0)
    return offsets, torch.where(flat == experts, -1, slots).view(ids.shape)


def _plain_select_grad(s, c):
    logits, ids, dw = s["logits"].float(), s["ids"].long(), s["dweights"]
    scores = _scores(logits, c)
    w = _weights(scores, ids, c)
    dw = torch.where(ids < 0, 0.0, dw)
    if c["renormalize"]:
        z = torch.where(ids < 0, 0.0, scores.gather(1, ids.clamp(min=0))).sum(1, keepdim=True)
        dw = (dw - (dw * w).sum(1, keepdim=True)) / torch.where(z == 0, 1.0, z)
        dw = torch.where(ids < 0, 0.0, dw)
    ds = torch.zeros_like(scores).scatter_add_(1, ids.clamp(min=0), dw)
    if c["score"] == "sigmoid":
        d = ds * scores * (1 - scores)
    else:
        d = scores * (ds - (ds * scores).sum(1, keepdim=True))
    return d.to(s["logits"].dtype)


def _plain_dispatch(x, slots, out):
    rows, k = slots.shape
    at = slots.reshape(-1).long()
    pairs = x[:, None, :].expand(rows, k, -1).reshape(rows * k, -1)
    taken = at >= 0
    out[at[taken]] = pairs[taken].to(out.dtype)
    return out


def _picked(rows, slots):
    """The row of each pair in fp32, zeros where it has none: [tokens, k, width]."""
    got = rows[slots.clamp(min=0).long()].float()
    return torch.where(slots[..., None] < 0, 0.0, got)


def _plain_combine(rows, slots, weights):
    got = _picked(rows, slots)
    if weights is not None:
        got = got * weights[..., None]
    return got.sum(1).to(rows.dtype)


def _plain_rows_grad(s):
    slots, dy = s["slots"], s["dy"].float()
    dweights = (_picked(s["results"], slots) * dy[:, None, :]).sum(2)
    at = slots.reshape(-1).long()
    taken = at >= 0
    each = (s["weights"][..., None] * dy[:, None, :]).reshape(at.numel(), -1)
    s["sent"][at[taken]] = each[taken].to(s["sent"].dtype)
    return {"dresults": s["sent"], "dweights": dweights, "dx": _plain_combine(s["dsent"], slots, None)}


def _plain_logprobs(s, c):
    logits, targets = s["logits"], s["targets"]
    x = logits.float() * c["scale"]
    top = x.amax(1, keepdim=True)
    x = x - top
    e = torch.exp(x)
    z = e.sum(1)
    log_z = torch.log(z)
    at = x.gather(1, targets.clamp(min=0)[:, None])[:, 0]
    out = {"logp": torch.where(targets < 0, 0.0, at - log_z), "lse": top[:, 0] + log_z,
           "entropy": log_z - torch.where(e > 0, e * x, 0.0).sum(1) / z}
    if c["top"]:
        bits = (logits.float() + 0.0).view(torch.int32).long()
        rank = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
        last = c["vocab"] - 1
        key = (rank << 20) + (last - torch.arange(c["vocab"], device=x.device))
        ids = last - (key.topk(c["top"], dim=1).values & ((1 << 20) - 1))
        out["top_ids"] = ids.int()
        out["top_values"] = x.gather(1, ids) - log_z[:, None]
    return out


def _plain_logprobs_grad(s, c):
    logits, targets = s["logits"], s["targets"]
    lp = logits.float() * c["scale"] - s["lse"][:, None]
    p = torch.exp(lp)
    dlogp = torch.where(targets < 0, 0.0, s["dlogp"])
    d = -p * (dlogp[:, None] + s["dentropy"][:, None] * (torch.where(p > 0, lp, 0.0) + s["entropy"][:, None]))
    d.scatter_add_(1, targets.clamp(min=0)[:, None], dlogp[:, None])
    return (d * c["scale"]).to(logits.dtype)


def _dither(total, step, device):
    """Two numbers from 0 to 65535 / 65536 for each element: its index, the step and the seed, mixed."""
    low = (1 << 32) - 1
    key = (SEED * 0x9E3779B1 + step * 0x6A09E667) & low
    x = (torch.arange(total, dtype=torch.int64, device=device) * 0x9E3779B1 + key) & low
    x = ((x ^ (x >> 16)) * 0x6A09E667) & low
    x = ((x ^ (x >> 15)) * 0x3C6EF373) & low
    x = x ^ (x >> 16)
    return (x & 0xFFFF).float() / 65536, (x >> 16).float() / 65536


def _to8(x, r, keep):
    """(e4m3 codes, e8m0 bytes) of a flat buffer: x / 2^n with the largest of a block in (224, 448], rounded down where
    the rest of the division by the code's step is below 1 - r; with `keep` what is not zero does not become zero."""
    b = x.view(-1, BLOCK)
    top = b.abs().amax(1)
    exps = (top.view(torch.int32) >> 23) - 127 - 8 + ((top.view(torch.int32) & 0x7FFFFF) > 0x600000).int()
    byte = torch.where(top == 0, 0, (exps + 127).clamp(0, 254))
    y = (b.double() * torch.exp2(127.0 - byte.double())[:, None]).float()
    exponent = ((y.abs().view(torch.int32) >> 23) - 127).clamp(min=-6)
    step = torch.exp2((exponent - 3).double())
    r = r.view(-1, BLOCK) if isinstance(r, torch.Tensor) else r
    code = torch.floor(y.abs().double() / step + r) * step
    if keep:
        code = torch.where(y > 0, code.clamp(min=2.0 ** -9), code)
    code = torch.copysign(code.clamp(max=448.0), y.double()).float().to(torch.float8_e4m3fn)
    return code.view(-1), byte.to(torch.uint8)


def _from8(codes, scales):
    return (codes.float().view(-1, BLOCK) * torch.exp2(scales.float() - 127)[:, None]).view(-1)


def _plain_adamw(s, c):
    s["step"] += 1
    t = s["step"]
    split = _starts(c)[c["count"]]               # matrices in front, vectors behind
    p = s["param"].float()
    g = s["grad"].float() * GRAD_SCALE
    wide = c["bits"] == 32
    m = s["m"] if wide else _from8(s["m"], s["m_scales"])
    v = s["v"] if wide else _from8(s["v"], s["v_scales"]).square()
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g * g * (1 - BETA2)
    u = torch.sqrt(v)
    update = m / (u / math.sqrt(1 - BETA2 ** t) + EPS) * (LR / (1 - BETA1 ** t))
    p[:split] *= 1 - LR * DECAY
    s["param"].copy_(p - update)
    out = {"param": s["param"], "m": s["m"], "v": s["v"]}
    if wide:
        s["m"].copy_(m)
        s["v"].copy_(v)
    else:
        rm, rv = _dither(p.numel(), t, p.device)
        for name, x, r, keep in (("m", m, rm, False), ("v", u, rv, True)):
            code, byte = _to8(x, r, keep)
            s[name].copy_(code)
            s[name + "_scales"].copy_(byte)
            out[name + "_scales"] = s[name + "_scales"].view(torch.float8_e8m0fnu)
    if s["copy"] is not None:
        out["copy"] = s["copy"].copy_(s["param"])
    return out


# ------------------------------------------------------ the library's calls

def _run_own(s, c):
    from bit_exact_xor_amd import dcr
    kind = c["kind"]
    if kind == "adamw":
        s["step"] += 1
        dcr.dcr_adamw_step(s["tensors"], s["step"], lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS, weight_decay=DECAY,
                           grad_scale=GRAD_SCALE, dither=SEED if c["bits"] == 8 else 0)
        out = {n: s[n] for n in ("param", "m", "v")}
        if c["bits"] == 8:
            out.update({n: s[n].view(torch.float8_e8m0fnu) for n in ("m_scales", "v_scales")})
        return out if s["copy"] is None else {**out, "copy": s["copy"]}
    rows = c["rows"]

    def empty(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="cuda")
    if kind.startswith("select"):
        score = dcr.SCORE_SOFTMAX if c["score"] == "softmax" else dcr.SCORE_SIGMOID
        if kind == "select":
            ids, weights = empty(rows, c["k"], dtype=torch.int32), empty(rows, c["k"])
            offsets, slots = empty(c["experts"] + 1, dtype=torch.int32), empty(rows, c["k"], dtype=torch.int32)
            dcr.dcr_experts_select(s["logits"], ids, weights, bias=s["bias"], score=score, groups=c["groups"],
                                   top_groups=c["top_groups"], renormalize=c["renormalize"])
            dcr.dcr_experts_order(ids, offsets, slots, s["workspace"])
            return {"ids": ids, "weights": weights, "offsets": offsets, "slots": slots}
        d = torch.empty_like(s["logits"])
        dcr.dcr_experts_select_grad(s["logits"], s["ids"], s["dweights"], d, score=score, renormalize=c["renormalize"])
        return d
    if kind == "rows":
        y = torch.empty_like(s["x"])
        dcr.dcr_experts_dispatch(s["x"], s["slots"], s["sent"])
        dcr.dcr_experts_combine(s["results"], s["slots"], s["weights"], y)
        return {"sent": s["sent"], "y": y}
    if kind == "rows_grad":
        dw, dx = torch.empty_like(s["weights"]), torch.empty_like(s["dy"])
        dcr.dcr_experts_combine_grad(s["dy"], s["results"], s["slots"], s["weights"], s["sent"], dw)
        dcr.dcr_experts_combine(s["dsent"], s["slots"], None, dx)
        return {"dresults": s["sent"], "dweights": dw, "dx": dx}
    if kind == "logprobs":
        out = {n: empty(rows) for n in ("logp", "lse", "entropy")}
        if c["top"]:
            out["top_ids"], out["top_values"] = empty(rows, c["top"], dtype=torch.int32), empty(rows, c["top"])
        dcr.dcr_logprobs(s["logits"], s["targets"], scale=c["scale"], workspace=s["workspace"], **out)
        return out
    d = empty(rows, c["vocab"], dtype=s["logits"].dtype)
    dcr.dcr_logprobs_grad(s["logits"], s["targets"], s["lse"], s["dlogp"], d, entropy=s["entropy"], dentropy=s["dentropy"],
                          scale=c["scale"])
    return d


# ------------------------------------------------------ the definition, in 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    return {"select": _exact_select, "select_grad": _exact_select_grad, "rows": _exact_rows, "rows_grad": _exact_rows_grad,
            "logprobs": _exact_logprobs, "logprobs_grad": _exact_logprobs_grad, "adamw": _exact_adamw}[case["kind"]](s, case)


def _exact_scores(x, c):
    if c["score"] == "sigmoid":
        return torch.sigmoid(x)
    return torch.nan_to_num(torch.softmax(x, 1), nan=0.0)


def _exact_select(s, c):
    x = s["logits"].double()
    open_ = torch.isfinite(x)
    score = _exact_scores(x, c)
    rank = score + (0 if s["bias"] is None else s["bias"].double())
    rank = rank.masked_fill(~open_, -math.inf)
    rows, e, groups = c["rows"], c["experts"], c["groups"]
    if c["top_groups"] < groups:
        parts = rank.unflatten(1, (groups, e // groups)).sort(dim=2, descending=True).values[..., :2]
        sums = parts.masked_fill(parts == -math.inf, 0).sum(2).masked_fill(parts[..., 0] == -math.inf, -math.inf)
        out = sums.argsort(dim=1, descending=True, stable=True)[:, c["top_groups"]:]
        of = torch.arange(e, device=x.device) // (e // groups)
        rank = rank.masked_fill((of[None, :, None] == out[:, None, :]).any(2), -math.inf)
    order = rank.argsort(dim=1, descending=True, stable=True)[:, :c["k"]]
    some = rank.gather(1, order) > -math.inf
    w = score.gather(1, order) * some
    if c["renormalize"]:
        w = torch.nan_to_num(w / w.sum(1, keepdim=True), nan=0.0)
    return {"ids": None, "weights": w, "offsets": None, "slots": None}


def _exact_select_grad(s, c):
    x = s["logits"].double().requires_grad_()
    ids = s["ids"].long()
    padded = torch.isinf(x.detach()).all(1, keepdim=True)
    live = x.masked_fill(padded, 0.0)
    score = torch.sigmoid(live) if c["score"] == "sigmoid" else torch.softmax(live, 1)
    w = score.gather(1, ids.clamp(min=0)) * (ids >= 0)
    if c["renormalize"]:
        w = w / w.sum(1, keepdim=True).masked_fill(padded, 1.0)
    w.masked_fill(ids < 0, 0.0).backward(s["dweights"].double())
    return x.grad


def _tables(slots):
    """(slots, tokens) of the pairs that have a slot."""
    token = torch.arange(slots.shape[0], device=slots.device)[:, None].expand_as(slots)
    has = slots > -1
    return slots[has].long(), token[has], has


def _exact_sum(rows, slots, weights):
    at, token, has = _tables(slots)
    out = torch.zeros(slots.shape[0], rows.shape[1], dtype=torch.float64, device=rows.device)
    for part in range(0, at.numel(), 16384):
        i = slice(part, part + 16384)
        part_rows = rows[at[i]].double()
        out.index_add_(0, token[i], part_rows if weights is None else part_rows * weights[has][i, None].double())
    return out


def _exact_rows(s, c):
    at, token, _has = _tables(s["slots"])
    sent = torch.zeros(s["sent"].shape, dtype=torch.float64, device=at.device)
    sent[at] = s["x"].double()[token]
    return {"sent": sent, "y": _exact_sum(s["results"], s["slots"], s["weights"])}


def _exact_rows_grad(s, c):
    at, token, has = _tables(s["slots"])
    dres = torch.zeros(s["sent"].shape, dtype=torch.float64, device=at.device)
    dw = torch.zeros(s["weights"].shape, dtype=torch.float64, device=at.device)
    got = []
    for part in range(0, at.numel(), 16384):
        i = slice(part, part + 16384)
        dy = s["dy"][token[i]].double()
        dres[at[i]] = dy * s["weights"][has][i, None].double()
        got.append(torch.linalg.vecdot(dy, s["results"][at[i]].double()))
    if got:
        dw[has] = torch.cat(got)
    return {"dresults": dres, "dweights": dw, "dx": _exact_sum(s["dsent"], s["slots"], None)}


def _exact_logprobs(s, c):
    out = {"logp": [], "lse": [], "entropy": [], "top_values": []}
    for x, t in zip(s["logits"].split(256), s["targets"].split(256)):
        x = x.double().mul(c["scale"])
        z = torch.logsumexp(x, 1, keepdim=True)
        lp = x - z
        out["lse"].append(z[:, 0])
        out["logp"].append(lp.gather(1, t.clamp(min=0)[:, None])[:, 0].masked_fill(t < 0, 0.0))
        out["entropy"].append(-(lp.exp() * lp.masked_fill(lp == -math.inf, 0.0)).sum(1))
        if c["top"]:
            out["top_values"].append(lp.topk(c["top"], dim=1).values)
    got = {k: torch.cat(v) for k, v in out.items() if v}
    return {**got, "top_ids": None} if c["top"] else got


def _exact_logprobs_grad(s, c):
    d = torch.empty(c["rows"], c["vocab"], dtype=torch.float64, device="cuda")
    for part in range(0, c["rows"], 256):
        i = slice(part, part + 256)
        lp = s["logits"][i].double() * c["scale"] - s["lse"][i, None].double()
        p = lp.exp()
        t, up = s["targets"][i], s["dlogp"][i].double()
        hot = torch.zeros_like(p)
        hot[torch.arange(len(t), device=p.device), t.clamp(min=0)] = 1.0
        hot = (hot - p) * up.masked_fill(t < 0, 0.0)[:, None]
        soft = p * (lp.masked_fill(p == 0, 0.0) + s["entropy"][i, None].double())
        d[i] = (hot - s["dentropy"][i, None].double() * soft) * c["scale"]
    return d


def _exact_codes(x, r, keep):
    """(code values, scales) of the 8-bit states, from the grid of e4m3 values."""
    grid = torch.tensor([i * 2.0 ** -9 for i in range(8)] + [(8 + f) * 2.0 ** (e - 10) for e in range(1, 16) for f in range(8)][:-1],
                        dtype=torch.float64, device=x.device)
    b = x.view(-1, BLOCK)
    top = b.abs().max(1).values
    scale = torch.exp2(torch.ceil(torch.log2(top / 448)).clamp(-127, 127))
    scale = torch.where(top == 0, 2.0 ** -127, scale)
    y = (b / scale[:, None]).view(-1)
    mag = y.abs()
    low = (torch.searchsorted(grid, mag, right=True) - 1).clamp(max=len(grid) - 1)
    high = (low + 1).clamp(max=len(grid) - 1)
    gap = (grid[high] - grid[low]).clamp(min=2.0 ** -9)
    got = torch.where((mag - grid[low]) / gap + r.double() >= 1, grid[high], grid[low])
    if keep:
        got = torch.where((mag > 0) & (got == 0), grid[1], got)
    return torch.copysign(got, y), scale


def _exact_adamw(s, c):
    t = s["step"] + 1
    g = s["grad"].double() * GRAD_SCALE
    if c["bits"] == 32:
        m, v = s["m"].double(), s["v"].double()
    else:
        unit = {n: torch.exp2(s[n].double() - 127).repeat_interleave(BLOCK) for n in ("m_scales", "v_scales")}
        m, v = s["m"].double() * unit["m_scales"], (s["v"].double() * unit["v_scales"]) ** 2
    m, v = m.lerp(g, 1 - BETA1), v.lerp(g * g, 1 - BETA2)
    del g
    p = s["param"].double()
    split = _starts(c)[c["count"]]
    step = m / (1 - BETA1 ** t) / ((v / (1 - BETA2 ** t)).sqrt() + EPS)
    step[:split] += DECAY * p[:split]
    p -= LR * step
    del step
    out = {"param": p}
    if c["bits"] == 32:
        out.update(m=m, v=v)
    else:
        rm, rv = _dither(p.numel(), t, p.device)
        out["m"], out["m_scales"] = _exact_codes(m, rm, False)
        out["v"], out["v_scales"] = _exact_codes(v.sqrt(), rv, True)
    return out if s["copy"] is None else {**out, "copy": p}


if __name__ == "__main__":
    print(*listed(), *(draw(random.Random(i)) for i in range(6)), sep="\n")
