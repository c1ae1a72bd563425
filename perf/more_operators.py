"""Workloads of the operators at the two ends of a model, where its rows meet the
vocabulary: the embedding lookup with a scale (``Ctx.embed``) and its gradient
over sorted tokens (``Ctx.embed_grad``), and the cross entropy of the output
layer over the grammar's allowed tokens, taken in pieces of the vocabulary with
no logits kept (``Ctx.head_loss``), with its gradients by the hidden rows and by
the weight (``Ctx.head_grad``).

``own`` chooses what ``run`` computes: False, the operators' plain form in
elementary torch operations in 32 bits; True, the calls a user of the package
makes.  Token ids and targets are int32 on the device, -1 (CG_NO_TOKEN) where a
row has none; ``pad`` > 0 makes the matrices rows of wider buffers.
"""

from __future__ import annotations

import functools
import math

import torch

own = False

NO_TOKEN = -1          # CG_NO_TOKEN in an int32 tensor


def listed():
    return [
        # the log-probability of one token of a lone request, 32000-token vocabulary: latency
        dict(name="head_loss_1x32000x1024", op="head_loss", rows=1, V=32000, D=1024, dtype="bf16", pad=0, mask=True,
             temp=1.0),
        # scoring the throughput workload's batch: 256 rows of 128256 tokens under the grammar's masks
        dict(name="head_loss_256x128256x4096", op="head_loss", rows=256, V=128256, D=4096, dtype="bf16", pad=0,
             mask=True, temp=0.7),
        # an evaluation pass over a batch of positions, no grammar on them
        dict(name="head_loss_4096x151936x1024", op="head_loss", rows=4096, V=151936, D=1024, dtype="bf16", pad=0,
             mask=False, temp=1.0),
        # the backward pass alone, from the kept normaliser, over the rows of a small batch
        dict(name="head_grad_192x32000x2048", op="head_grad", rows=192, V=32000, D=2048, dtype="bf16", pad=0, mask=True,
             temp=1.0),
        # a training step of the output layer, loss and gradients, the largest: 4096 positions of 128256 tokens
        dict(name="head_train_4096x128256x2048", op="head_train", rows=4096, V=128256, D=2048, dtype="bf16", pad=0,
             mask=False, temp=1.0),
        # float rows and weight, an odd vocabulary and an odd width in wider buffers, masked
        dict(name="head_train_333x32003x509_f32", op="head_train", rows=333, V=32003, D=509, dtype="f32", pad=7,
             mask=True, temp=1.0),
        # the next inputs of a decode batch: one token a row
        dict(name="embed_256x128256x4096", op="embed", rows=256, V=128256, D=4096, dtype="bf16", pad=0, scale=1.0),
        # a long prompt's tokens
        dict(name="embed_32768x128256x4096", op="embed", rows=32768, V=128256, D=4096, dtype="bf16", pad=0,
             scale=64.0),
        # the gradient of a training batch's tokens
        dict(name="embed_grad_8192x128256x2048", op="embed_grad", rows=8192, V=128256, D=2048, dtype="bf16", pad=0,
             scale=1.0),
        # float gradients of an odd vocabulary and width; common tokens come hundreds of times
        dict(name="embed_grad_20000x4013x1001_f32", op="embed_grad", rows=20000, V=4013, D=1001, dtype="f32", pad=0,
             scale=0.5),
        # a step of a student whose table is both its embedding and its output layer, under the masks
        dict(name="tied_step_2048x32000x1024", op="tied", rows=2048, V=32000, D=1024, dtype="bf16", pad=0, mask=True,
             temp=1.0, scale=1.0),
    ]


def draw(rng):
    """One more case: vocabularies of 500 to 152000 tokens (mostly odd sizes), widths of 32 to 4096, 1 to 32768 rows."""
    between = lambda lo, hi: int(math.exp(rng.uniform(math.log(lo), math.log(hi))))  # noqa: E731
    op = rng.choice(["head_loss", "head_grad", "head_train", "tied", "embed", "embed_grad"])
    V, D = between(500, 152000), between(32, 4096)
    V = V if rng.random() < 0.7 else max(512, V // 64 * 64)
    D = D if rng.random() < 0.4 else max(32, D // 64 * 64)
    case = dict(op=op, V=V, D=D, dtype=rng.choice(["bf16", "bf16", "f32"]), pad=rng.choice([0, 0, 5, 64]))
    if op.startswith("embed"):
        case["rows"] = between(1, max(2, min(32768, 2 ** 27 // D)))
        case["scale"] = rng.choice([1.0, 0.5, float(D) ** 0.5])
        return case
    products = 1.0e12 if case["dtype"] == "bf16" else 1.0e11   # multiplications of one matrix product
    case["rows"] = between(1, max(2, min(4096, products / (V * D))))
    case["mask"] = rng.random() < 0.6
    case["temp"] = rng.choice([1.0, 1.0, 0.7, 1.5])
    if op == "tied":
        case["scale"] = rng.choice([1.0, 2.0])
    return case


# ---- inputs -----------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _matrix(case, rows, g, scale):
    """[rows, D] normal values in a buffer of D + pad columns."""
    D, ld = case["D"], case["D"] + case["pad"]
    buf = torch.randn((rows, ld), generator=g, device="cuda")
    buf *= scale
    return (buf.to(torch.bfloat16) if case["dtype"] == "bf16" else buf)[:, :D]


def _tokens(rows, V, g):
    """Ids as text has them: token t at a rate like t ** -0.75, the commonest a
    few percent of all; every sixteenth row is padding."""
    t = (V * torch.rand(rows, generator=g, device="cuda") ** 4).to(torch.int32).clamp_(max=V - 1)
    at = torch.arange(rows, device="cuda")
    return torch.where(at % 16 == 7, torch.full_like(t, NO_TOKEN), t)


def _targets(rows, V, g):
    t = torch.randint(0, V, (rows,), generator=g, device="cuda").to(torch.int32)
    at = torch.arange(rows, device="cuda")
    return torch.where(at % 16 == 9, torch.full_like(t, NO_TOKEN), t)


def _bitmask(rows, V, target, g):
    """Masks as grammar states give them: most rows inside a string (nearly all
    tokens allowed), some at punctuation (a few tokens), a forced token now and
    then, and a dead row.  The target is an allowed token except in a row of 31."""
    W = (V + 31) // 32
    r = torch.arange(rows, device="cuda")
    share = torch.full((rows,), 0.93, device="cuda")
    share[r % 4 == 1] = 0.002
    share[r % 8 == 6] = 0.3
    bits = torch.zeros((rows, W * 32), dtype=torch.bool, device="cuda")
    bits[:, :V] = torch.rand((rows, V), generator=g, device="cuda") < share[:, None]
    bits[r[r % 16 == 11]] = False                     # a forced token: the target alone
    there = target >= 0
    bits[r[there], target[there].long()] = True
    odd = r[there & (r % 31 == 17)]
    bits[odd, target[odd].long()] = False
    bits[r[r % 97 == 13]] = False
    w = bits.view(rows, W, 32).to(torch.int64) << torch.arange(32, device="cuda")
    w = w.sum(2)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32).contiguous()


@functools.lru_cache(maxsize=None)
def _ctx(V):
    """The context a program keeps: one small grammar and a vocabulary of V tokens."""
    import grammar_constrained_decoding_gb300 as cg
    grammar = cg.Grammar.compile('root ::= "a"', "gbnf")
    return cg.Ctx([grammar], cg.Vocab([i.to_bytes(3, "big") for i in range(V)]))


def prepare(case, seed):
    g = _gen(seed)
    rows, V, D, op = case["rows"], case["V"], case["D"], case["op"]
    s = {"case": case}
    if own:
        s["ctx"] = _ctx(V)
    new = lambda *shape: torch.empty(shape, dtype=s["w"].dtype if len(shape) == 2 else torch.float32, device="cuda")  # noqa: E731
    if op in ("embed", "embed_grad"):
        s["tok"] = _tokens(rows, V, g)
        s["w"] = _matrix(case, V if op == "embed" else rows, g, 1.0)     # the table, or the rows' gradients
        s["out"] = new(rows if op == "embed" else V, D)
        return s
    s["w"] = _matrix(case, V, g, D ** -0.5)
    s["target"] = _targets(rows, V, g)
    s["mask"] = _bitmask(rows, V, s["target"], g) if case["mask"] else None
    s["up"] = torch.rand(rows, generator=g, device="cuda") / rows
    s["loss"], s["lse"], s["dw"] = new(rows), new(rows), new(V, D)
    if op == "tied":
        # the last tokens' rows themselves are the hidden rows: a student of one table
        s["w"].mul_(3.0)
        s["tok"] = _tokens(rows, V, g)
        s["h"] = new(rows, D)
    else:
        # logits of deviation 2; the target's is raised by up to 14, as a trained model's are
        h = _matrix(case, rows, g, 2.0)
        up = 14.0 * torch.rand((rows, 1), generator=g, device="cuda")
        h += (up * s["w"][s["target"].clamp(min=0).long()].float()).to(h.dtype)
        s["h"] = h
    s["dh"] = new(rows, D)
    s["norm"] = torch.empty((rows, 2), dtype=torch.float32, device="cuda")
    if op == "head_grad":
        # what the forward pass left: the loss, and the normaliser as maximum and sum
        _plain_loss(s, _plain_logits(s, s["h"].float()))
    return s


# ---- the plain form ---------------------------------------------------------------

def _allowed(mask, V):
    at = torch.arange(V, device=mask.device)
    return ((mask[:, at >> 5] >> (at & 31).to(torch.int32)) & 1).bool()


def _plain_logits(s, h):
    x = h @ s["w"].float().T
    return x if s["mask"] is None else x.masked_fill_(~_allowed(s["mask"], x.shape[1]), -math.inf)


def _target(s, x):
    """(the targets' places, which rows have a target that is allowed)."""
    at = s["target"].long().clamp(min=0)[:, None]
    return at, ((s["target"] >= 0)[:, None] & (x.gather(1, at) > -math.inf))


def _plain_loss(s, x):
    """Overwrites x with exp((x - m) / T)."""
    T = s["case"]["temp"]
    top = x.amax(1, keepdim=True)
    alive = top > -math.inf
    at, there = _target(s, x)
    z = x.sub_(torch.where(alive, top, torch.zeros_like(top))).mul_(1.0 / T)
    zt = torch.where(there, z.gather(1, at), torch.zeros_like(top))
    e = z.exp_()
    hit = e.gather(1, at)
    rest = e.scatter_(1, at, 0.0).sum(1, keepdim=True)          # without the target: a loss near 0 keeps its precision
    total = rest + hit
    e.scatter_(1, at, hit)
    loss = torch.log1p(rest / zt.exp())
    s["loss"].copy_(torch.where(there, loss, torch.zeros_like(loss))[:, 0])
    s["lse"].copy_(torch.where(alive, top / T + total.log(), torch.full_like(top, -math.inf))[:, 0])
    s["norm"].copy_(torch.cat([top, total], 1))
    return e


def _plain_grad(s, x, e, h):
    """From e = exp((x - m) / T) (x, where given, is turned into it) to the gradients."""
    T = s["case"]["temp"]
    at = s["target"].long().clamp(min=0)[:, None]
    m, total = s["norm"][:, :1], s["norm"][:, 1:]
    if e is None:
        e = x.sub_(torch.where(m > -math.inf, m, torch.zeros_like(m))).mul_(1.0 / T).exp_()
    scale = torch.where(s["loss"] > 0, s["up"] / T, torch.zeros_like(s["up"]))[:, None]
    p = e.mul_(torch.where(total > 0, scale / total, torch.zeros_like(total)))
    p.scatter_(1, at, torch.where(scale != 0, torch.expm1(-s["loss"])[:, None] * scale, p.gather(1, at)))
    s["dh"].copy_(p @ s["w"].float())
    s["dw"].copy_(p.T @ h)
    return s["dh"], s["dw"]


def _plain_embed(table, tok, scale):
    x = table[tok.clamp(min=0).long()].float() * scale
    return torch.where((tok >= 0)[:, None], x, torch.zeros_like(x))


def _plain_embed_grad(rows, tok, scale, V):
    """The sums of the rows' gradients by token, in 32 bits."""
    out = torch.zeros((V + 1, rows.shape[1]), dtype=torch.float32, device=rows.device)
    out.index_add_(0, torch.where(tok >= 0, tok, torch.full_like(tok, V)).long(), rows.float())
    return out[:V].mul_(scale)


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "embed":
        s["out"].copy_(_plain_embed(s["w"], s["tok"], case["scale"]))
        return [s["out"]]
    if op == "embed_grad":
        s["out"].copy_(_plain_embed_grad(s["w"], s["tok"], case["scale"], case["V"]))
        return [s["out"]]
    if op == "tied":
        s["h"].copy_(_plain_embed(s["w"], s["tok"], case["scale"]))
    h = s["h"].float()
    x = _plain_logits(s, h)
    if op == "head_grad":
        return list(_plain_grad(s, x, None, h))
    e = _plain_loss(s, x)
    if op == "head_loss":
        return [s["loss"], s["lse"]]
    dh, dw = _plain_grad(s, None, e, h)
    if op == "head_train":
        return [s["loss"], s["lse"], dh, dw]
    dw.copy_(dw.float() + _plain_embed_grad(dh, s["tok"], case["scale"], case["V"]))
    return [s["loss"], s["lse"], dw]


def run(state):
    s, case, op = state, state["case"], state["case"]["op"]
    if not own:
        return _plain(s)
    ctx = s["ctx"]
    if op == "embed":
        ctx.embed(s["w"], s["tok"], s["out"], scale=case["scale"])
        return [s["out"]]
    if op == "embed_grad":
        ctx.embed_grad(s["w"], s["tok"], s["out"], scale=case["scale"])
        return [s["out"]]
    if op == "tied":
        ctx.embed(s["w"], s["tok"], s["h"], scale=case["scale"])
    if op != "head_grad":
        ctx.head_loss(s["h"], s["w"], s["target"], s["loss"], temp=case["temp"], bitmask=s["mask"], out_lse=s["lse"],
                      out_norm=s["norm"] if op != "head_loss" else None)
        if op == "head_loss":
            return [s["loss"], s["lse"]]
    ctx.head_grad(s["h"], s["w"], s["target"], s["loss"], s["norm"], out_grad_hidden=s["dh"], out_grad_weight=s["dw"],
                  temp=case["temp"], bitmask=s["mask"], grad_loss=s["up"])
    if op == "head_grad":
        return [s["dh"], s["dw"]]
    if op == "head_train":
        return [s["loss"], s["lse"], s["dh"], s["dw"]]
    ctx.embed_grad(s["dh"], s["tok"], s["dw"], scale=case["scale"], accumulate=True)
    return [s["loss"], s["lse"], s["dw"]]


# ---- work and the operators' definition in 64 bits --------------------------------

def work(case):
    rows, V, D, size, op = case["rows"], case["V"], case["D"], 2 if case["dtype"] == "bf16" else 4, case["op"]
    if op == "embed":
        return {"bytes": rows * (2 * D * size + 4), "flops": rows * D}
    if op == "embed_grad":
        return {"bytes": rows * (D * size + 4) + V * D * size, "flops": rows * D}
    product = 2 * rows * V * D
    read = (rows + V) * D * size + (rows * ((V + 31) // 32) * 4 if case["mask"] else 0)
    if op == "head_loss":
        return {"bytes": read + rows * 12, "flops": product}
    b = read + (rows + V) * D * size + rows * 24
    if op == "tied":
        b = read - rows * D * size + V * D * size + rows * 24
    return {"bytes": b, "flops": 3 * product}


def _exact_x(s, lo, hi, h, w):
    """Rows lo..hi of the logits in 64 bits, -inf where the mask forbids, and their targets."""
    x = h[lo:hi] @ w.T
    if s["mask"] is not None:
        words = s["mask"][lo:hi].long() & 0xFFFFFFFF
        bit = (words[:, :, None] >> torch.arange(32, device=x.device)) & 1
        x = x.masked_fill_(bit.reshape(hi - lo, -1)[:, :x.shape[1]] == 0, -math.inf)
    t = s["target"][lo:hi].long()
    xt = x.gather(1, t.clamp(min=0)[:, None])[:, 0]
    return x, t.clamp(min=0), (t >= 0) & (xt > -math.inf), xt


def _exact_loss(s, lo, hi, h, w):
    """(loss, log of the sum, normaliser as maximum and sum) of rows lo..hi; the loss as
    log(1 + the others' sum over the target's term), which keeps one near 0."""
    T = s["case"]["temp"]
    x, t, there, xt = _exact_x(s, lo, hi, h, w)
    top = x.amax(1)
    total = ((x - torch.where(top > -math.inf, top, torch.zeros_like(top))[:, None]) / T).exp().sum(1)
    others = torch.logsumexp(x.scatter(1, t[:, None], -math.inf) / T, 1)
    gap = torch.where(there, others - xt / T, torch.full_like(top, -math.inf))
    return torch.logaddexp(gap, torch.zeros_like(gap)), torch.logsumexp(x / T, 1), torch.stack([top, total], 1)


def _exact_grad(s, lo, hi, h, w):
    """(gradient by the rows lo..hi of h, by w) of the sum of up * loss."""
    T = s["case"]["temp"]
    x, t, there, _ = _exact_x(s, lo, hi, h, w)
    p = torch.softmax(x / T, 1).nan_to_num_(0.0)
    hit = p.gather(1, t[:, None])
    p.scatter_(1, t[:, None], 0.0)
    p.scatter_(1, t[:, None], torch.where(hit[:, 0] < 0.5, hit[:, 0] - 1.0, -p.sum(1))[:, None])
    p *= (s["up"][lo:hi].double() / T * there)[:, None]
    return p @ w, p.T @ h[lo:hi]


def exact(case, seed):
    s = prepare(case, seed)
    op, V, rows = case["op"], case["V"], case["rows"]
    if op in ("embed", "embed_grad"):
        there = s["tok"] >= 0
        if op == "embed":
            out = torch.zeros((rows, case["D"]), dtype=torch.float64, device="cuda")
            out[there] = s["w"][s["tok"][there].long()].double() * case["scale"]
        else:
            out = torch.zeros((V, case["D"]), dtype=torch.float64, device="cuda")
            out.index_add_(0, s["tok"][there].long(), s["w"][there].double())
            out *= case["scale"]
        return [out]
    w = s["w"].double()
    if op == "tied":
        # the embedding's output is held in the table's type: its rounding is part of the definition
        there = s["tok"] >= 0
        h = torch.zeros((rows, case["D"]), dtype=torch.float64, device="cuda")
        h[there] = (w[s["tok"][there].long()] * case["scale"]).to(s["w"].dtype).double()
    else:
        h = s["h"].double()
    step = max(1, int(6e7 // V))
    cuts = [(lo, min(rows, lo + step)) for lo in range(0, rows, step)]
    out = []
    if op != "head_grad":
        parts = [_exact_loss(s, lo, hi, h, w) for lo, hi in cuts]
        out = [torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])]
    if op == "head_loss":
        return out
    dh, dw = [], torch.zeros((V, case["D"]), dtype=torch.float64, device="cuda")
    for lo, hi in cuts:
        a, b = _exact_grad(s, lo, hi, h, w)
        dh.append(a)
        dw += b
    dh = torch.cat(dh)
    if op == "tied":
        there = s["tok"] >= 0
        dw.index_add_(0, s["tok"][there].long(), dh[there] * case["scale"])
        return out + [dw]
    return out + [dh, dw]
