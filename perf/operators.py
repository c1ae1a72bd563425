"""Workloads of the vocabulary-row operators: sampling with per-row
temperature, top-k, top-p and min-p from given random numbers
(``Ctx.sample_rows``), the best tokens of each row with their log-probabilities
(``Ctx.top_logprobs``) and distillation from a teacher's recorded top logits
(``Ctx.distill_loss``, ``Ctx.distill_grad``).

``own`` chooses what ``run`` computes: False, the operators' plain form in
elementary torch operations in 32 bits; True, the calls a user of the package
makes.  Every pass takes logits [rows, V] on the device (contiguous, or rows of
a wider buffer when ``pad`` > 0), optionally the grammar's bitmask u32 [rows, W].
"""

from __future__ import annotations

import functools
import math

import torch

own = False

NO_TOKEN = -1          # CG_NO_TOKEN in an int32 tensor
U_LO, U_HI = 2.0 ** -32, 1.0 - 2.0 ** -24


def listed():
    return [
        # a lone chat request on the 32000-token vocabulary: the latency of one decode step
        dict(name="sample_1x32000", op="sample", rows=1, V=32000, dtype="bf16", pad=0, mask=True, logits="peaked",
             params="chat"),
        # a small server batch, every request with settings of its own, under the grammar's mask
        dict(name="sample_32x128256_mixed", op="sample", rows=32, V=128256, dtype="bf16", pad=0, mask=True,
             logits="peaked", params="mixed"),
        # the throughput workload: flat logits, T = 0.7, top-p 0.9, a nucleus of thousands of tokens
        dict(name="sample_256x128256_topp", op="sample", rows=256, V=128256, dtype="bf16", pad=0, mask=True,
             logits="flat", params="topp"),
        # the widest batch: mixed requests over 151936 tokens, no grammar on them
        dict(name="sample_512x151936_mixed", op="sample", rows=512, V=151936, dtype="bf16", pad=0, mask=False,
             logits="peaked", params="mixed"),
        # float logits of an odd vocabulary whose rows sit in a padded buffer
        dict(name="sample_48x32003_f32", op="sample", rows=48, V=32003, dtype="f32", pad=29, mask=True,
             logits="flat", params="chat"),
        # logprobs of a few requests: the 20 best allowed tokens of each step
        dict(name="top20_8x128256", op="top", rows=8, V=128256, dtype="bf16", pad=0, mask=True, logits="peaked",
             n=20),
        # a teacher's record over a batch of positions: 64 tokens a position
        dict(name="top64_2048x32000", op="top", rows=2048, V=32000, dtype="bf16", pad=0, mask=False, logits="flat",
             n=64),
        # float logits, odd vocabulary, a short list
        dict(name="top5_96x4013_f32", op="top", rows=96, V=4013, dtype="f32", pad=0, mask=True, logits="flat", n=5),
        # a training step's loss and gradient together, the largest: 2048 positions of 128256 tokens
        dict(name="distill_2048x128256", op="distill", rows=2048, V=128256, dtype="bf16", pad=0, mask=False,
             logits="flat", n=64, temp=2.0, grad=True),
        # an evaluation pass: the loss alone, under the grammar's mask
        dict(name="distill_loss_512x128256", op="distill", rows=512, V=128256, dtype="bf16", pad=0, mask=True,
             logits="peaked", n=64, temp=1.0, grad=False),
        # the backward pass alone, from the kept normaliser and an upstream gradient
        dict(name="distill_grad_512x151936", op="distill_grad", rows=512, V=151936, dtype="bf16", pad=0, mask=True,
             logits="flat", n=32, temp=1.5),
        # float logits of an odd vocabulary: loss and gradient
        dict(name="distill_64x32003_f32", op="distill", rows=64, V=32003, dtype="f32", pad=0, mask=True,
             logits="flat", n=50, temp=1.0, grad=True),
    ]


def draw(rng):
    """One more case: vocabularies of 500 to 152000 tokens (mostly odd sizes), 1 to 2048 rows."""
    op = rng.choice(["sample", "sample", "top", "distill", "distill_grad"])
    V = int(math.exp(rng.uniform(math.log(500), math.log(152000))))
    V = V if rng.random() < 0.7 else max(512, V // 64 * 64)
    most = 2048 if op != "sample" else 512
    cells = 2.0e8 if op.startswith("distill") else 6.0e7
    rows = int(math.exp(rng.uniform(0.0, math.log(max(2.0, min(most, cells / V))))))
    case = dict(op=op, rows=max(1, rows), V=V, dtype=rng.choice(["bf16", "bf16", "f32"]),
                pad=rng.choice([0, 0, 5, 64]), mask=rng.random() < 0.7, logits=rng.choice(["flat", "peaked"]))
    if op == "sample":
        case["params"] = rng.choice(["chat", "mixed", "topp", "full"])
    else:
        case["n"] = int(math.exp(rng.uniform(0.0, math.log(128))))
    if op.startswith("distill"):
        case["temp"] = rng.choice([0.7, 1.0, 2.0])
        if op == "distill":
            case["grad"] = rng.random() < 0.7
    return case


# ---- inputs -----------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _logits(case, g):
    """flat: N(0, 2) with 5% of the tokens 4 higher, the repository's synthetic
    workloads; peaked: N(0, 2) and 24 tokens a row raised by up to 14, as a
    trained model's rows are."""
    rows, V, ld = case["rows"], case["V"], case["V"] + case["pad"]
    buf = torch.randn((rows, ld), generator=g, device="cuda")
    buf *= 2.0
    if case["logits"] == "flat":
        buf += 4.0 * (torch.rand((rows, ld), generator=g, device="cuda") < 0.05)
    else:
        at = torch.randint(0, V, (rows, 24), generator=g, device="cuda")
        buf.scatter_add_(1, at, 14.0 * torch.rand((rows, 24), generator=g, device="cuda"))
    buf = buf.to(torch.bfloat16) if case["dtype"] == "bf16" else buf
    return buf[:, :V]


def _bitmask(rows, V, g):
    """Masks as grammar states give them: most rows inside a string (nearly all
    tokens allowed), some at punctuation (a few tokens), a forced token now
    and then, and a dead row."""
    W = (V + 31) // 32
    r = torch.arange(rows, device="cuda")
    share = torch.full((rows,), 0.93, device="cuda")
    share[r % 4 == 1] = 0.002
    share[r % 8 == 6] = 0.3
    bits = torch.zeros((rows, W * 32), dtype=torch.bool, device="cuda")
    bits[:, :V] = torch.rand((rows, V), generator=g, device="cuda") < share[:, None]
    forced = r[r % 16 == 11]
    bits[forced] = False
    bits[forced, (forced * 977 + 5) % V] = True
    bits[r[r % 97 == 13]] = False
    w = bits.view(rows, W, 32).to(torch.int64) << torch.arange(32, device="cuda")
    w = w.sum(2)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32).contiguous()


def _params(case):
    """Per-row settings: chat, one usual setting for every row; topp, the
    throughput workload's; full, temperature alone; mixed, eight kinds of
    request in turn (the last draws from every allowed token)."""
    r = torch.arange(case["rows"], device="cuda")
    if case["params"] == "chat":
        t, k, p, m = [0.7], [50], [0.9], [0.0]
    elif case["params"] == "topp":
        t, k, p, m = [0.7], [0], [0.9], [0.0]
    elif case["params"] == "full":
        t, k, p, m = [1.0], [0], [1.0], [0.0]
    else:
        t = [0.7, 0.0, 1.0, 1.0, 0.8, 1.3, 0.6, 1.0]
        k = [50, 0, 0, 0, 40, 0, 0, 0]
        p = [0.9, 1.0, 0.95, 1.0, 1.0, 0.98, 0.8, 1.0]
        m = [0.0, 0.0, 0.0, 0.05, 0.02, 0.1, 0.0, 0.0]
    pick = lambda v, dt: torch.tensor(v, dtype=dt, device="cuda")[r % len(v)].contiguous()  # noqa: E731
    return pick(t, torch.float32), pick(k, torch.int32), pick(p, torch.float32), pick(m, torch.float32)


@functools.lru_cache(maxsize=None)
def _ctx(V):
    """The context a program keeps: one small grammar and a vocabulary of V tokens."""
    import grammar_constrained_decoding_gb300 as cg
    grammar = cg.Grammar.compile('root ::= "a"', "gbnf")
    return cg.Ctx([grammar], cg.Vocab([i.to_bytes(3, "big") for i in range(V)]))


def prepare(case, seed):
    g = _gen(seed)
    rows, V = case["rows"], case["V"]
    s = {"case": case, "x": _logits(case, g), "mask": _bitmask(rows, V, g) if case["mask"] else None}
    if own:
        s["ctx"] = _ctx(V)
    if case["op"] == "sample":
        s["temp"], s["top_k"], s["top_p"], s["min_p"] = _params(case)
        s["u"] = torch.rand((rows, V), generator=g, device="cuda")
        s["tok"] = torch.empty(rows, dtype=torch.int32, device="cuda")
        s["lp"] = torch.empty(rows, dtype=torch.float32, device="cuda")
    elif case["op"] == "top":
        s["ids"] = torch.empty((rows, case["n"]), dtype=torch.int32, device="cuda")
        s["lps"] = torch.empty((rows, case["n"]), dtype=torch.float32, device="cuda")
        s["lse"] = torch.empty(rows, dtype=torch.float32, device="cuda")
    else:
        # the teacher's record: the best tokens of a model near the student; every
        # fifth row's list is half empty
        K = min(case["n"], V)
        t = s["x"].float() + torch.randn((rows, V), generator=g, device="cuda")
        t_max = t.amax(1, keepdim=True)
        norm = t_max + (t - t_max).exp_().sum(1, keepdim=True).log_()
        best, ids = torch.topk(t, K, dim=1)
        ids = ids.to(torch.int32)
        half = (torch.arange(rows, device="cuda") % 5 == 1)[:, None] & (torch.arange(K, device="cuda") >= (K + 1) // 2)
        s["ids"] = torch.where(half, torch.full_like(ids, NO_TOKEN), ids).contiguous()
        s["teacher"] = (best - norm).contiguous()
        s["loss"] = torch.empty(rows, dtype=torch.float32, device="cuda")
        s["lse"] = torch.empty(rows, dtype=torch.float32, device="cuda")
        s["up"] = torch.rand(rows, generator=g, device="cuda") / rows
        if case["op"] == "distill_grad" or case["grad"]:
            s["dx"] = torch.empty((rows, V), dtype=s["x"].dtype, device="cuda")
        if case["op"] == "distill_grad":
            xd = _masked(s["x"].double(), s["mask"])
            s["lse"] = torch.logsumexp(xd / case["temp"], 1).float()
    return s


# ---- the plain form ---------------------------------------------------------------

def _allowed(mask, V):
    at = torch.arange(V, device=mask.device)
    return ((mask[:, at >> 5] >> (at & 31).to(torch.int32)) & 1).bool()


def _masked(x, mask):
    if mask is None:
        return x
    return torch.where(_allowed(mask, x.shape[1]), x, torch.full_like(x, -math.inf))


def _plain_sample(s):
    x = _masked(s["x"].float(), s["mask"])
    V = x.shape[1]
    top = x.amax(1, keepdim=True)
    alive = top > -math.inf
    greedy = s["temp"][:, None] == 0
    d = torch.where(alive, x - top, torch.full_like(x, -math.inf))
    z = d / torch.where(greedy, torch.ones_like(top), s["temp"][:, None])
    e = z.exp()
    total = e.sum(1, keepdim=True)
    best = torch.sort(d, dim=1, descending=True).values
    k = s["top_k"][:, None].long()
    k = torch.where(k == 0, torch.full_like(k, V), k).clamp(max=V)
    cut = best.gather(1, k - 1)
    p = s["top_p"][:, None]
    eb = (best / torch.where(greedy, torch.ones_like(top), s["temp"][:, None])).exp() * (best >= cut)
    cum = eb.cumsum(1)
    reach = cum >= p * cum[:, -1:]
    first = torch.where(reach.any(1, keepdim=True), reach.int().argmax(1, keepdim=True),
                        torch.full_like(k, V - 1))
    cut = torch.where(p < 1, torch.maximum(cut, best.gather(1, first)), cut)
    keep = (d >= cut) & (z >= s["min_p"][:, None].log()) & (d > -math.inf)
    keep = torch.where(greedy, d == 0, keep)
    gumbel = -(-s["u"].clamp(U_LO, U_HI).log()).log()
    score = torch.where(keep, torch.where(greedy, torch.zeros_like(z), z + gumbel), torch.full_like(z, -math.inf))
    at = torch.arange(V, device=x.device)[None, :]
    tok = torch.where(keep & (score == score.amax(1, keepdim=True)), at, torch.full_like(at, V)).amin(1)
    lp = (z - total.log()).gather(1, tok.clamp(max=V - 1)[:, None])[:, 0]
    alive = alive[:, 0]
    s["tok"].copy_(torch.where(alive, tok, torch.full_like(tok, NO_TOKEN)).to(torch.int32))
    s["lp"].copy_(torch.where(alive, lp, torch.full_like(lp, -math.inf)))
    return s["tok"], s["lp"]


def _plain_top(s):
    x = _masked(s["x"].float(), s["mask"])
    n = min(s["case"]["n"], x.shape[1])
    top = x.amax(1, keepdim=True)
    alive = top > -math.inf
    d = torch.where(alive, x - top, torch.full_like(x, -math.inf))
    log_total = d.exp().sum(1, keepdim=True).log()
    vals, ids = torch.sort(d, dim=1, descending=True, stable=True)
    vals, ids = vals[:, :n], ids[:, :n]
    s["ids"].fill_(NO_TOKEN)
    s["lps"].fill_(-math.inf)
    there = vals > -math.inf
    s["ids"][:, :n] = torch.where(there, ids, torch.full_like(ids, NO_TOKEN)).to(torch.int32)
    s["lps"][:, :n] = torch.where(there, vals - log_total, torch.full_like(vals, -math.inf))
    s["lse"].copy_(torch.where(alive, top + log_total, torch.full_like(top, -math.inf))[:, 0])
    return s["ids"], s["lps"], s["lse"]


def _teacher(s, x):
    """(weights q of the teacher's listed tokens, their ids, which count)."""
    ids = s["ids"].long()
    at = ids.clamp(min=0)
    there = (ids >= 0) & (x.gather(1, at) > -math.inf)
    t = torch.where(there, s["teacher"], torch.full_like(s["teacher"], -math.inf)) / s["case"]["temp"]
    t_max = t.amax(1, keepdim=True)
    t = torch.where(there, t - t_max, torch.full_like(t, -math.inf))
    log_sum = t.exp().sum(1, keepdim=True).log()
    log_q = torch.where(there, t - log_sum, torch.zeros_like(t))
    return torch.where(there, log_q.exp(), torch.zeros_like(t)), log_q, at, there


def _plain_grad(s, x, p, q, at, there, up):
    T = s["case"]["temp"]
    dx = torch.where(there.any(1, keepdim=True), p, torch.zeros_like(p))
    dx = dx.scatter_add(1, at, -q)
    s["dx"].copy_(dx * (T * up[:, None]))
    return s["dx"]


def _plain_distill(s):
    T = s["case"]["temp"]
    x = _masked(s["x"].float(), s["mask"])
    q, log_q, at, there = _teacher(s, x)
    if s["case"]["op"] == "distill_grad":
        p = (x / T - s["lse"][:, None]).exp()
        p = torch.where(x > -math.inf, p, torch.zeros_like(p))
        return [_plain_grad(s, x, p, q, at, there, s["up"])]
    top = x.amax(1, keepdim=True)
    alive = top > -math.inf
    z = torch.where(alive, (x - top) / T, torch.full_like(x, -math.inf))
    total = z.exp().sum(1, keepdim=True)
    log_total = total.log()
    zk = torch.where(there, z.gather(1, at), torch.zeros_like(q))
    part = torch.where(there, q * (log_q - zk + log_total), torch.zeros_like(q))
    s["loss"].copy_(part.sum(1) * (T * T))
    s["lse"].copy_(torch.where(alive, top / T + log_total, torch.full_like(top, -math.inf))[:, 0])
    out = [s["loss"], s["lse"]]
    if s["case"]["grad"]:
        p = torch.where(alive, z.exp() / total, torch.zeros_like(z))
        out.append(_plain_grad(s, x, p, q, at, there, s["up"]))
    return out


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"sample": _plain_sample, "top": _plain_top, "distill": _plain_distill,
                "distill_grad": _plain_distill}[op](s)
    ctx = s["ctx"]
    if op == "sample":
        ctx.sample_rows(s["x"], s["u"], s["tok"], bitmask=s["mask"], temp=s["temp"], top_k=s["top_k"],
                        top_p=s["top_p"], min_p=s["min_p"], out_logprob=s["lp"])
        return s["tok"], s["lp"]
    if op == "top":
        ctx.top_logprobs(s["x"], s["ids"], s["lps"], bitmask=s["mask"], out_lse=s["lse"])
        return s["ids"], s["lps"], s["lse"]
    T = s["case"]["temp"]
    if op == "distill_grad":
        ctx.distill_grad(s["x"], s["ids"], s["teacher"], s["lse"], s["dx"], temp=T, bitmask=s["mask"],
                         grad_loss=s["up"])
        return [s["dx"]]
    dx = s["dx"] if s["case"]["grad"] else None
    ctx.distill_loss(s["x"], s["ids"], s["teacher"], s["loss"], temp=T, bitmask=s["mask"], out_lse=s["lse"],
                     out_grad=dx, grad_loss=s["up"] if dx is not None else None)
    return [s["loss"], s["lse"]] + ([dx] if dx is not None else [])


# ---- work and the operators' definition in 64 bits --------------------------------

def work(case):
    rows, V, size = case["rows"], case["V"], 2 if case["dtype"] == "bf16" else 4
    cells = rows * V
    b = cells * size + (rows * ((V + 31) // 32) * 4 if case["mask"] else 0)
    if case["op"] == "sample":
        b += rows * (16 + 4 + 8)                    # settings, one random number at least, token and log-probability
        full = {"full": rows, "mixed": rows // 8}.get(case["params"], 0)
        b += int(full * V * 4 * (0.8 if case["mask"] else 1.0))   # rows without a cut need every allowed token's number
        return {"bytes": b, "flops": 4 * cells}     # difference, scale, exponential, sum
    K = min(case["n"], V)
    if case["op"] == "top":
        return {"bytes": b + rows * (8 * case["n"] + 4), "flops": 3 * cells}
    b += rows * (8 * K + 12)
    if case["op"] == "distill_grad" or case["grad"]:
        b += cells * size
    return {"bytes": b, "flops": (4 if case["op"] == "distill" else 3) * cells}


def _exact_rows(s, lo, hi):
    """Rows lo..hi in 64 bits: values with -inf where the mask forbids, and the allowed set."""
    x = s["x"][lo:hi].double()
    if s["mask"] is not None:
        words = s["mask"][lo:hi].long() & 0xFFFFFFFF
        bit = (words[:, :, None] >> torch.arange(32, device=x.device)) & 1
        x = x.masked_fill(bit.reshape(hi - lo, -1)[:, :x.shape[1]] == 0, -math.inf)
    return x


def _exact_sample(s, lo, hi):
    toks, lps = [], []
    x = _exact_rows(s, lo, hi)
    for i in range(hi - lo):
        ids = torch.nonzero(x[i] > -math.inf)[:, 0]
        if ids.numel() == 0:
            toks.append(NO_TOKEN)
            lps.append(-math.inf)
            continue
        v = x[i][ids]
        T = float(s["temp"][lo + i])
        if T == 0:
            j = int((v == v.max()).int().argmax())
            toks.append(int(ids[j]))
            lps.append(float(v[j] - torch.logsumexp(v, 0)))
            continue
        logp = torch.log_softmax(v / T, 0)
        k, p, m = int(s["top_k"][lo + i]), float(s["top_p"][lo + i]), float(s["min_p"][lo + i])
        keep = torch.ones_like(v, dtype=torch.bool)
        if 0 < k < v.numel():
            keep &= v >= torch.topk(v, k).values[-1]
        if p < 1:
            w = torch.where(keep, logp.exp(), torch.zeros_like(v))
            order = torch.argsort(v, descending=True)
            cum = torch.cumsum(w[order], 0)
            j = int((cum < p * w.sum()).sum().clamp(max=v.numel() - 1))
            keep &= v >= v[order[j]]
        if m > 0:
            keep &= (v - v.max()) / T >= math.log(min(m, 1.0))
        u = s["u"][lo + i][ids].double().clamp(U_LO, U_HI)
        score = torch.where(keep, logp - torch.log(-torch.log(u)), torch.full_like(v, -math.inf))
        j = int((score == score.max()).int().argmax())
        toks.append(int(ids[j]))
        lps.append(float(logp[j]))
    return torch.tensor(toks, dtype=torch.int32, device=x.device), torch.tensor(lps, dtype=torch.float64, device=x.device)


def _exact_top(s, lo, hi):
    n = s["case"]["n"]
    x = _exact_rows(s, lo, hi)
    m = min(n, x.shape[1])
    lse = torch.logsumexp(x, 1)
    order = torch.argsort(x, dim=1, descending=True, stable=True)[:, :m]
    v = x.gather(1, order)
    ids = torch.full((hi - lo, n), NO_TOKEN, dtype=torch.int32, device=x.device)
    lps = torch.full((hi - lo, n), -math.inf, dtype=torch.float64, device=x.device)
    ids[:, :m] = order.masked_fill(v == -math.inf, NO_TOKEN).to(torch.int32)
    lps[:, :m] = torch.where(v == -math.inf, v, v - lse[:, None])
    return ids, lps, lse


def _exact_distill(s, lo, hi):
    T = s["case"]["temp"]
    x = _exact_rows(s, lo, hi)
    ids, t = s["ids"][lo:hi].long(), s["teacher"][lo:hi].double() / T
    z = x / T
    lse = torch.logsumexp(z, 1)
    listed_ = ids >= 0
    zk = z.gather(1, ids.clamp(min=0))
    listed_ &= zk > -math.inf
    q = torch.softmax(t.masked_fill(~listed_, -math.inf), 1).nan_to_num(0.0)
    log_pk = (zk - lse[:, None]).masked_fill(~listed_, 0.0)
    loss = T * T * (torch.special.xlogy(q, q) - q * log_pk).sum(1)
    if s["case"]["op"] == "distill" and not s["case"]["grad"]:
        return loss, lse
    used = listed_.any(1)
    p = (z - lse[:, None]).exp().masked_fill(~used[:, None] | (x == -math.inf), 0.0)
    p.scatter_add_(1, ids.clamp(min=0), -q)
    dx = p * (T * s["up"][lo:hi].double()[:, None])
    return [dx] if s["case"]["op"] == "distill_grad" else [loss, lse, dx]


def exact(case, seed):
    s = prepare(case, seed)
    step = max(1, int(4e7 // case["V"]))
    f = {"sample": _exact_sample, "top": _exact_top}.get(case["op"], _exact_distill)
    parts = [f(s, lo, min(case["rows"], lo + step)) for lo in range(0, case["rows"], step)]
    return [torch.cat(c) for c in zip(*parts)]
