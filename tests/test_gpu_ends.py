"""GPU tests of the embedding and the output layer together and at their edges:
autograd, streams, threads, captured graphs, large offsets, values that are not
finite, refusals.  Bounds of the sums: test_gpu_head.py."""

import os
import subprocess
import sys
import threading

import numpy as np
import pytest

from tests.rows_ctx import ctx_of
from tests.test_gpu_head import Exact, generator, make_bits, make_targets, matrix, pack, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def contexts_end_with_the_module():
    yield
    ctx_of.cache_clear()


def new_ctx(V, stream=None):
    import grammar_constrained_decoding_gb300 as cg
    return cg.Ctx([cg.Grammar.compile('root ::= "a"', "gbnf")], cg.Vocab([i.to_bytes(3, "big") for i in range(V)]), stream)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tied_step(dtype):
    """One table as both ends, through the calls as a training loop makes them: the gradient of the output
    layer, then the embedding's added to it, against the 64-bit gradients of what each call was given."""
    import torch
    V, B, D, T = 3001, 300, 96, 0.8
    ctx, g = ctx_of(V), generator(5)
    table = matrix(V, D, dtype, 0, 0, g, 0.3)
    tok = torch.randint(-1, V, (B,), generator=g, device="cuda").int()
    bits = make_bits(B, V, g)
    target, mask = make_targets(B, V, bits, g), pack(bits)
    up = torch.rand(B, generator=g, device="cuda")
    h, dh, dw = torch.empty(B, D, dtype=table.dtype, device="cuda"), torch.empty(B, D, dtype=table.dtype, device="cuda"), torch.empty_like(table)
    loss, norm = torch.empty(B, device="cuda"), torch.empty(B, 2, device="cuda")
    ctx.embed(table, tok, h, scale=2.0)
    ctx.head_loss(h, table, target, loss, temp=T, bitmask=mask, out_norm=norm)
    ctx.head_grad(h, table, target, loss, norm, dh, dw, temp=T, bitmask=mask, grad_loss=up)
    head = dw.double()
    e = Exact(h, table, target, T, bits, up.double(), dtype)
    e.check_grad(dh, dw)
    ctx.embed_grad(dh, tok, dw, scale=2.0, accumulate=True)
    assert ctx.status() == 0
    there = tok >= 0
    want, size = head.clone(), head.abs()
    want.index_add_(0, tok[there].long(), 2.0 * dh[there].double())
    size.index_add_(0, tok[there].long(), 2.0 * dh[there].double().abs())
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    assert bool(((dw.double() - want).abs() <= 10 * 2.0 ** -24 * size + half * want.abs() * 1.01 + 1e-38).all())


def test_gradients_against_differences():
    """Autograd through embed() and head_loss() on a float table against central differences of the 64-bit loss
    (step 1e-4: truncation about 1e-8; the kernels' 32 bits give the 5e-6)."""
    import torch
    import grammar_constrained_decoding_gb300 as cg
    V, B, D, T = 53, 6, 9, 1.3
    ctx, g = ctx_of(V), generator(2)
    table = torch.randn((V, D), generator=g, device="cuda")
    tok = torch.tensor([3, 7, 3, -1, 52, 0], dtype=torch.int32, device="cuda")
    target = torch.tensor([1, 7, -1, 4, 52, 30], dtype=torch.int32, device="cuda")
    bits = torch.rand((B, V), generator=g, device="cuda") < 0.7
    bits[torch.arange(B), target.clamp(min=0).long()] = True
    bits[5, 30] = False
    w = torch.randn(B, generator=g, device="cuda")

    def total(t):
        h = torch.where((tok >= 0)[:, None], 0.5 * t[tok.clamp(min=0).long()], 0.0)
        x = (h @ t.T / T).masked_fill(~bits, -torch.inf)
        loss = torch.logsumexp(x, 1) - x.gather(1, target.clamp(min=0).long()[:, None])[:, 0]
        counts = (target >= 0) & bits.gather(1, target.clamp(min=0).long()[:, None])[:, 0]
        return (torch.where(counts, loss, 0.0) * w.double()).sum()

    t32 = table.clone().requires_grad_()
    loss = cg.head_loss(ctx, cg.embed(ctx, t32, tok, 0.5), t32, target, T, pack(bits))
    (loss * w).sum().backward()
    assert loss[2] == 0 and loss[5] == 0 and abs(float((loss.detach() * w).sum() - total(table.double()))) < 1e-5
    for v in range(V):
        for d in range(D):
            hi, lo = table.double(), table.double()
            hi[v, d] += 1e-4
            lo[v, d] -= 1e-4
            diff = float(total(hi) - total(lo)) / 2e-4
            assert abs(diff - float(t32.grad[v, d])) < 5e-6, (v, d)


def test_autograd_wants_no_more_than_it_needs():
    import torch
    import grammar_constrained_decoding_gb300 as cg
    V, B, D = 600, 20, 32
    ctx = ctx_of(V)
    h, w = torch.randn(B, D, device="cuda"), torch.randn(V, D, device="cuda")
    t = torch.randint(0, V, (B,), device="cuda").int()
    both = [x.clone().requires_grad_() for x in (h, w)]
    cg.head_loss(ctx, *both, t).sum().backward()
    for i in (0, 1):
        one = [x.clone() for x in (h, w)]
        one[i].requires_grad_()
        cg.head_loss(ctx, *one, t).sum().backward()
        assert torch.equal(one[i].grad, both[i].grad) and one[1 - i].grad is None


def test_on_another_stream():
    """Inputs made and gradients used on a stream that is not the context's; the workspace is the context's stream's."""
    import torch
    import grammar_constrained_decoding_gb300 as cg
    V, B, D = 32003, 200, 96
    ctx = ctx_of(V)
    base = torch.randn(V, D, device="cuda")
    tok, target = (torch.randint(0, V, (B,), device="cuda").int() for _ in range(2))

    def step():
        t = (base * 0.3).requires_grad_()
        loss = cg.head_loss(ctx, cg.embed(ctx, t, tok), t, target)
        loss.sum().backward()
        return loss.detach().clone(), t.grad.clone()

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [step() for _ in range(5)]
    torch.cuda.synchronize()
    for loss, grad in got:
        assert torch.equal(loss, want[0]) and torch.equal(grad, want[1])


def test_threads_on_one_context():
    """Two threads call on one context, whose stream they share: each has a workspace of its own."""
    import torch
    V, B, D, n = 5000, 150, 64, 20
    ctx = ctx_of(V)
    inputs = []
    for k in range(2):
        g = generator(k)
        inputs.append((matrix(B, D, "bf16", 0, 0, g, 1.0), matrix(V, D, "bf16", 0, 0, g, 0.3),
                       torch.randint(0, V, (B,), generator=g, device="cuda").int()))

    def step(k, out):
        h, w, t = inputs[k]
        loss, norm = torch.empty(B, device="cuda"), torch.empty(B, 2, device="cuda")
        dh, dw, de = torch.empty_like(h), torch.empty_like(w), torch.empty_like(w)
        ctx.head_loss(h, w, t, loss, out_norm=norm)
        ctx.head_grad(h, w, t, loss, norm, dh, dw)
        ctx.embed_grad(dh, t, de)
        out.append((loss, dh, dw, de))

    want, got = [[], []], [[], []]
    for k in range(2):
        step(k, want[k])
    torch.cuda.synchronize()
    threads = [threading.Thread(target=lambda k=k: [step(k, got[k]) for _ in range(n)]) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert ctx.status() == 0
    for k in range(2):
        assert len(got[k]) == n
        for out in got[k]:
            assert all(torch.equal(a, b) for a, b in zip(out, want[k][0]))


CAPTURE = """
import torch
import grammar_constrained_decoding_gb300 as cg

def run(V, B, D, dtype):
    side = torch.cuda.Stream()
    ctx = cg.Ctx([cg.Grammar.compile('root ::= "a"', "gbnf")], cg.Vocab([i.to_bytes(3, "big") for i in range(V)]), side)
    g = torch.Generator(device="cuda").manual_seed(V)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)
    ids = lambda: torch.randint(0, V, (B,), generator=g, device="cuda").int()
    table, tok, target = rand(V, D), ids(), ids()
    new = lambda: [torch.empty(B, D, dtype=dtype, device="cuda"), torch.empty(B, device="cuda"), torch.empty(B, 2, device="cuda"),
                   torch.empty(B, D, dtype=dtype, device="cuda"), torch.empty(V, D, dtype=dtype, device="cuda")]
    def calls(h, loss, norm, dh, dw):
        ctx.embed(table, tok, h, scale=0.3)
        ctx.head_loss(h, table, target, loss, out_norm=norm)
        ctx.head_grad(h, table, target, loss, norm, dh, dw)
        ctx.embed_grad(dh, tok, dw, accumulate=True)
    torch.cuda.synchronize()
    sets, graphs = [new(), new()], []
    for out in sets:   # two graphs: each has a workspace of its own
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            calls(*out)
    want = new()
    for _ in range(3):
        table.copy_(rand(V, D))
        tok.copy_(ids())
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for graph in graphs:
                graph.replay()
            calls(*want)   # eager calls beside the graphs, on a workspace that is kept
            for graph in graphs:
                graph.replay()
        torch.cuda.synchronize()
        assert ctx.status() == 0
        for out in sets:
            for a, b in zip(out, want):
                assert torch.equal(a, b) and torch.isfinite(a.float()).all()
    # the two graphs at once, on two streams
    table.copy_(rand(V, D))
    torch.cuda.synchronize()
    others = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for s, graph in zip(others, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        calls(*want)
    torch.cuda.synchronize()
    assert ctx.status() == 0
    for out in sets:
        for a, b in zip(out, want):
            assert torch.equal(a, b)

run(1003, 70, 40, torch.bfloat16)
run(5000, 300, 129, torch.bfloat16)    # rows off the 16-byte grid
run(2000, 150, 72, torch.float32)
print("captured")
"""


def test_captured_first():
    """The calls captured in a graph as the first calls of a process, twice, and replayed beside eager calls."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CAPTURE], cwd=root, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_same_bits_every_time(dtype):
    import torch
    first = run(300, 20000, 200, dtype)
    for _ in range(3):
        for a, b in zip(run(300, 20000, 200, dtype), first):
            assert torch.equal(a, b)


@pytest.mark.parametrize("B,V,D,dtype", [(70001, 500, 16, "bf16"), (3, 500, 65536, "bf16"), (9, 388005, 40, "bf16"), (66000, 513, 8, "f32")])
def test_extremes(B, V, D, dtype):
    run(B, V, D, dtype, masked=B < 100)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B", [1, 7, 9, 17, 40, 63])
def test_few_rows_after_a_call_full_of_nan(B, dtype):
    """Tiles that few rows fill in part: what an earlier launch left in shared memory reaches nothing."""
    import torch
    V, D = 40000, 136
    ctx, dt = ctx_of(V), torch.bfloat16 if dtype == "bf16" else torch.float32
    h, w = (torch.full((n, D), float("nan"), dtype=dt, device="cuda") for n in (128, V))
    target = torch.zeros(128, dtype=torch.int32, device="cuda")
    loss, norm = torch.empty(128, device="cuda"), torch.empty((128, 2), device="cuda")
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    for masked in (True, False):
        ctx.head_loss(h, w, target, loss, out_norm=norm)
        ctx.head_grad(h, w, target, loss, norm, dh, dw)
        assert not loss.any() and ctx.status() == 0
        run(B, V, D, dtype, masked=masked)


@pytest.mark.parametrize("pad", [2 ** 23, 2 ** 23 + 1])
def test_rows_beyond_32_bit_offsets(pad):
    """Pitches that take the last rows of the weight and of its gradient past 2^32 elements, on the 16-byte grid
    and off it."""
    import torch
    V, B, D = 514, 130, 64
    ctx, g = ctx_of(V), generator(0)
    wide = [torch.empty((V - 1) * (D + pad) + D, dtype=torch.bfloat16, device="cuda").as_strided((V, D), (D + pad, 1)) for _ in range(2)]
    w, dw = wide
    w.copy_(torch.randn((V, D), generator=g, device="cuda") * 0.3)
    h = matrix(B, D, "bf16", 0, 0, g, 1.0)
    target = torch.randint(V - 20, V, (B,), generator=g, device="cuda").int()
    loss, lse, norm = (torch.empty(s, device="cuda") for s in ((B,), (B,), (B, 2)))
    dh = torch.empty_like(h)
    ctx.head_loss(h, w, target, loss, out_lse=lse, out_norm=norm)
    ctx.head_grad(h, w, target, loss, norm, dh, dw)
    out = torch.empty_like(h)
    ctx.embed(w, target, out)
    assert ctx.status() == 0 and torch.equal(out, w[target.long()])
    e = Exact(h, w, target, 1.0, None, torch.ones(B, dtype=torch.float64, device="cuda"), "bf16")
    e.check_loss(loss, lse, norm)
    e.check_grad(dh, dw)
    before = dw.clone()
    ctx.embed_grad(dh, target, dw, accumulate=True)
    want = before.double().index_add_(0, target.long(), dh.double())
    assert bool(((dw.double() - want).abs() <= 2.0 ** -8 * want.abs() * 1.01 + 2.0 ** -16).all())


def test_values_that_are_not_finite():
    """Forbidden tokens' logits reach nothing whatever they are; a NaN logit is not allowed, +inf counts as the
    largest finite value."""
    import torch
    V, B, D = 700, 40, 32
    ctx, g = ctx_of(V), generator(9)
    h, w = matrix(B, D, "bf16", 0, 0, g, 1.0), matrix(V, D, "bf16", 0, 0, g, 1.0)
    bits = torch.ones((B, V), dtype=torch.bool, device="cuda")
    bits[:, [5, 300, 699]] = False
    target = torch.randint(6, 290, (B,), generator=g, device="cuda").int()
    new = lambda: (torch.empty(B, device="cuda"), torch.empty(B, device="cuda"), torch.empty(B, 2, device="cuda"))  # noqa: E731
    clean, dirty, open_ = new(), new(), new()
    ctx.head_loss(h, w, target, clean[0], bitmask=pack(bits), out_lse=clean[1], out_norm=clean[2])
    w[5], w[300], w[699] = float("nan"), float("inf"), float("-inf")
    ctx.head_loss(h, w, target, dirty[0], bitmask=pack(bits), out_lse=dirty[1], out_norm=dirty[2])
    for a, b in zip(clean, dirty):
        assert torch.equal(a, b)
    # without the mask: the rows of inf give NaN or infinities of either sign (inf - inf, or all products of one sign)
    w[300] = w[699] = float("nan")
    ctx.head_loss(h, w, target, open_[0], out_lse=open_[1], out_norm=open_[2])
    for a, b in zip(clean, open_):
        assert torch.equal(a, b)
    h[3], h[3, 0], w[300], w[300, 0] = 0, 1, 0, float("inf")        # 1 inf + 0 0 ... : row 3's logit of 300 is +inf, others' +-inf
    h[:, 0] = h[:, 0].abs() + 0.5
    target[3] = 300
    ctx.head_loss(h, w, target, open_[0], out_lse=open_[1], out_norm=open_[2])
    big = float(np.finfo(np.float32).max)
    assert bool((open_[2][:, 0] == big).all()) and bool((open_[2][:, 1] == 1).all())
    assert open_[0][3] == 0 and bool((open_[0][[0, 1, 2, 4]] >= 0.99 * big).all())
    assert ctx.status() == 0
    # a NaN target is not allowed: the row does not count
    target[7] = 5
    ctx.head_loss(h, w, target, open_[0])
    assert open_[0][7] == 0


@pytest.mark.parametrize("up", [1.0, 1 / 85, -1 / 4095])
def test_one_gradient_for_all_rows_is_rounded_once(up):
    """bf16 terms under one g: the targets' terms are g / T (1 - p), p at most 0.1 here, rounded in units of g / T's
    significand to 2^-9 relative of a value next to a power of two, evenly spread: 2^-9 / sqrt 3.  The other terms
    are spread over many tokens, so their roundings count less than a third of that.  With the result's own
    rounding of 2^-8 / sqrt 3 or less on average over significands (sqrt(1/2) of it): 1.3 of what it gives alone."""
    import torch
    V, B, D, T = 4000, 300, 64, 0.85
    ctx, g = ctx_of(V), generator(3)
    h, w = matrix(B, D, "bf16", 0, 0, g, 1.0), matrix(V, D, "bf16", 0, 0, g, D ** -0.5)
    target = torch.randint(0, V, (B,), generator=g, device="cuda").int()
    loss, lse, norm = (torch.empty(s, device="cuda") for s in ((B,), (B,), (B, 2)))
    dh, dw, ups = torch.empty_like(h), torch.empty_like(w), torch.full((B,), up, device="cuda")
    ctx.head_loss(h, w, target, loss, temp=T, out_lse=lse, out_norm=norm)
    ctx.head_grad(h, w, target, loss, norm, dh, dw, temp=T, grad_loss=ups)
    e = Exact(h, w, target, T, None, ups.double(), "bf16")
    assert float(e.loss.min()) > 2.4   # p at most 0.1
    for got, want in ((dh, e.d @ e.w), (dw, e.d.T @ e.h)):
        once = float((want.bfloat16().double() - want).norm())
        assert float((got.double() - want).norm()) <= 1.3 * once


@pytest.mark.parametrize("B,D,pad", [(130, 136, 0), (200, 70, 1), (300, 72, 8), (700, 33, 7)])
def test_gradient_by_rows_is_rounded_once(B, D, pad):
    """bf16 terms under a g for each row: the targets' terms count whole, the others (p at most 0.1) are spread over
    many tokens, so their roundings of 2^-9 / sqrt 3 shrink with the number of them: below a third of the result's
    own.  1.3 of that alone, as above; one rounding more would make it 1.41."""
    import torch
    V, T = 4000, 0.85
    ctx, g = ctx_of(V), generator(B)
    h, w = matrix(B, D, "bf16", pad, 0, g, 1.0), matrix(V, D, "bf16", pad, 0, g, D ** -0.5)
    target = torch.randint(0, V, (B,), generator=g, device="cuda").int()
    target[5], target[9] = -1, V - 1
    loss, lse, norm = (torch.empty(s, device="cuda") for s in ((B,), (B,), (B, 2)))
    dh, up = torch.empty(B, D, dtype=h.dtype, device="cuda"), torch.rand(B, generator=g, device="cuda") - 0.3
    ctx.head_loss(h, w, target, loss, temp=T, out_lse=lse, out_norm=norm)
    ctx.head_grad(h, w, target, loss, norm, dh, temp=T, grad_loss=up)
    e = Exact(h, w, target, T, None, up.double(), "bf16")
    e.check_grad(dh, None)
    assert float(e.loss[target >= 0].min()) > 2.4
    want = e.d @ e.w
    assert float((dh.double() - want).norm()) <= 1.3 * float((want.bfloat16().double() - want).norm())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("B", [40, 200])
def test_a_gradient_that_is_not_finite_stays_visible(B, masked, dtype):
    """Rows whose g is infinite or NaN: their gradients, and those of the tokens that they allow, are not finite
    either; other rows, and tokens that they forbid, are as without them."""
    import torch
    V, D = 900, 40
    ctx, g = ctx_of(V), generator(B + masked)
    h, w = matrix(B, D, dtype, 0, 0, g, 1.0), matrix(V, D, dtype, 0, 0, g, 0.3)
    bad, half = torch.tensor([3, 17, 33], device="cuda"), V // 2
    bits = None
    if masked:
        bits = torch.rand((B, V), generator=g, device="cuda") < 0.8
        bits[bad, :half] = True
        bits[bad, half:] = False
    target = torch.randint(0, half, (B,), generator=g, device="cuda").int()
    if masked:
        bits.scatter_(1, target.long()[:, None], True)
    up = torch.rand(B, generator=g, device="cuda") - 0.3
    up[bad] = torch.tensor([torch.inf, torch.nan, -torch.inf], device="cuda")
    loss, lse, norm = (torch.empty(s, device="cuda") for s in ((B,), (B,), (B, 2)))
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    mask = pack(bits) if masked else None
    ctx.head_loss(h, w, target, loss, bitmask=mask, out_lse=lse, out_norm=norm)
    ctx.head_grad(h, w, target, loss, norm, dh, dw, bitmask=mask, grad_loss=up)
    assert ctx.status() == 0
    good = torch.ones(B, dtype=torch.bool, device="cuda")
    good[bad] = False
    assert not dh[bad].isfinite().any() and not dw[:half].isfinite().any()
    assert masked or not dw.isfinite().any()
    # the others against the definition without those rows (a row of g = 0 gives terms of 0)
    e = Exact(h, w, target, 1.0, bits, torch.where(good, up, 0.0).double(), dtype)
    dh[bad] = 0
    e.check_grad(dh, None)
    if masked:
        e.d, e.w = e.d[:, half:].contiguous(), e.w[half:]
        e.check_grad(None, dw[half:])


def test_rows_that_do_not_count():
    import torch
    from grammar_constrained_decoding_gb300._lib import CG_DEV_BAD_TOKEN
    V, B, D = 600, 6, 24
    ctx, g = ctx_of(V), generator(4)
    h, w = matrix(B, D, "f32", 0, 0, g, 1.0), matrix(V, D, "f32", 0, 0, g, 1.0)
    bits = torch.ones((B, V), dtype=torch.bool, device="cuda")
    bits[1] = False
    bits[2] = False
    bits[2, 17] = True
    bits[3, 17] = False
    target = torch.tensor([-1, 17, 17, 17, V, 17], dtype=torch.int32, device="cuda")
    loss, lse, norm = torch.empty(B, device="cuda"), torch.empty(B, device="cuda"), torch.empty(B, 2, device="cuda")
    dh, dw = torch.full_like(h, 9.0), torch.full_like(w, 9.0)
    ctx.head_loss(h, w, target, loss, bitmask=pack(bits), out_lse=lse, out_norm=norm)
    assert ctx.status() == CG_DEV_BAD_TOKEN and ctx.status() == 0
    # none, nothing allowed, the only allowed token, a forbidden one, past the vocabulary: all 0
    assert loss[:5].tolist() == [0.0] * 5 and loss[5] > 0
    assert lse[1] == -torch.inf and norm[1].tolist() == [-torch.inf, 0.0] and abs(float(lse[2] - h[2] @ w[17])) < 1e-4
    ctx.head_grad(h, w, target, loss, norm, dh, dw, bitmask=pack(bits))
    assert ctx.status() == 0
    assert not dh[:5].any() and bool(dh[5].any())
    e = Exact(h, w, torch.where(target == V, -1, target), 1.0, bits, torch.ones(B, dtype=torch.float64, device="cuda"), "f32")
    e.check_grad(dh, dw)


def test_empty_batch():
    import torch
    V, D = 600, 24
    ctx = ctx_of(V)
    none, w, dw = torch.empty((0, D), device="cuda"), torch.ones((V, D), device="cuda"), torch.ones((V, D), device="cuda")
    t, f = torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty(0, device="cuda")
    ctx.head_loss(none, w, t, f)
    ctx.head_grad(none, w, t, f, torch.empty((0, 2), device="cuda"), none, dw)
    assert not dw.any() and ctx.status() == 0


def test_refusals():
    import torch
    import grammar_constrained_decoding_gb300 as cg
    V, B, D = 600, 5, 24
    ctx = ctx_of(V)
    h, w, t = torch.ones((B, D), device="cuda"), torch.ones((V, D), device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    loss, norm = torch.full((B,), 7.0, device="cuda"), torch.full((B, 2), 7.0, device="cuda")
    dh, dw = torch.full((B, D), 7.0, device="cuda"), torch.full((V, D), 7.0, device="cuda")
    big = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    for args, kw in [((h, w[1:], t, loss), {}), ((h, w[:, 1:], t, loss), {}), ((h, w.bfloat16(), t, loss), {}), ((h, w, t.long(), loss), {}),
                     ((h, w, t[1:], loss), {}), ((h, w, t, loss[1:]), {}), ((h.cpu(), w, t, loss), {}), ((h.half(), w.half(), t, loss), {}),
                     ((h, w, t, loss), dict(temp=0.0)), ((h, w, t, loss), dict(temp=-1.0)), ((h, w, t, loss), dict(temp=float("nan"))),
                     ((h, w, t, loss), dict(temp=float("inf"))), ((h, w, t, loss), dict(bitmask=t)), ((h[0], w, t, loss), {}),
                     ((h, w, t, loss), dict(workspace=big[:16])), ((h, w, t, loss), dict(workspace=big[4:])),
                     ((h, w, t, loss), dict(out_norm=loss)), ((h.t(), w, t, loss), {}), ((h[:, :0], w[:, :0], t, loss), {})]:
        with pytest.raises((cg.CgError, IndexError)):
            ctx.head_loss(*args, **kw)
    for bad in (dh.half(), dh[0], dh.long(), dh.cpu()):
        with pytest.raises(cg.CgError):
            ctx.embed_workspace(bad, t)
    both = torch.ones((V, 2 * D), device="cuda")
    for args, kw in [((h, w, t, loss, norm), {}), ((h, w, t, loss, norm, h, dw), {}), ((h, w, t, loss, norm, dh, w), {}),
                     ((h, w, t, loss, norm, dh, dw[1:]), {}), ((h, w, t, loss, norm, dw[:B], dw), {}), ((h, w, t, loss, loss, dh, dw), {}),
                     ((h, w, t, loss, norm, dh.bfloat16(), dw), {}), ((h, w, t, loss, norm, dh, dw), dict(workspace=big[:16])),
                     ((h, w, t, loss, norm, dh, dw), dict(grad_loss=norm)), ((h, both[:, :D], t, loss, norm, None, both[:, 1:D + 1]), {})]:
        with pytest.raises(cg.CgError):
            ctx.head_grad(*args, **kw)
    assert bool((loss == 7).all()) and bool((dh == 7).all()) and bool((dw == 7).all()) and ctx.status() == 0
    ctx.head_loss(h, both[:, :D], t, loss, out_norm=norm)
    ctx.head_grad(h, both[:, :D], t, loss, norm, None, both[:, D:])   # other columns of the same buffer
    assert ctx.status() == 0


def test_example_trains_on_the_tokens():
    """The example's second student runs, and its gradients are the formula's (test_gradients_against_differences)."""
    import torch
    from examples.grammar_distill import generate, train_on_tokens
    import grammar_constrained_decoding_gb300 as cg
    from workloads import GRAMMARS, make_vocab
    V = 512
    spec, vocab = GRAMMARS["calc_call"], make_vocab("tiny", V, 0)
    ctx = cg.Ctx([cg.Grammar.compile(spec.source, spec.kind)], cg.Vocab(vocab))
    teacher = torch.randn(V, V, device="cuda").to(torch.bfloat16)
    last, mask, ids, best, tokens = generate(ctx, teacher, 0, 0, 16, 8, 4, seed=1)
    first, final = train_on_tokens(ctx, last, tokens, mask, epochs=3)
    assert np.isfinite(first) and np.isfinite(final) and ctx.status() == 0
