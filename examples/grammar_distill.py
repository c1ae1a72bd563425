"""Distilling a constrained generator: sampling, record and training steps together.

A teacher (a table of next-token logits by last token) generates under a grammar,
each row with sampling settings of its own; for every position the best tokens
of its masked row are recorded.  A student table of the same shape learns from
the record under the same masks.  A second, narrow student learns from the
generated tokens themselves: one table is its embedding and its output layer.

    embed -> fill_bitmask -> sample_rows -> top_logprobs -> accept   (generation)
    embed -> distill -> backward -> step                             (training on the record)
    embed -> head_loss -> backward -> step                           (training on the tokens)

Run: python examples/grammar_distill.py
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import grammar_constrained_decoding_gb300 as cg  # noqa: E402
from workloads import GRAMMARS, make_vocab  # noqa: E402

PROMPT = b'calculate({"expression":"'


def generate(ctx, teacher, start, first, rows, steps, n_best, seed):
    """(last tokens, bitmasks, record ids, record logits, tokens), one entry per row and step."""
    V, W = ctx.V, ctx.W
    g = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda shape, dt: torch.empty(shape, dtype=dt, device="cuda")  # noqa: E731
    # every row has its own request: temperature, top-k, top-p, min-p
    r = torch.arange(rows, device="cuda")
    temp = torch.tensor([0.7, 1.0, 0.0, 1.3], device="cuda")[r % 4].contiguous()
    top_k = torch.tensor([20, 0, 0, 0], dtype=torch.int32, device="cuda")[r % 4].contiguous()
    top_p = torch.tensor([1.0, 0.9, 1.0, 1.0], device="cuda")[r % 4].contiguous()
    min_p = torch.tensor([0.0, 0.0, 0.0, 0.05], device="cuda")[r % 4].contiguous()
    states = torch.full((rows,), start, dtype=torch.int32, device="cuda").view(torch.uint32)
    counts = torch.zeros(rows, dtype=torch.int32, device="cuda").view(torch.uint32)
    last = torch.full((rows,), first, dtype=torch.int32, device="cuda")
    logits = new((rows, V), teacher.dtype)
    tok, flags = new((rows,), torch.int32), new((rows,), torch.uint8)
    out = []
    for _ in range(steps):
        mask, ids, best = new((rows, W), torch.int32), new((rows, n_best), torch.int32), new((rows, n_best), torch.float32)
        ctx.embed(teacher, last, logits)
        uniform = torch.rand((rows, V), generator=g, device="cuda")
        ctx.fill_bitmask(states, mask)
        ctx.sample_rows(logits, uniform, tok, bitmask=mask, temp=temp, top_k=top_k, top_p=top_p, min_p=min_p)
        ctx.top_logprobs(logits, ids, best, bitmask=mask)
        out.append((last, mask, ids, best, tok.clone()))
        ctx.accept(states, tok.view(torch.uint32), states, flags, counts=counts, max_tokens=256)
        last = tok.clamp(min=0)
    return [torch.cat(part) for part in zip(*out)]


def train_on_tokens(ctx, last, tokens, mask, width=64, epochs=30):
    """Mean cross entropy before and after training a table [V, width] that is both ends of the student (a row
    without a token has no target and does not count)."""
    torch.manual_seed(1)
    table = (0.3 * torch.randn(ctx.V, width, device="cuda")).requires_grad_()
    opt = torch.optim.Adam([table], lr=0.05)
    losses = []
    for _ in range(epochs):
        opt.zero_grad()
        loss = cg.head_loss(ctx, cg.embed(ctx, table, last), table, tokens, bitmask=mask).mean()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return losses[0].item(), losses[-1].item()


def main(rows=64, steps=24, n_best=16, epochs=30, verbose=True):
    """Returns the mean loss before and after training."""
    V = 512
    spec = GRAMMARS["calc_call"]
    grammar, vocab = cg.Grammar.compile(spec.source, spec.kind), make_vocab("tiny", V, 0)
    ctx = cg.Ctx([grammar], cg.Vocab(vocab))
    # the rows' prompt: the call up to its first free token
    _, start, _ = grammar.try_input(PROMPT)
    torch.manual_seed(0)
    teacher = (2.0 * torch.randn(V, V, device="cuda")).to(torch.bfloat16)
    student = torch.zeros(V, V, device="cuda", requires_grad=True)
    last, mask, ids, best, tokens = generate(ctx, teacher, start, vocab.index(PROMPT[-1:]), rows, steps, n_best, seed=1)
    opt = torch.optim.Adam([student], lr=0.3)
    first = None
    for epoch in range(epochs):
        opt.zero_grad()
        loss = cg.distill(ctx, cg.embed(ctx, student, last), ids, best, temp=1.0, bitmask=mask).mean()
        loss.backward()
        opt.step()
        first = loss.item() if first is None else first
        if verbose and epoch % 10 == 0:
            print(f"epoch {epoch}: loss {loss.item():.4f}")
    final = cg.distill(ctx, cg.embed(ctx, student.detach(), last), ids, best, temp=1.0, bitmask=mask).mean().item()
    if verbose:
        print(f"loss {first:.4f} -> {final:.4f} over {last.numel()} positions")
        print("on the tokens: loss %.4f -> %.4f" % train_on_tokens(ctx, last, tokens, mask))
    assert ctx.status() == 0
    return first, final


if __name__ == "__main__":
    main()
