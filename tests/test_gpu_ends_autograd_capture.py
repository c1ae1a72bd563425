"""The autograd forms of the model's two ends, forward and backward captured in a graph: on the context's own stream,
and on another one."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

PROGRAM = """
import torch
import grammar_constrained_decoding_gb300 as cg

def run(V, B, D, dtype, own):
    stream, capture = torch.cuda.Stream(), torch.cuda.Stream()
    ctx = cg.Ctx([cg.Grammar.compile('root ::= "a"', "gbnf")], cg.Vocab([i.to_bytes(3, "big") for i in range(V)]), stream)
    if own:
        capture = stream
    g = torch.Generator(device="cuda").manual_seed(V)
    new = lambda: (0.3 * torch.randn((V, D), generator=g, device="cuda")).to(dtype)
    ids = lambda: torch.randint(0, V, (B,), generator=g, device="cuda").int()
    table, tok, target = new().requires_grad_(), ids(), ids()

    def step(t):
        loss = cg.head_loss(ctx, cg.embed(ctx, t, tok, 0.5), t, target, 0.9)
        (grad,) = torch.autograd.grad(loss.mean(), t)
        return loss.detach(), grad

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=capture):
        loss, grad = step(table)
    for _ in range(3):
        with torch.no_grad():
            table.copy_(new())
        tok.copy_(ids())
        target.copy_(ids())
        torch.cuda.synchronize()
        with torch.cuda.stream(capture):
            graph.replay()
        torch.cuda.synchronize()
        want = step(table.detach().clone().requires_grad_())
        with torch.cuda.stream(capture):
            graph.replay()       # beside eager calls' memory
        torch.cuda.synchronize()
        assert ctx.status() == 0
        assert torch.equal(loss, want[0]) and torch.equal(grad, want[1]) and grad.float().isfinite().all() and bool(grad.any())

for own in (True, False):
    run(1003, 70, 40, torch.bfloat16, own)
    run(5000, 300, 129, torch.bfloat16, own)
    run(2000, 150, 72, torch.float32, own)
    run(2000, 5, 72, torch.float32, own)
print("captured")
"""


def test_autograd_forms_captured():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=root, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout + r.stderr
