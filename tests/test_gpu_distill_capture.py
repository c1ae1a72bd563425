"""The distillation calls captured in a graph as the first calls of a process:
they allocate nothing and ask the device nothing that a capture forbids."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

PROGRAM = """
import torch
import grammar_constrained_decoding_gb300 as cg

def run(V, B, K, dtype):
    side = torch.cuda.Stream()
    ctx = cg.Ctx([cg.Grammar.compile('root ::= "a"', "gbnf")], cg.Vocab([i.to_bytes(3, "big") for i in range(V)]), side)
    g = torch.Generator(device="cuda").manual_seed(V)
    rand = lambda: (torch.randn((B, V), generator=g, device="cuda") * 2).to(dtype)
    x = rand()
    ids = torch.randint(0, V, (B, K), generator=g, device="cuda").int()
    t = torch.randn((B, K), generator=g, device="cuda")
    up = torch.randn(B, generator=g, device="cuda")
    new = lambda: [torch.empty(B, device="cuda"), torch.empty(B, device="cuda"), torch.empty(B, device="cuda"),
                   torch.empty_like(x), torch.empty_like(x)]
    got, want = new(), new()
    def calls(loss, lse, loss2, both, alone):
        ctx.distill_loss(x, ids, t, loss, out_lse=lse, temp=1.5)
        ctx.distill_loss(x, ids, t, loss2, temp=1.5, out_grad=both, grad_loss=up)
        ctx.distill_grad(x, ids, t, lse, alone, temp=1.5, grad_loss=up)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        calls(*got)
    for _ in range(2):
        x.copy_(rand())
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        calls(*want)
        torch.cuda.synchronize()
        assert ctx.status() == 0
        for a, b in zip(got, want):
            assert torch.equal(a, b)
            assert torch.isfinite(a.float()).all()

run(5003, 9, 12, torch.bfloat16)       # rows that are held
run(40000, 300, 12, torch.bfloat16)    # rows that stream
run(40003, 200, 70, torch.float32)
print("captured")
"""


def test_distill_calls_captured_first():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=root, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout + r.stderr
