"""Refusals of tensors that are not on the context's device, on a GPU."""

import numpy as np
import pytest

from tests.rows_ctx import f32_dev

pytestmark = pytest.mark.gpu


def test_distill_refuses_a_host_tensor_on_a_context_of_another_stream():
    """The refusal comes before anything is done with the tensor on the context's stream."""
    import torch
    import grammar_constrained_decoding_gb300 as cg
    V, B, K = 64, 2, 3
    side = torch.cuda.Stream()
    ctx = cg.Ctx([cg.Grammar.compile('root ::= "a"', "gbnf")], cg.Vocab([i.to_bytes(3, "big") for i in range(V)]), side)
    x, ids, t = torch.zeros((B, V), device="cuda"), torch.zeros((B, K), dtype=torch.int32, device="cuda"), f32_dev(np.zeros((B, K)))
    for bad in ((x.cpu(), ids, t), (x, ids.cpu(), t), (x, ids, t.cpu())):
        with pytest.raises(cg.CgError):
            cg.distill(ctx, *bad)
    assert torch.isfinite(cg.distill(ctx, x, ids, t)).all() and ctx.status() == 0
