"""The ring of chunks that rows stream through: a slot, the bitmask's part of it
included, is filled again only after every lane has read it."""

import pytest

from tests.rows_ctx import ctx_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V,dtype,B,K", [(131072, "bf16", 500, 300), (65536, "f32", 400, 64), (30001, "bf16", 2000, 5)])
def test_masked_streamed_rows_give_the_same_bits_every_time(V, dtype, B, K):
    """Many rows through each ring with a bitmask, copied (16-byte rows of it) or read byte by
    byte, under the load of the gradient's stores; over the logits and beside them."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(V)
    x = (torch.randn((B, V), generator=g, device="cuda") * 2).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    mask = torch.randint(-2 ** 31, 2 ** 31, (B, (V + 31) // 32), generator=g, device="cuda").to(torch.int32)
    ids = torch.randint(0, V, (B, K), generator=g, device="cuda").int()
    t = torch.randn((B, K), generator=g, device="cuda")
    ctx, first = ctx_of(V), None
    for _ in range(25):
        loss, loss2, loss3, lse = (torch.empty(B, device="cuda") for _ in range(4))
        norm = torch.empty((B, 2), device="cuda")
        both, alone, over = torch.empty_like(x), torch.empty_like(x), x.clone()
        ctx.distill_loss(x, ids, t, loss, bitmask=mask, out_lse=lse, out_norm=norm)
        ctx.distill_loss(x, ids, t, loss2, bitmask=mask, out_grad=both)
        ctx.distill_grad(x, ids, t, None, alone, bitmask=mask, norm=norm)
        ctx.distill_loss(over, ids, t, loss3, bitmask=mask, out_grad=over)
        got = [loss, lse, norm, loss2, both, alone]
        if first is None:
            first = got
        assert all(torch.equal(a, b) for a, b in zip(got, first))
        assert torch.equal(over, both) and torch.equal(loss3, loss2)
    assert ctx.status() == 0
