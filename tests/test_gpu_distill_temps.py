"""Temperatures at the ends of what a call takes: T^2 alone need not be a float."""

import numpy as np
import pytest

from oracle import rows as R
from tests.gpu_helpers import empty, host, u32
from tests.rows_ctx import ctx_of, f32_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("temp", [1e20, 3e38, 1e-3, 1e-30])
@pytest.mark.parametrize("V,B", [(70, 6), (40000, 300)])
def test_one_allowed_token_has_no_loss(temp, V, B):
    """p and q of a row's only token are 1 at every temperature: loss and gradient are 0."""
    import torch
    rng = np.random.default_rng(V)
    x = torch.full((B, V), float("-inf"))
    at = rng.integers(0, V, B)
    x[torch.arange(B), torch.from_numpy(at)] = torch.from_numpy(rng.normal(0, 3, B).astype(np.float32))
    x = x.cuda()
    ids, t = u32(np.stack([at, rng.integers(0, V, B)], 1)), f32_dev(rng.normal(0, 2, (B, 2)))
    ctx = ctx_of(V)
    loss, loss2, norm = empty((B,), torch.float32), empty((B,), torch.float32), empty((B, 2), torch.float32)
    both, alone = torch.empty_like(x), torch.empty_like(x)
    ctx.distill_loss(x, ids, t, loss, temp=temp, out_norm=norm)
    ctx.distill_loss(x, ids, t, loss2, temp=temp, out_grad=both)
    ctx.distill_grad(x, ids, t, None, alone, temp=temp, norm=norm)
    assert ctx.status() == 0
    assert (loss == 0).all() and (loss2 == 0).all() and (both == 0).all() and (alone == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_cold_rows(dtype):
    """T = 0.01: p and q are nearly one token each, losses of hundreds of T^2 nats."""
    import torch
    V, B, K, temp = 4013, 8, 20, 0.01
    rng = np.random.default_rng(4)
    x = torch.from_numpy(rng.normal(0, 2, (B, V)).astype(np.float32)).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    v = x.double().numpy()
    ids, t = rng.integers(0, V, (B, K)).astype(np.uint32), rng.normal(0, 2, (B, K)).astype(np.float32)
    loss, ctx = empty((B,), torch.float32), ctx_of(V)
    ctx.distill_loss(x.cuda(), u32(ids), f32_dev(t), loss, temp=temp)
    assert ctx.status() == 0
    T = float(np.float32(temp))
    for b in range(B):
        want = R.distill_row(v[b], ids[b], t[b], T)[0]
        # terms of up to |x - m| / T nats, each good to 4 roundings, weights q to 3 roundings of |t - m| / T
        span = (v[b].max() - v[b].min()) / T
        spread = (t[b].max() - t[b].min()) / T
        assert abs(float(host(loss)[b]) - want) <= T * T * span * (8 + 3 * spread + K) * 2.0 ** -24, b
