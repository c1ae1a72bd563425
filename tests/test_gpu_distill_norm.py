"""The backward pass of the distillation loss on rows whose log-normaliser does
not fit 32 bits: float logits far from zero and logits of +inf (which count as
the largest finite value).

Tolerances.  p carries the normaliser's error (rel_sum) and that of its own
argument z = (x - m) / T, whose difference, scale and product round once each:
3 |z| 2^-24, with 16 x 2^-24 for the quotient, q and the factors; the result is
rounded to the dtype once more.
"""

import numpy as np
import pytest

from oracle import rows as R
from tests.gpu_helpers import empty, host, u32
from tests.rows_ctx import ctx_of, f32_dev, rel_sum

pytestmark = pytest.mark.gpu

KINDS = ["million", "minus_million", "thousands", "inf", "lowest"]


def make(rng, B, V, kind):
    """Rows, and of each the tokens that hold most of its mass."""
    x = rng.normal(0, 2, (B, V))
    high = np.stack([rng.choice(V, 3, replace=False) for _ in range(B)])
    if kind == "million":
        x += 1.0e6
    elif kind == "minus_million":
        x -= 1.0e6
    elif kind == "thousands":
        x *= 1.0e3
    elif kind == "inf":
        for b in range(B):
            x[b, high[b]] = np.inf
    elif kind == "lowest":
        x[:] = -np.inf
        for b in range(B):
            x[b, high[b]] = -R.MAX_F32
    return x.astype(np.float32), high


def to_dtype(x, dtype):
    import torch
    t = torch.from_numpy(x).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    if dtype == "bf16":  # the lowest finite float rounds to -inf
        t = torch.where(torch.from_numpy(x == np.float32(-R.MAX_F32)), torch.tensor(-R.MAX_BF16).to(t.dtype), t)
    return t.cuda(), t.double().numpy()


def check_grad(got, x, ids, t, temp, up, dtype, rows):
    half_ulp = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -23
    V = x.shape[1]
    for b in rows:
        row = R.allowed_logits(x[b], None, dtype)
        _, _, g = R.distill_row(row, ids[b], t[b], temp)
        z = np.abs(np.where(row > -np.inf, row - row.max(), 0.0)) / temp
        p = np.where(row > -np.inf, R.log_softmax(row / temp)[0], -np.inf)
        p = np.where(p > -700.0, np.exp(np.maximum(p, -700.0)), 0.0)
        q = np.isin(np.arange(V), ids[b])
        scale = abs(float(up[b])) * temp
        arg = np.minimum(z, 700.0)   # beyond it p is nothing
        tol = scale * (p * (rel_sum(V) + (3 * arg + 16) * 2.0 ** -24) + q * (rel_sum(V) + 64 * 2.0 ** -24))
        want = g * float(up[b])
        tol += np.abs(want) * half_ulp + 1e-37
        assert (np.abs(got[b] - want) <= tol).all(), (b, np.abs(got[b] - want).max())


def lists(rng, B, K, V, high):
    ids = np.stack([rng.choice(V, K, replace=False) for _ in range(B)]).astype(np.uint32)
    ids[:, 0] = high[:, 0]
    return ids, rng.normal(0, 2, (B, K)).astype(np.float32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("temp", [0.5, 1.0, 2.5])
def test_autograd_gradient_of_rows_far_from_zero(kind, dtype, temp):
    from grammar_constrained_decoding_gb300 import distill
    V, B, K = 1003, 5, 9
    rng = np.random.default_rng([V, len(kind)])
    xs, high = make(rng, B, V, kind)
    x, v = to_dtype(xs, dtype)
    ids, t = lists(rng, B, K, V, high)
    up = rng.normal(0, 1, B).astype(np.float32)
    x.requires_grad_()
    loss = distill(ctx_of(V), x, u32(ids), f32_dev(t), temp)
    loss.backward(f32_dev(up))
    check_grad(x.grad.double().cpu().numpy(), v, ids, t, temp, up, dtype, range(B))


@pytest.mark.parametrize("V,B,dtype", [(40003, 250, "bf16"), (30011, 180, "f32")])
def test_autograd_gradient_of_many_long_rows_far_from_zero(V, B, dtype):
    """The same through rows that stream."""
    from grammar_constrained_decoding_gb300 import distill
    K, temp = 40, 0.5
    rng = np.random.default_rng(V)
    parts = [make(rng, B // 5, V, kind) for kind in KINDS]
    xs, high = np.concatenate([a for a, _ in parts]), np.concatenate([h for _, h in parts])
    x, v = to_dtype(xs, dtype)
    ids, t = lists(rng, B, K, V, high)
    up = rng.normal(0, 1, B).astype(np.float32)
    x.requires_grad_()
    distill(ctx_of(V), x, u32(ids), f32_dev(t), temp).backward(f32_dev(up))
    check_grad(x.grad.double().cpu().numpy(), v, ids, t, temp, up, dtype, range(0, B, 7))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_loss_and_gradient_where_infinite_logits_share_the_mass(dtype):
    """Three logits of +inf, the teacher's list among them: p is a third each, in
    the loss and in the gradient that is written with it."""
    V, B, K = 515, 4, 3
    import torch
    rng = np.random.default_rng(11)
    xs, high = make(rng, B, V, "inf")
    x, v = to_dtype(xs, dtype)
    t = rng.normal(0, 2, (B, K)).astype(np.float32)
    ids = high.astype(np.uint32)
    loss, up = empty((B,), torch.float32), rng.normal(0, 1, B).astype(np.float32)
    g = torch.full_like(x, float("nan"))
    ctx = ctx_of(V)
    ctx.distill_loss(x, u32(ids), f32_dev(t), loss, temp=1.0, out_grad=g, grad_loss=f32_dev(up))
    assert ctx.status() == 0
    check_grad(g.double().cpu().numpy(), v, ids, t, 1.0, up, dtype, range(B))
    for b in range(B):
        want = R.distill_row(R.allowed_logits(v[b], None, dtype), ids[b], t[b], 1.0)[0]
        # a sum of K terms, each q times a few nats: the roundings of the logarithms and of the sum
        assert abs(float(host(loss)[b]) - want) <= 8 * (rel_sum(V) + (K + 16) * 2.0 ** -24)


def test_kept_normaliser_and_refusals():
    """out_norm holds the maximum and the sum; the backward pass takes one form of it."""
    import torch
    from grammar_constrained_decoding_gb300 import CgError, _lib
    V, B, K = 700, 5, 4
    rng = np.random.default_rng(3)
    x = f32_dev(rng.normal(0, 2, (B, V)))
    mask = torch.zeros((B, (V + 31) // 32), dtype=torch.int32, device="cuda") - 1
    mask[2] = 0
    ids, t = u32(rng.integers(0, V, (B, K))), f32_dev(rng.normal(0, 1, (B, K)))
    ctx = ctx_of(V)
    loss, lse, norm = empty((B,), torch.float32), empty((B,), torch.float32), empty((B, 2), torch.float32)
    for g in (None, torch.empty_like(x)):
        norm.fill_(float("nan"))
        ctx.distill_loss(x, ids, t, loss, temp=1.5, bitmask=mask, out_lse=lse, out_norm=norm, out_grad=g)
        got = host(norm)
        assert ctx.status() == 0 and got[2].tolist() == [-np.inf, 0.0]
        for b in (0, 1, 3, 4):
            v = host(x)[b].astype(np.float64)
            assert got[b, 0] == v.max()
            assert abs(got[b, 1] / np.exp((v - v.max()) / 1.5).sum() - 1) <= rel_sum(V) + 32 * 2.0 ** -24
    alone = torch.empty_like(x)
    ctx.distill_grad(x, ids, t, None, alone, temp=1.5, bitmask=mask, norm=norm)
    assert ctx.status() == 0 and (alone[2] == 0).all() and torch.allclose(alone, g, rtol=0, atol=1.5 * 2.0 ** -20)  # p + q <= 2
    for bad in (dict(lse=None), dict(lse=lse, norm=norm), dict(lse=None, norm=lse), dict(lse=None, norm=norm.T.contiguous())):
        with pytest.raises(CgError) as e:
            ctx.distill_grad(x, ids, t, out_grad=alone, **bad)
        assert e.value.code == _lib.CG_E_ARG
