"""GPU tests of the output layer's values at the ends of their types' ranges."""

import pytest

from tests.rows_ctx import ctx_of
from tests.test_gpu_head import generator, pack

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def contexts_end_with_the_module():
    yield
    ctx_of.cache_clear()


@pytest.mark.parametrize("T", [1.0, 1e34, 3e38])
@pytest.mark.parametrize("B,masked", [(3, False), (3, True), (40, False), (40, True), (200, False), (200, True)])
def test_a_product_that_overflows_counts_as_the_largest_value(B, masked, T):
    """Finite rows whose product with one token's is +inf in 32 bits: it counts as the largest finite value, and
    its gradient's term is g / T p as any other's.  T so large that the exponentials of all tokens are of one size
    (1e34: the maximum's alone is left; 3e38: exp(-1.13) for the others), or 1.  Losses: the exponent is off by
    2^-22 of its size (at most 4e4) where it counts; tolerance 1e-4 of the value.  Terms: rounded to bf16, 2^-8,
    and 1e-4 for what the loss is off."""
    import torch
    V, D = 600, 8
    ctx, g = ctx_of(V), generator(B)
    h = torch.zeros((B, D), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((V, D), dtype=torch.bfloat16, device="cuda")
    h[:, 0], w[77, 0] = 2.0 ** 127, 4.0                    # 2^129
    h[:, 1:] = torch.randn((B, D - 1), generator=g, device="cuda").bfloat16()
    w[:, 1:] = torch.randn((V, D - 1), generator=g, device="cuda").bfloat16()
    target = torch.randint(100, V, (B,), generator=g, device="cuda").int()
    bits = torch.ones((B, V), dtype=torch.bool, device="cuda")
    if masked:
        bits[:, :50] = False
    up = torch.full((B,), T * 0.75, device="cuda")         # g / T = 0.75
    loss, norm = torch.empty(B, device="cuda"), torch.empty((B, 2), device="cuda")
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    mask = pack(bits) if masked else None
    ctx.head_loss(h, w, target, loss, temp=T, bitmask=mask, out_norm=norm)
    ctx.head_grad(h, w, target, loss, norm, dh, dw, temp=T, bitmask=mask, grad_loss=up)
    assert ctx.status() == 0
    big = float(torch.finfo(torch.float32).max)
    x = (h.double() @ w.double().T).clamp(max=big).masked_fill(~bits, -torch.inf)
    p = torch.softmax(x / T, 1)
    at = target.long()[:, None]
    want = torch.logsumexp(x / T, 1) - x.gather(1, at)[:, 0] / T
    assert bool(((loss.double() - want).abs() <= 1e-4 * want).all())
    d = 0.75 * p.scatter_add(1, at, torch.full((B, 1), -1.0, dtype=torch.float64, device="cuda"))
    for got, a, b in ((dw[:, 1:], d.T, h[:, 1:].double()), (dh[:, 1:], d, w[:, 1:].double())):
        size = a.abs() @ b.abs()
        assert bool(((got.double() - a @ b).abs() <= (2.0 ** -7 + 2e-4) * size + 1e-30).all())
    assert bool((dh[:, 0].double() - 0.75 * 4 * p[:, 77]).abs().max() <= (2.0 ** -7 + 2e-4) * 3)
