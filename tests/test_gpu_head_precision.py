"""GPU tests of how many bits the output layer's gradients keep, against the definition in 64 bits.

`once` is the 2-norm of what rounding the exact gradient to bf16 alone leaves: its elements'
significands are spread evenly, so that is a share of 2^-8 / sqrt 3 to 2^-9 / sqrt 3 each.  A second
rounding of the same size, independent of it, would make sqrt 2 = 1.41 of it; 1.3 tells the two apart."""

import pytest

from tests.rows_ctx import ctx_of
from tests.test_gpu_head import Exact, generator, matrix

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def contexts_end_with_the_module():
    yield
    ctx_of.cache_clear()


def gradients(B, V, D, T, up, target, g, pad=0):
    """(exact definition, gradient by the rows, by the weight) of unmasked bf16 rows."""
    import torch
    ctx = ctx_of(V)
    h, w = matrix(B, D, "bf16", pad, 0, g, 1.0), matrix(V, D, "bf16", pad, 0, g, D ** -0.5)
    loss, norm = torch.empty(B, device="cuda"), torch.empty((B, 2), device="cuda")
    dh, dw = torch.empty((B, D), dtype=h.dtype, device="cuda"), torch.empty((V, D), dtype=h.dtype, device="cuda")
    ctx.head_loss(h, w, target, loss, temp=T, out_norm=norm)
    ctx.head_grad(h, w, target, loss, norm, dh, dw, temp=T, grad_loss=up)
    assert ctx.status() == 0
    return Exact(h, w, target, T, None, up.double(), "bf16"), dh, dw


def off_in_roundings(got, want):
    once = float((want.bfloat16().double() - want).norm())
    return float((got.double() - want).norm()) / once


@pytest.mark.parametrize("B", [150, 300, 700])
@pytest.mark.parametrize("first", ["zeros", "no targets", "all but the last"])
def test_the_rows_that_count_set_the_unit(B, first):
    """One g for all rows that count, g / T halfway between two bf16 values; rows that do not count come first: the
    prompt's, weighted with 0, or rows without a target and with another g.  Rounded in a unit that is not g / T's,
    each target's term is off by 2^-8 the same way: 1.9 to 2.5 of one rounding (worked out for these sizes in 64
    bits); in the right one by 1.02, as test_one_gradient_for_all_rows_is_rounded_once has it."""
    import torch
    V, D, T = 4000, 64, 0.85
    g = generator(B)
    target = torch.randint(0, V, (B,), generator=g, device="cuda").int()
    up = torch.full((B,), T * (1 + 2.0 ** -8), device="cuda")
    if first == "zeros":
        up[:40] = 0
    elif first == "no targets":
        target[:3] = -1
        up[:3] = T
    else:
        up[:-20] = 0
    e, dh, dw = gradients(B, V, D, T, up, target, g)
    assert float(e.loss[target >= 0].min()) > 2.4
    assert off_in_roundings(dh, e.d @ e.w) <= 1.3
    assert off_in_roundings(dw, e.d.T @ e.h) <= 1.3


@pytest.mark.parametrize("kind", ["halfway", "random"])
@pytest.mark.parametrize("B,D,pad", [(1, 64, 0), (2, 72, 8), (17, 64, 0), (40, 70, 1), (128, 64, 0)])
def test_few_rows_terms_keep_two_parts(B, D, pad, kind):
    """Up to 128 rows, under a g for each: both gradients as close as one rounding of the result.  `halfway`: each g
    so that its target's term lies halfway between two bf16 values; a term of one part alone would be off by 2^-8
    (1.6 to 2.9 of one rounding for these sizes, worked out in 64 bits; with both parts 1.00)."""
    import torch
    V, T = 4000, 0.85
    g = generator(B)
    target = torch.randint(0, V, (B,), generator=g, device="cuda").int()
    state = g.get_state()
    e, _, _ = gradients(B, V, D, T, torch.ones(B, device="cuda"), target, g, pad)
    if kind == "halfway":
        up = (T * (1 + 2.0 ** -8) / -torch.expm1(-e.loss)).float() * 2.0 ** (torch.arange(B, device="cuda") % 5 - 2)
    else:
        up = torch.rand(B, generator=g, device="cuda") - 0.3
    g.set_state(state)     # the same rows and weight
    e, dh, dw = gradients(B, V, D, T, up, target, g, pad)
    assert float(e.loss.min()) > 1e-2
    assert off_in_roundings(dh, e.d @ e.w) <= 1.3
    assert off_in_roundings(dw, e.d.T @ e.h) <= 1.3
