"""GPU tests of the output layer's cross entropy and its gradients against the
definition in 64 bits.

Tolerances.  A product of two bf16 values is exact in 32 bits.  The tensor cores
add 16 products to a sum at a time, each time to within 2^-22 of the magnitudes
summed so far: a logit of D products is off by at most
    ex = (D / 16 + 2) 2^-22 sum |h w|.
Float matrices are multiplied as three bf16 parts: 2^-22 more a product, and the
five small products' passes add 5 2^-7 of the steps.  Normalisers: exponentials to
2^-21, chains of at most 160 + V / 4096 additions and rescalings of 2^-22.  Every
p is then off by ep = 2 ex / T + 2^-21 + (164 + V / 4096) 2^-22 relative, and so is a
loss near 0; a larger one by the rounding of its own parts besides.

Gradients: each term d is off by ep, and by 2^-8 where it is rounded to bf16 (2^-24
as three parts); sums over K terms add (K / 16 + 2) 2^-22 of their magnitudes, the
sums over pieces and splits 2^-24 each (at most 100 here); the result is rounded once.
An exponential below 2^-126 is zero: the term k exp(..), k <= max |g| / T, is then off by
up to k 2^-126, and a term that is itself below 2^-126 (no longer a normal bf16) by that
much: (1 + max |g| / T) 2^-126 a term, times what it is multiplied with, sum |w| or sum |h|.
"""

import functools

import numpy as np
import pytest

from tests.rows_ctx import ctx_of

pytestmark = pytest.mark.gpu
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def contexts_end_with_the_module():
    yield
    ctx_of.cache_clear()


def generator(seed):
    import torch
    return torch.Generator(device="cuda").manual_seed(seed)


def matrix(rows, D, dtype, pad, shift, g, std):
    import torch
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    flat = torch.full((max(rows, 1) * (D + pad) + shift + 64,), float("nan"), dtype=dt, device="cuda")
    m = flat[shift:shift + rows * (D + pad)].view(rows, D + pad)[:, :D]
    m.copy_(std * torch.randn((rows, D), generator=g, device="cuda"))
    return m


def make_bits(B, V, g):
    """Rows: all, dense, sparse, one token, none, in turn."""
    import torch
    r = torch.arange(B, device="cuda") % 5
    share = torch.tensor([2.0, 0.9, 0.01, -1.0, -1.0], device="cuda")[r]
    bits = torch.rand((B, V), generator=g, device="cuda") < share[:, None]
    one = torch.nonzero(r == 3)[:, 0]
    bits[one, torch.randint(0, V, (one.numel(),), generator=g, device="cuda")] = True
    return bits


def pack(bits):
    import torch
    B, V = bits.shape
    W = (V + 31) // 32
    full = torch.zeros((B, W * 32), dtype=torch.int64, device="cuda")
    full[:, :V] = bits
    w = (full.view(B, W, 32) << torch.arange(32, device="cuda")).sum(2)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32).contiguous()


def make_targets(B, V, bits, g):
    """Allowed ones for most rows that have any; some without a target, some with a forbidden one."""
    import torch
    t = torch.randint(0, V, (B,), generator=g, device="cuda")
    if bits is not None:
        pick = torch.where(bits, torch.rand(bits.shape, generator=g, device="cuda"), -1.0).argmax(1)
        t = torch.where(torch.arange(B, device="cuda") % 7 == 5, t, pick)
    t = torch.where(torch.arange(B, device="cuda") % 11 == 9, -1, t)
    return t.to(torch.int32)


class Exact:
    """The definition in 64 bits, and the bounds above."""

    def __init__(self, h, w, target, T, bits, up, dtype):
        import torch
        h, w = h.double(), w.double()
        (B, D), V = h.shape, w.shape[0]
        steps, f32 = (D / 16 + 2) * 2.0 ** -22, dtype == "f32"
        self.ex = float((h.norm(dim=1).max() * w.norm(dim=1).max())) * (steps * (1 + 5 / 128) + 2.0 ** -22 if f32 else steps)
        x = h @ w.T
        if bits is not None:
            x.masked_fill_(~bits, -torch.inf)
        t = target.long().clamp(min=0)[:, None]
        xt = x.gather(1, t)
        there = (target >= 0)[:, None] & (xt > -torch.inf)
        others = torch.logsumexp(x.scatter(1, t, -torch.inf) / T, 1, keepdim=True)
        gap = torch.where(there, others - xt / T, torch.tensor(-torch.inf, dtype=torch.float64, device="cuda"))
        self.loss = torch.logaddexp(gap, torch.zeros_like(gap))[:, 0]
        self.lse = torch.logsumexp(x / T, 1)
        self.m = x.amax(1)
        self.S = torch.where(self.m > -torch.inf, ((self.lse - self.m / T).exp()), 0.0)
        self.ep = 2 * self.ex / T + 2.0 ** -21 + (164 + V / 4096) * 2.0 ** -22
        size = torch.where(self.m > -torch.inf, self.m.abs(), 0.0) / T
        self.off = 2 * self.ex / T + self.ep + 2.0 ** -22 * (size + 1)      # of a loss or an lse
        d = torch.softmax(x / T, 1).nan_to_num_(0.0)
        d.scatter_(1, t, torch.where(there, torch.expm1(-self.loss)[:, None], d.gather(1, t)))
        self.d = d * (there & (self.loss > 0)[:, None]) * (up / T)[:, None]
        self.h, self.w, self.dtype, self.B, self.V, self.T = h, w, dtype, B, V, T
        self.up, self.there = up, there[:, 0]

    def check_loss(self, loss, lse, norm):
        import torch
        loss, lse, norm = loss.double(), lse.double(), norm.double()
        off = (loss - self.loss).abs()
        assert bool((off <= self.off + self.loss * 2.0 ** -22).all()), float(off.max() / self.off.max())
        near = self.loss < 0.5
        assert bool((off[near] <= self.loss[near] * (self.ep + 2.0 ** -20) + 1e-37).all())
        alive = self.m > -torch.inf
        assert bool((lse[~alive] == -torch.inf).all()) and bool((norm[~alive, 1] == 0).all())
        assert bool(((lse - self.lse).abs() <= self.off)[alive].all())
        assert bool(((norm[:, 0] - self.m).abs() <= self.ex + 2.0 ** -23 * self.m.abs())[alive].all())
        kept = norm[:, 0] / self.T + norm[:, 1].log()
        assert bool(((kept - self.lse).abs() <= self.off)[alive].all())

    def check_grad(self, dh, dw):
        import torch
        term = self.ep + (2.0 ** -8 if self.dtype == "bf16" else 2.0 ** -22) + 2.0 ** -21
        # p is also off where the maximum itself is: counted in ep; expm1 and the scale's roundings: 2^-21
        for got, a, b, K in ((dh, self.d, self.w, self.V), (dw, self.d.T, self.h, self.B)):
            if got is None:
                continue
            want, size = a @ b, a.abs() @ b.abs()
            tiny = (1 + float(self.up.abs().max()) / self.T) * 2.0 ** -126 * b.abs().sum(0)
            bound = size * (term + (K / 16 + 2) * 2.0 ** -22 * 1.05 + 100 * 2.0 ** -24) + HALF[self.dtype] * want.abs() * 1.01 + tiny
            off = (got.double() - want).abs()
            assert bool((off <= bound + 1e-37).all()), float((off / (bound + 1e-37)).max())
            # and on the whole: roundings are independent, half of the bound's 2-norm would be a bias
            norm = float(want.norm())
            if norm:
                # (two roundings of relative size up to 2^-8, evenly spread: 2^-8 / sqrt 3 each at most)
                rms = 2 * 2.0 ** -8 / 3 ** 0.5 + self.ep if self.dtype == "bf16" else self.ep + (K / 16 + 110) * 2.0 ** -22
                assert float((got.double() - want).norm()) <= norm * rms * 2, float((got.double() - want).norm()) / norm


def run(B, V, D, dtype, pad=0, shift=0, masked=True, T=1.0, seed=0, std=2.0, which="both"):
    import torch
    ctx, g = ctx_of(V), generator(seed + B + V + D)
    h, w = matrix(B, D, dtype, pad, shift, g, std), matrix(V, D, dtype, pad, shift, g, D ** -0.5)
    bits = make_bits(B, V, g) if masked else None
    target = make_targets(B, V, bits, g)
    # some rows' targets far above the others: losses near 0
    boost = torch.where(torch.arange(B, device="cuda") % 3 == 0, 16.0, 0.0)[:, None] * w[target.clamp(min=0).long()].float()
    h += (boost / (w[target.clamp(min=0).long()].float().norm(dim=1, keepdim=True) ** 2 + 1e-30)).to(h.dtype)
    up = torch.rand(B, generator=g, device="cuda") - 0.3
    mask = pack(bits) if masked else None
    loss, lse, norm = (torch.full(s, 5.0, device="cuda") for s in ((B,), (B,), (B, 2)))
    ws = torch.full((ctx.head_workspace(h, w),), 255, dtype=torch.uint8, device="cuda")
    ctx.head_loss(h, w, target, loss, temp=T, bitmask=mask, out_lse=lse, out_norm=norm, workspace=ws)
    dt = h.dtype
    flats = [torch.full((n * (D + pad) + shift + 64,), 777.0, dtype=dt, device="cuda") for n in (B, V)]
    dh, dw = (f[shift:shift + n * (D + pad)].view(n, D + pad)[:, :D] for f, n in zip(flats, (B, V)))
    dh, dw = dh if which != "dw" else None, dw if which != "dh" else None
    ws = torch.full((ctx.head_workspace(h, w, grad=True),), 255, dtype=torch.uint8, device="cuda")
    ctx.head_grad(h, w, target, loss, norm, dh, dw, temp=T, bitmask=mask, grad_loss=up, workspace=ws)
    assert ctx.status() == 0
    e = Exact(h, w, target, T, bits, up.double(), dtype)
    e.check_loss(loss, lse, norm)
    e.check_grad(dh, dw)
    for f, m in zip(flats, (dh, dw)):
        keep = torch.ones(f.shape, dtype=torch.bool, device="cuda")
        if m is not None:
            keep.as_strided(m.shape, m.stride(), m.storage_offset()).fill_(False)
        assert bool((f[keep].float() == 776.0).all() if dtype == "bf16" else (f[keep] == 777.0).all())
    return loss, lse, norm, dh, dw


SIZES = [(1, 512, 64), (2, 500, 8), (5, 513, 1), (31, 777, 100), (128, 600, 72), (129, 1000, 64), (256, 512, 256), (257, 4013, 129),
         (300, 32003, 264), (700, 5000, 1000)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,V,D", SIZES)
def test_head_matches_definition(B, V, D, dtype):
    run(B, V, D, dtype)
    run(B, V, D, dtype, masked=False, T=0.7, seed=1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,shift", [(8, 0), (1, 0), (0, 3), (4, 4), (56, 8)])
def test_head_layouts(pad, shift, dtype):
    run(150, 1500, 136, dtype, pad, shift, T=1.5)
    run(60, 1500, 130, dtype, pad, shift, masked=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [1, 3, 7, 65, 129, 130, 135, 191, 193, 257, 261])
def test_head_leaves_what_lies_beside_its_rows(D, dtype):
    """Rows on the 16-byte grid whose last elements do not end there: what follows them stays."""
    pad = -D % (8 if dtype == "bf16" else 4)
    for B in (20, 150):
        run(B, 800, D, dtype, pad, 0)


@pytest.mark.parametrize("which", ["dh", "dw"])
def test_head_one_gradient(which):
    run(200, 3000, 96, "bf16", which=which)


@pytest.mark.parametrize("B,V,D,dtype", [(4096, 40000, 64, "bf16"), (64, 151936, 1001, "bf16"), (2, 128256, 512, "bf16"),
                                         (1500, 32003, 96, "f32"), (1000, 151936, 128, "bf16")])
def test_head_in_several_pieces(B, V, D, dtype):
    """More terms, or more of a weight laid out, than one piece holds; many splits; few rows of a large vocabulary."""
    run(B, V, D, dtype, masked=V < 100000)


@pytest.mark.parametrize("T", [1e-3, 0.05, 50.0])
def test_head_temperatures(T):
    run(70, 1000, 64, "bf16", T=T, std=0.01 if T < 0.01 else 2.0)


@pytest.mark.parametrize("B", [1, 2, 3, 4, 5, 8, 9])
@pytest.mark.parametrize("V,D,pad,shift", [(500, 1, 0, 0), (777, 131, 1, 0), (4013, 516, 0, 3), (4013, 516, 4, 4), (513, 9001, 3, 0), (600, 24580, 0, 0)])
def test_head_few_float_rows(B, V, D, pad, shift):
    """Multiplied without the tensor cores (products in 32 bits, in shorter chains: the bounds above hold), on and
    off the 16-byte grid, in one stretch of the columns and in several."""
    run(B, V, D, "f32", pad, shift, masked=B != 3, T=0.8)
    if B < 3:
        run(B, V, D, "f32", pad, shift, which="dh" if B == 1 else "dw")
