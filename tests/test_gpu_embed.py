"""GPU tests of the embedding lookup and its gradient against 64-bit sums.

Tolerances.  The lookup multiplies in 32 bits and rounds once: equal to the same
product rounded by torch.  A gradient's sum of n rows is a chain of n additions
in 32 bits, whatever the grouping: off by at most n 2^-24 times the sum of
magnitudes, one more rounding for the scale and one for the addition to what is
there, then half a step of the dtype (2^-8 bf16, 2^-24 float).
"""

import numpy as np
import pytest

from tests.rows_ctx import ctx_of

pytestmark = pytest.mark.gpu
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def contexts_end_with_the_module():
    yield
    ctx_of.cache_clear()


def torch_dtype(dtype):
    import torch
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def matrix(rows, D, dtype, pad, shift, g, fill=None):
    """([rows, D] in a buffer of D + pad columns that begins `shift` elements in, the buffer)."""
    import torch
    flat = torch.full((max(rows, 1) * (D + pad) + shift + 64,), 777.0, dtype=torch_dtype(dtype), device="cuda")
    m = flat[shift:shift + rows * (D + pad)].view(rows, D + pad)[:, :D]
    if fill is None:
        m.copy_(torch.randn((rows, D), generator=g, device="cuda"))
    else:
        m.fill_(fill)
    return m, flat


def tokens_of(kind, N, V, rng):
    import torch
    if kind == "zipf":
        t = np.minimum((V * rng.random(N) ** 4).astype(np.int64), V - 1)
    elif kind == "same":
        t = np.full(N, V // 2)
    elif kind == "two":
        t = rng.integers(0, 2, N) * (V - 1)
    elif kind == "none":
        t = np.full(N, -1)
    elif kind == "runs":
        t = np.repeat(rng.permutation(V)[:N // 31 + 1], 31)[:N]
    else:
        t = rng.integers(0, V, N)
    if kind in ("zipf", "uniform"):
        t[rng.random(N) < 0.1] = -1
    return torch.tensor(t.astype(np.int32), device="cuda")


def generator(seed):
    import torch
    return torch.Generator(device="cuda").manual_seed(seed)


def untouched(flat, m):
    """What lies between and around the matrix's rows still holds the fill."""
    import torch
    keep = torch.ones(flat.shape, dtype=torch.bool, device="cuda")
    keep.as_strided(m.shape, m.stride(), m.storage_offset()).fill_(False)
    return bool((flat[keep].float() == torch.tensor(777.0).to(flat.dtype).float()).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,D,pad,shift", [(1, 500, 32, 0, 0), (1, 32000, 4096, 0, 0), (7, 513, 1, 0, 0), (33, 1000, 257, 0, 0),
                                             (256, 4013, 1001, 7, 3), (1000, 512, 100, 4, 4), (5000, 777, 36, 0, 2),
                                             (4097, 32003, 128, 0, 0)])
def test_lookup(N, V, D, pad, shift, dtype):
    import torch
    ctx, g, rng = ctx_of(V), generator(N + D), np.random.default_rng([N, V, D])
    table, _ = matrix(V, D, dtype, pad, shift, g)
    tok = tokens_of("uniform", N, V, rng)
    for scale in (1.0, 0.37):
        out, flat = matrix(N, D, dtype, pad + 1, shift, g, fill=5.0)
        ctx.embed(table, tok, out, scale=scale)
        assert ctx.status() == 0
        want = torch.where((tok >= 0)[:, None], (table[tok.clamp(min=0).long()].float() * np.float32(scale)), 0.0).to(out.dtype)
        assert torch.equal(out, want) and untouched(flat, out)


def check_grad(N, V, D, dtype, kind, pad=0, shift=0, scale=1.0, accumulate=False, seed=0):
    import torch
    ctx, g, rng = ctx_of(V), generator(seed + N), np.random.default_rng([N, V, D, seed])
    grad, _ = matrix(N, D, dtype, pad, shift, g)
    tok = tokens_of(kind, N, V, rng)
    out, flat = matrix(V, D, dtype, pad, shift, g, fill=None if accumulate else float("nan"))
    base = out.double() if accumulate else torch.zeros((V, D), dtype=torch.float64, device="cuda")
    work = torch.full((ctx.embed_workspace(grad, tok),), 255, dtype=torch.uint8, device="cuda")
    ctx.embed_grad(grad, tok, out, scale=scale, accumulate=accumulate, workspace=work)
    assert ctx.status() == 0 and untouched(flat, out)
    there = tok >= 0
    at = tok[there].long()
    total, size = torch.zeros_like(base), torch.zeros_like(base)
    total.index_add_(0, at, grad[there].double())
    size.index_add_(0, at, grad[there].double().abs())
    n = torch.bincount(at, minlength=V).double()[:, None]
    s = float(np.float32(scale))
    want = base + s * total
    bound = (n + 2) * 2.0 ** -24 * (abs(s) * size + base.abs()) + HALF[dtype] * want.abs() * 1.01 + 1e-38
    off = (out.double() - want).abs()
    assert bool((off <= bound).all()), float((off / bound).max())
    if accumulate:   # tokens that do not occur are left as they were, bit for bit
        assert torch.equal(out[n[:, 0] == 0].double(), base[n[:, 0] == 0])
    return out.clone()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,D,kind", [(1, 500, 32, "uniform"), (2, 513, 33, "same"), (31, 512, 64, "same"),
                                        (1000, 4013, 1001, "zipf"), (1025, 600, 40, "two"), (2048, 777, 8, "runs"),
                                        (2049, 32003, 129, "zipf"), (5000, 512, 260, "uniform"), (9000, 70000, 24, "zipf"),
                                        (20000, 4013, 64, "zipf"), (40001, 1000, 16, "same"), (300, 1000, 48, "none")])
def test_gradient(N, V, D, kind, dtype):
    check_grad(N, V, D, dtype, kind)
    check_grad(N, V, D, dtype, kind, accumulate=True, scale=-0.73, seed=1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,shift", [(1, 0), (3, 5), (8, 8), (4, 2), (0, 1)])
def test_gradient_layouts(pad, shift, dtype):
    """Every alignment gives the sums of the widest: the grouping does not go by it."""
    import torch
    a = check_grad(3000, 700, 136, dtype, "zipf", pad, shift, 2.0)
    b = check_grad(3000, 700, 136, dtype, "zipf", 0, 0, 2.0)
    assert torch.equal(a, b)


def test_gradient_of_many_rows():
    """A long run over more than a thousand chunks, and rows of 18 digits of sorting bits."""
    check_grad(200000, 151936, 64, "bf16", "zipf")
    check_grad(131072, 600, 128, "f32", "same")


def test_gradient_is_the_same_every_time():
    import torch
    first = check_grad(6000, 512, 200, "f32", "zipf")
    for _ in range(3):
        assert torch.equal(check_grad(6000, 512, 200, "f32", "zipf"), first)


def test_rows_beyond_32_bit_offsets():
    """A table and a gradient of more than 2^32 bytes: the last rows are found."""
    import torch
    V, D, N = 40000, 32768, 3
    ctx = ctx_of(V)
    table = torch.zeros((V, D), dtype=torch.float32, device="cuda")
    table[-1], table[V // 2] = 3.0, 2.0
    tok = torch.tensor([V - 1, V // 2, V - 1], dtype=torch.int32, device="cuda")
    out = torch.empty((N, D), dtype=torch.float32, device="cuda")
    ctx.embed(table, tok, out)
    assert out[:, 0].tolist() == [3.0, 2.0, 3.0] and out[:, -1].tolist() == [3.0, 2.0, 3.0]
    ctx.embed_grad(out, tok, table)
    assert ctx.status() == 0
    assert table[-1, -1].item() == 6.0 and table[V // 2, 0].item() == 2.0 and float(table.sum(dtype=torch.float64)) == 8.0 * D


def test_bad_tokens_are_recorded_and_count_as_none():
    import torch
    from grammar_constrained_decoding_gb300._lib import CG_DEV_BAD_TOKEN
    V, D = 600, 24
    ctx = ctx_of(V)
    table = torch.randn((V, D), device="cuda")
    tok = torch.tensor([3, V, 5, -2], dtype=torch.int32, device="cuda")
    out = torch.full((4, D), 9.0, device="cuda")
    ctx.embed(table, tok, out, scale=2.0)
    assert ctx.status() == CG_DEV_BAD_TOKEN
    assert torch.equal(out[[0, 2]], 2.0 * table[[3, 5]]) and not out[[1, 3]].any()
    grad = torch.randn((4, D), device="cuda")
    dt = torch.full((V, D), 9.0, device="cuda")
    ctx.embed_grad(grad, tok, dt)
    assert ctx.status() == CG_DEV_BAD_TOKEN and ctx.status() == 0
    want = torch.zeros((V, D), device="cuda")
    want[3], want[5] = grad[0], grad[2]
    assert torch.equal(dt, want)


def test_empty_batch():
    import torch
    V, D = 600, 24
    ctx = ctx_of(V)
    none, tok = torch.empty((0, D), device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    table = torch.ones((V, D), device="cuda")
    ctx.embed(table, tok, none)
    ctx.embed_grad(none, tok, table, accumulate=True)
    assert bool((table == 1).all())
    ctx.embed_grad(none, tok, table)
    assert not table.any() and ctx.status() == 0


def test_refusals():
    import torch
    import grammar_constrained_decoding_gb300 as cg
    V, D, N = 600, 24, 4
    ctx = ctx_of(V)
    table, tok = torch.ones((V, D), device="cuda"), torch.zeros(N, dtype=torch.int32, device="cuda")
    out = torch.full((N, D), 7.0, device="cuda")
    both = torch.ones((V, D + N), device="cuda")
    for args, kw in [((table[1:], tok, out), {}), ((table, tok.long(), out), {}), ((table, tok, out.bfloat16()), {}),
                     ((table, tok, out[:, 1:]), {}), ((table.cpu(), tok, out), {}), ((table, tok[None], out), {}),
                     ((table, tok, out), dict(scale=float("nan"))), ((table, tok, out), dict(scale=float("inf"))),
                     ((table.half(), tok, out.half()), {}), ((table, tok, table[:N]), {}), ((table.t(), tok, out), {}),
                     ((both[:, :D], tok, both[:N, 1:D + 1]), {})]:
        with pytest.raises(cg.CgError):
            ctx.embed(*args, **kw)
    ctx.embed(both[:, :2], tok, both[:N, 2:4])   # other columns of the same buffer
    grad = torch.ones((N, D), device="cuda")
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    big = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    for args, kw in [((grad, tok, table[1:]), {}), ((grad, tok, table.bfloat16()), {}), ((table[:N], tok, table), {}),
                     ((grad, tok, table), dict(workspace=small)), ((grad, tok, table), dict(workspace=big[1:])),
                     ((grad, tok, table), dict(workspace=big.cpu())), ((grad, tok[:2], table), {})]:
        with pytest.raises(cg.CgError):
            ctx.embed_grad(*args, **kw)
    assert bool((out == 7).all()) and bool((table == 1).all()) and ctx.status() == 0
