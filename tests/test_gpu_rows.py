"""GPU parity of the per-row operators (sample_rows, top_logprobs,
distill_loss, distill_grad) against the float64 oracle, at the sizes, masks,
layouts and values where they can go wrong.

Tolerances.  Normalisers are sums of V exponentials in 32 bits, each good to
2^-21 (the exponential's 2^-22 and its argument), added in chains of at most
V / 512 + 32 terms, each addition good to 2^-24; a log-probability adds the
rounding of its own value.  ``rel_sum(V)`` is that bound.  Sampled ids agree
unless the oracle's gap or margin is below 1e-5, as for cg_mask_and_sample.
"""

import functools

import numpy as np
import pytest

from oracle import rows as R
from oracle.step import pack_bitmask
from tests.gpu_helpers import empty, host, u32

pytestmark = pytest.mark.gpu
TIE = 1e-5


def rel_sum(V):
    return 2.0 ** -21 + (V / 512 + 32) * 2.0 ** -24


@functools.lru_cache(maxsize=None)
def ctx_of(V):
    import grammar_constrained_decoding_gb300 as cg
    return cg.Ctx([cg.Grammar.compile('root ::= "a"', "gbnf")], cg.Vocab([i.to_bytes(3, "big") for i in range(V)]))


@pytest.fixture(scope="module", autouse=True)
def contexts_end_with_the_module():
    yield
    ctx_of.cache_clear()


def make_rows(rng, B, V, kind):
    if kind == "flat":
        x = rng.normal(0, 2, (B, V)) + 4.0 * (rng.random((B, V)) < 0.05)
    elif kind == "peaked":
        x = rng.normal(0, 2, (B, V))
        for b in range(B):
            x[b, rng.integers(0, V, min(V, 20))] += 14 * rng.random(min(V, 20))
    elif kind == "equal":
        x = np.full((B, V), -3.25)
    elif kind == "two":
        x = np.where(rng.random((B, V)) < 0.5, 1.0, 0.0)
    elif kind == "wide":
        x = rng.normal(0, 1, (B, V)) * 10.0 ** rng.integers(-30, 30, (B, V))
    elif kind == "negative":
        x = -np.abs(rng.normal(0, 8, (B, V))) - 30
    elif kind == "special":
        x = rng.normal(0, 3, (B, V))
        pick = rng.integers(0, 8, (B, V))
        x[pick == 0] = np.nan
        x[pick == 1] = -np.inf
        for b in range(0, B, 2):
            x[b, rng.integers(0, V, 3)] = np.inf
        x[B - 1] = -np.inf
    return x.astype(np.float32)


def make_mask(rng, B, V):
    """Rows: all, dense, sparse, one token, none, in turn."""
    m = np.zeros((B, V), dtype=bool)
    for b in range(B):
        m[b] = (True, rng.random(V) < 0.9, rng.random(V) < 0.01, np.arange(V) == rng.integers(V), False)[b % 5]
    return m


def to_dev(x, dtype, pad=0, shift=0):
    """([B, V] device rows with the given row padding and start offset, the values kept as float64)."""
    import torch
    B, V = x.shape
    t = torch.from_numpy(x)
    t = t.to(torch.bfloat16) if dtype == "bf16" else t
    flat = torch.full((B * (V + pad) + shift + 64,), float("nan"), dtype=t.dtype, device="cuda")
    rows = flat[shift:shift + B * (V + pad)].view(B, V + pad)[:, :V]
    rows.copy_(t)
    return rows, t.to(torch.float64).numpy()


def words(mask):
    return None if mask is None else u32(np.stack([pack_bitmask(m) for m in mask]))


def f32(a):
    import torch
    return torch.tensor(np.asarray(a, dtype=np.float32), device="cuda")


SETTINGS = [(0.7, 50, 0.9, 0.0), (0.0, 0, 1.0, 0.0), (1.0, 0, 0.95, 0.0), (1.0, 0, 1.0, 0.05), (0.8, 40, 1.0, 0.02),
            (1.0, 0, 1.0, 0.0), (2.0, 0, 0.999, 0.0), (1.3, 1, 0.5, 0.0), (0.05, 1000, 0.5, 0.0),
            (1.0, 3000, 1.0, 0.0), (5.0, 2000, 0.98, 0.001), (1.0, 0, 0.0, 0.0), (1.0, 0, 1.0, 1.0),
            (1e-3, 0, 0.9, 0.0), (50.0, 0, 0.9, 0.0), (1.0, 10 ** 9, 2.0, 0.0)]


def check_sample(V, dtype, kind, masked, B=20, pad=0, shift=0, seed=0, u_of=None, settings=SETTINGS):
    import torch
    rng = np.random.default_rng([V, seed, len(kind)])
    x, v = to_dev(make_rows(rng, B, V, kind), dtype, pad, shift)
    mask = make_mask(rng, B, V) if masked else None
    s = [settings[b % len(settings)] for b in range(B)]
    u = rng.random((B, V)).astype(np.float32) if u_of is None else u_of(rng, B, V)
    tok, lp = empty((B,), torch.int32), empty((B,), torch.float32)
    ctx = ctx_of(V)
    ctx.sample_rows(x, f32(u), tok, bitmask=words(mask), temp=f32([a[0] for a in s]),
                    top_k=u32([a[1] for a in s]), top_p=f32([a[2] for a in s]), min_p=f32([a[3] for a in s]),
                    out_logprob=lp)
    assert ctx.status() == 0
    g_tok, g_lp = host(tok).view(np.uint32), host(lp).astype(np.float64)
    close = 0
    for b in range(B):
        row = R.allowed_logits(v[b], None if mask is None else mask[b], dtype)
        T, k, p, mp = (np.float32(s[b][0]), s[b][1], np.float32(s[b][2]), np.float32(s[b][3]))
        want = R.sample_rows_row(row, float(T), k, float(p), float(mp), u[b])
        tie = TIE * max(1.0, abs(want.logprob) if np.isfinite(want.logprob) else 1.0)
        if g_tok[b] != want.tok:
            assert want.gap < tie or want.margin < tie, (b, s[b], int(g_tok[b]), want)
            close += 1
            continue
        if want.tok == R.NO_TOKEN:
            assert g_lp[b] == -np.inf
        elif abs(want.logprob) < 1e30:
            assert abs(g_lp[b] - want.logprob) <= rel_sum(V) + abs(want.logprob) * 2.0 ** -21, (b, g_lp[b], want)
    assert close <= B // 4


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 7, 33, 512, 4013, 32003, 128256])
def test_sample_rows_matches_oracle(V, dtype):
    check_sample(V, dtype, "flat", True)
    check_sample(V, dtype, "peaked", False, seed=1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["equal", "two", "wide", "negative", "special"])
def test_sample_rows_on_hard_values(kind, dtype):
    for V in (97, 5003, 40000):
        check_sample(V, dtype, kind, kind != "special")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,shift", [(0, 0), (1, 0), (3, 1), (8, 5), (0, 7), (13, 8)])
def test_sample_rows_layouts(pad, shift, dtype):
    check_sample(8192, dtype, "flat", True, pad=pad, shift=shift)
    check_sample(8191, dtype, "peaked", True, pad=pad, shift=shift)


def test_sample_rows_few_and_many_rows():
    check_sample(32000, "bf16", "peaked", False, B=1)
    check_sample(2048, "bf16", "flat", True, B=700)
    check_sample(151936, "f32", "flat", True, B=5)
    check_sample(262149, "bf16", "flat", True, B=6)
    check_sample(262149, "f32", "peaked", False, B=4)


def test_sample_rows_extreme_random_numbers():
    """0, 1, NaN and values outside [0, 1] are clamped: the draw still lands in the kept set."""
    def u_of(rng, B, V):
        u = rng.choice(np.array([0.0, 1.0, np.nan, -1.0, 2.0, 0.5], dtype=np.float32), (B, V))
        return u.astype(np.float32)
    check_sample(3001, "bf16", "flat", True, u_of=u_of)


def test_sample_rows_shared_numbers_and_defaults():
    """One row of numbers for the batch, all settings left out; the same call
    with the row repeated gives the same tokens."""
    import torch
    B, V = 6, 5000
    rng = np.random.default_rng(4)
    x, v = to_dev(make_rows(rng, B, V, "peaked"), "bf16")
    u = rng.random((1, V)).astype(np.float32)
    ctx = ctx_of(V)
    a, b, c = (empty((B,), torch.int32) for _ in range(3))
    ctx.sample_rows(x, f32(u), a)
    ctx.sample_rows(x, f32(np.repeat(u, B, 0)), b)
    ctx.sample_rows(x, f32(u).expand(B, V), c)
    want = [R.sample_rows_row(R.allowed_logits(r, None, "bf16"), 1.0, 0, 1.0, 0.0, u[0]) for r in v]
    assert host(a).tolist() == host(b).tolist() == host(c).tolist()
    assert all(int(t) == w.tok or w.gap < TIE for t, w in zip(host(a), want))


def test_sample_rows_bad_settings_are_recorded():
    import torch
    V = 100
    ctx = ctx_of(V)
    x, _ = to_dev(np.zeros((6, V), dtype=np.float32), "f32")
    u, tok, lp = f32(np.full((6, V), 0.5)), empty((6,), torch.int32), empty((6,), torch.float32)
    nan, inf = float("nan"), float("inf")
    for kw in (dict(temp=f32([1, -1, 1, 1, 1, 1])), dict(temp=f32([1, nan, 1, 1, 1, 1])),
               dict(temp=f32([1, inf, 1, 1, 1, 1])), dict(top_p=f32([1, nan, 1, 1, 1, 1])),
               dict(min_p=f32([0, nan, 0, 0, 0, 0]))):
        ctx.sample_rows(x, u, tok, out_logprob=lp, **kw)
        assert ctx.status() == 10                                 # CG_DEV_BAD_PARAM
        got = host(tok)
        assert got[1] == -1 and host(lp)[1] == -np.inf and (got[[0, 2, 3, 4, 5]] == 0).all()
    ctx.sample_rows(x, None, tok, temp=f32([0] * 6))
    assert ctx.status() == 0 and (host(tok) == 0).all()
    ctx.sample_rows(x, None, tok, temp=f32([0, 0, 1, 0, 0, 0]))
    assert ctx.status() == 10 and host(tok)[2] == -1


def check_top(V, dtype, kind, masked, n, B=20, pad=0, shift=0):
    import torch
    rng = np.random.default_rng([V, n, len(kind)])
    x, v = to_dev(make_rows(rng, B, V, kind), dtype, pad, shift)
    mask = make_mask(rng, B, V) if masked else None
    ids, lps, lse = empty((B, n), torch.int32), empty((B, n), torch.float32), empty((B,), torch.float32)
    ctx = ctx_of(V)
    ctx.top_logprobs(x, ids, lps, bitmask=words(mask), out_lse=lse)
    assert ctx.status() == 0
    g_ids, g_lps, g_lse = host(ids).view(np.uint32), host(lps).astype(np.float64), host(lse).astype(np.float64)
    for b in range(B):
        row = R.allowed_logits(v[b], None if mask is None else mask[b], dtype)
        w_ids, w_lps, w_lse = R.top_logprobs_row(row, n)
        assert np.array_equal(g_ids[b], w_ids), b
        there = w_ids != R.NO_TOKEN
        assert (g_lps[b][~there] == -np.inf).all()
        if np.abs(w_lse) < 1e30:
            assert (np.abs(g_lps[b][there] - w_lps[there]) <= rel_sum(V) + np.abs(w_lps[there]) * 2.0 ** -21).all(), b
            assert abs(g_lse[b] - w_lse) <= rel_sum(V) + abs(w_lse) * 2.0 ** -22, b
        elif w_lse == -np.inf:
            assert g_lse[b] == -np.inf


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,n", [(1, 1), (7, 9), (513, 5), (4013, 64), (32003, 20), (32003, 1024), (128256, 128),
                                 (600, 600), (1024, 1024)])
def test_top_logprobs_matches_oracle(V, n, dtype):
    check_top(V, dtype, "flat", True, n)
    check_top(V, dtype, "peaked", False, n, pad=3, shift=1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["equal", "two", "wide", "negative", "special"])
def test_top_logprobs_on_hard_values(kind, dtype):
    check_top(97, dtype, kind, True, 40)
    check_top(50000, dtype, kind, True, 300)
    check_top(20011, dtype, kind, False, 1000)


def test_top_logprobs_few_and_many_rows():
    check_top(128256, "bf16", "peaked", True, 20, B=1)
    check_top(151936, "f32", "flat", True, 64, B=5)
    check_top(262149, "bf16", "flat", True, 1000, B=5)
    check_top(1000, "bf16", "flat", True, 30, B=900)


def teacher_list(rng, B, V, K, repeat):
    """Ids and logits of B lists: some entries unlisted, some ids twice, some logits not numbers."""
    ids = rng.integers(0, V, (B, K)).astype(np.uint32)
    if not repeat:
        for b in range(B):
            ids[b, :min(K, V)] = rng.permutation(V)[:K]
            ids[b, min(K, V):] = R.NO_TOKEN
    t = rng.normal(0, 3, (B, K)).astype(np.float32)
    ids[rng.random((B, K)) < 0.1] = R.NO_TOKEN
    t[rng.random((B, K)) < 0.03] = -np.inf
    t[rng.random((B, K)) < 0.03] = np.nan
    ids[B - 1] = R.NO_TOKEN
    if B > 2:
        t[B - 2] = -np.inf
    return ids, t


def check_distill(V, dtype, kind, masked, K, temp, B=12, pad=0, shift=0, gpad=0, gshift=0, inplace=False, repeat=False):
    import torch
    rng = np.random.default_rng([V, K, B, len(kind)])
    x, v = to_dev(make_rows(rng, B, V, kind), dtype, pad, shift)
    mask = make_mask(rng, B, V) if masked else None
    ids, t = teacher_list(rng, B, V, K, repeat)
    up = rng.normal(0, 1, B).astype(np.float32)
    ctx = ctx_of(V)
    args = dict(temp=temp, bitmask=words(mask))
    d_ids, d_t = u32(ids), f32(t)
    loss, lse, loss2 = (empty((B,), torch.float32) for _ in range(3))
    ctx.distill_loss(x, d_ids, d_t, loss, out_lse=lse, **args)
    new = lambda: to_dev(np.full((B, V), np.nan, dtype=np.float32), dtype, gpad, gshift)[0]  # noqa: E731
    back = new()
    ctx.distill_grad(x, d_ids, d_t, lse, back, grad_loss=f32(up), **args)
    both = x if inplace else new()
    ctx.distill_loss(x, d_ids, d_t, loss2, out_grad=both, grad_loss=f32(up), **args)
    assert ctx.status() == 0
    g_loss, g_lse = np.stack([host(loss), host(loss2)]).astype(np.float64), host(lse).astype(np.float64)
    T = float(np.float32(temp))
    for b in range(B):
        row = R.allowed_logits(v[b], None if mask is None else mask[b], dtype)
        w_loss, w_lse, w_grad = R.distill_row(row, ids[b], t[b], T)
        if w_lse == -np.inf:
            assert g_lse[b] == -np.inf and (g_loss[:, b] == 0.0).all()
        elif np.abs(w_lse) < 1e6:
            assert abs(g_lse[b] - w_lse) <= rel_sum(V) + abs(w_lse) * 2.0 ** -22, b
            # the largest term of the sum bounds what its roundings add
            live = [i for i in ids[b] if i < V and row[i] > -np.inf]
            big = max([abs(row[i] / T - w_lse) for i in live], default=0.0) + 8 * abs(np.nan_to_num(t[b], neginf=0)).max() / T
            tol = T * T * (rel_sum(V) + (K + 16) * 2.0 ** -24 + big * 2.0 ** -20)
            assert (np.abs(g_loss[:, b] - w_loss) <= tol).all(), (b, g_loss[:, b], w_loss)
        scale = T * float(up[b])
        half_ulp = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -23
        for name, g, rel in (("fused", both, rel_sum(V)),
                             ("alone", back, rel_sum(V) + (abs(w_lse) + 1) * 2.0 ** -20 if np.isfinite(w_lse) else 0.0)):
            got = g[b].double().cpu().numpy()
            part = np.abs(w_grad / T) + np.isin(np.arange(V), ids[b])   # p + q bounds
            tol = np.abs(scale * w_grad / T) * half_ulp + abs(scale) * part * (rel + 64 * 2.0 ** -24) + 1e-37
            if np.abs(w_lse) < 1e6 or not np.isfinite(w_lse):
                assert (np.abs(got - scale * w_grad / T) <= tol).all(), (name, b, np.abs(got - scale * w_grad / T).max())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,K", [(1, 1), (7, 3), (33, 40), (4013, 64), (32003, 50), (128256, 64), (9000, 1024)])
def test_distill_matches_oracle(V, K, dtype):
    check_distill(V, dtype, "flat", True, K, 2.0)
    check_distill(V, dtype, "peaked", False, K, 0.7, repeat=V > 64)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["equal", "two", "negative", "special"])
def test_distill_on_hard_values(kind, dtype):
    check_distill(97, dtype, kind, True, 20, 1.0, repeat=True)
    check_distill(20011, dtype, kind, True, 33, 1.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,shift,gpad,gshift", [(0, 0, 0, 0), (1, 0, 0, 0), (3, 1, 3, 1), (8, 5, 2, 0), (0, 7, 0, 3)])
def test_distill_layouts(pad, shift, gpad, gshift, dtype):
    check_distill(8191, dtype, "flat", True, 17, 1.0, pad=pad, shift=shift, gpad=gpad, gshift=gshift)
    check_distill(4096, dtype, "flat", False, 17, 1.0, pad=pad, shift=shift, inplace=True)


def test_distill_few_and_many_rows():
    check_distill(128256, "bf16", "flat", False, 64, 1.0, B=1)
    check_distill(151936, "f32", "flat", True, 8, 1.0, B=5)
    check_distill(262149, "bf16", "flat", True, 32, 1.0, B=5)
    check_distill(515, "bf16", "flat", True, 8, 1.0, B=600)


@pytest.mark.parametrize("B,V,dtype,masked,K,pad", [
    (1500, 1003, "f32", True, 1024, 0),       # rows of a block in turn, a list longer than the row
    (700, 9001, "bf16", True, 33, 3),         # ... off the 16-byte grid, the mask's bytes one by one
    (400, 65536, "bf16", True, 64, 64),       # the mask by copies
    (140, 40000, "f32", False, 5, 0),         # two blocks a row
    (70, 100003, "bf16", True, 700, 5),       # four
    (9, 262149, "bf16", False, 64, 0),        # eight
])
def test_distill_loss_alone_over_many_rows(B, V, dtype, masked, K, pad):
    """The loss without a gradient streams rows through each cluster in turn."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(B)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = torch.full((B, V + pad), float("nan"), dtype=dt, device="cuda")[:, :V]
    x.copy_(torch.randn((B, V), generator=g, device="cuda") * 3)
    x[::7, ::5] = float("nan")
    x[::5, 3] = float("-inf")
    mask, xd = None, torch.where(torch.isnan(x), -np.inf, x.double())
    if masked:
        mask = torch.randint(-2 ** 31, 2 ** 31, (B, (V + 31) // 32), generator=g, device="cuda").to(torch.int32)
        mask[B // 2] = 0
        at = torch.arange(V, device="cuda")
        xd = torch.where(((mask[:, at >> 5] >> (at & 31).int()) & 1).bool(), xd, -np.inf)
    ids = torch.randint(0, V, (B, K), generator=g, device="cuda").int()
    t = torch.randn((B, K), generator=g, device="cuda") * 2
    ids[::3, K // 2] = -1
    loss, lse = torch.empty(B, device="cuda"), torch.empty(B, device="cuda")
    torch.cuda.synchronize()
    ctx = ctx_of(V)
    ctx.distill_loss(x, ids, t, loss, bitmask=mask, out_lse=lse, temp=1.25)
    assert ctx.status() == 0
    torch.cuda.synchronize()
    w_lse = torch.logsumexp(xd / 1.25, 1)
    xl = torch.where(ids >= 0, xd.gather(1, ids.clamp_min(0).long()), -np.inf)
    q = torch.softmax(torch.where(xl > -np.inf, t.double(), -np.inf) / 1.25, 1)       # NaN where none is listed
    log_q = torch.log_softmax(torch.where(xl > -np.inf, t.double(), -np.inf) / 1.25, 1)
    w_loss = 1.25 ** 2 * torch.where(q > 0, q * (log_q - (xl / 1.25 - w_lse[:, None])), 0.0).sum(1)
    live = w_lse > -np.inf
    assert torch.equal(lse == -np.inf, ~live) and (loss[~live] == 0).all()
    assert (torch.abs(lse - w_lse)[live] <= rel_sum(V) + w_lse[live].abs() * 2.0 ** -22).all()
    # terms up to 40 nats, each good to 2^-21 of its size
    assert (torch.abs(loss - w_loss)[live] <= 1.25 ** 2 * (rel_sum(V) + (K + 16) * 2.0 ** -24 + 40 * 2.0 ** -20)).all()


@pytest.mark.parametrize("B,V,dtype,masked,K,pad,inplace", [
    (1500, 1003, "f32", True, 1024, 0, False),
    (1500, 1003, "bf16", False, 64, 2, True),
    (700, 40001, "bf16", True, 33, 0, False),
    (420, 65536, "bf16", True, 64, 64, True),
    (400, 200000, "bf16", False, 300, 0, False),
    (300, 70003, "f32", True, 1024, 3, True),
    (150, 40960, "f32", True, 20, 0, False),
])
def test_distill_gradient_over_many_rows(B, V, dtype, masked, K, pad, inplace):
    """Each cluster takes several rows in turn: the gradient with the loss and alone."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(B)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = torch.full((B, V + pad), float("nan"), dtype=dt, device="cuda")[:, :V]
    x.copy_(torch.randn((B, V), generator=g, device="cuda") * 2)
    x[::5, 3] = float("-inf")
    mask = None
    if masked:
        mask = torch.randint(-2 ** 31, 2 ** 31, (B, (V + 31) // 32), generator=g, device="cuda").to(torch.int32)
        mask[B // 2] = 0
    ids = torch.randint(0, V, (B, K), generator=g, device="cuda").int()
    t = torch.randn((B, K), generator=g, device="cuda") * 2
    ids[::3, K // 2] = -1
    ids[1] = -1
    up = torch.randn(B, generator=g, device="cuda")
    loss, lse = torch.empty(B, device="cuda"), torch.empty(B, device="cuda")
    ctx, src, grads = ctx_of(V), x.clone(), []
    for alone in (False, True):
        here = src.clone() if inplace else x
        dx = here if inplace else torch.full((B, V + pad), float("nan"), dtype=dt, device="cuda")[:, :V]
        if alone:
            ctx.distill_grad(here, ids, t, lse, dx, temp=1.25, bitmask=mask, grad_loss=up)
        else:
            ctx.distill_loss(here, ids, t, loss, temp=1.25, bitmask=mask, out_lse=lse, out_grad=dx, grad_loss=up)
        grads.append(dx)
    assert ctx.status() == 0
    half_ulp = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -23
    for lo in range(0, B, 200):
        rows = slice(lo, min(lo + 200, B))
        xd = src[rows].double()
        if masked:
            at = torch.arange(V, device="cuda")
            xd = torch.where(((mask[rows][:, at >> 5] >> (at & 31).int()) & 1).bool(), xd, -np.inf)
        p = torch.nan_to_num(torch.softmax(xd / 1.25, 1))
        i = ids[rows]
        xl = torch.where(i >= 0, xd.gather(1, i.clamp_min(0).long()), -np.inf)
        q = torch.nan_to_num(torch.softmax(torch.where(xl > -np.inf, t[rows].double(), -np.inf) / 1.25, 1))
        any_listed = (xl > -np.inf).any(1, keepdim=True)
        q_v = torch.zeros_like(xd).scatter_add_(1, i.clamp_min(0).long(), torch.where(i >= 0, q, 0.0))
        scale = 1.25 * up[rows].double()[:, None]
        want = torch.where(any_listed, scale * (p - q_v), 0.0)
        w_lse = torch.logsumexp(xd / 1.25, 1, keepdim=True).nan_to_num(neginf=0.0)
        tol = want.abs() * half_ulp + scale.abs() * (p + q_v) * (rel_sum(V) + (w_lse.abs() + 1) * 2.0 ** -20 + 64 * 2.0 ** -24) + 1e-37
        for dx in grads:
            assert ((dx[rows].double() - want).abs() <= tol).all(), (lo, (dx[rows].double() - want).abs().max())


def test_distill_gradient_against_differences():
    """Autograd through distill() on float logits against central differences of
    the 64-bit loss (step 1e-4: truncation about 1e-8; the kernel's 32 bits give
    the 2e-6)."""
    import torch
    from grammar_constrained_decoding_gb300 import distill
    V, B, K, temp = 61, 4, 9, 1.5
    rng = np.random.default_rng(8)
    xs = rng.normal(0, 1.5, (B, V)).astype(np.float32)
    mask = make_mask(rng, B, V)
    ids, t = teacher_list(rng, B, V, K, True)
    x = torch.tensor(xs, device="cuda", requires_grad=True)
    w = rng.normal(0, 1, B).astype(np.float32)
    loss = distill(ctx_of(V), x, u32(ids), f32(t), temp, words(mask))
    (loss * f32(w)).sum().backward()
    got = x.grad.double().cpu().numpy()

    def total(a):
        return sum(float(w[b]) * R.distill_row(R.allowed_logits(a[b], mask[b], "f32"), ids[b], t[b], temp)[0]
                   for b in range(B))

    for b in range(B):
        for i in range(V):
            hi, lo = xs.astype(np.float64), xs.astype(np.float64)
            hi[b, i] += 1e-4
            lo[b, i] -= 1e-4
            assert abs((total(hi) - total(lo)) / 2e-4 - got[b, i]) < 2e-6, (b, i)


def test_distill_autograd_on_another_stream():
    """Inputs made and gradients used on a stream that is not the context's."""
    import torch
    from grammar_constrained_decoding_gb300 import distill
    V, B, K = 32003, 64, 16
    rng = np.random.default_rng(3)
    ids, t = teacher_list(rng, B, V, K, False)
    d_ids, d_t = u32(ids), f32(t)
    base = torch.randn(B, V, device="cuda")
    ctx = ctx_of(V)

    def both():
        x = (base * 2.0).requires_grad_()
        loss = distill(ctx, x, d_ids, d_t, 1.0)
        loss.sum().backward()
        return loss.detach().clone(), x.grad.clone()

    want = both()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [both() for _ in range(5)]
    torch.cuda.synchronize()
    for l, g in got:
        assert torch.equal(l, want[0]) and torch.equal(g, want[1])


def test_distill_bad_id_is_recorded():
    import torch
    V = 50
    ctx = ctx_of(V)
    x, v = to_dev(np.random.default_rng(0).normal(0, 1, (1, V)).astype(np.float32), "f32")
    loss = empty((1,), torch.float32)
    ctx.distill_loss(x, u32([[3, 50]]), f32([[0.0, 0.0]]), loss)
    assert ctx.status() == 2                                      # CG_DEV_BAD_TOKEN
    want = R.distill_row(v[0], np.array([3, R.NO_TOKEN]), np.zeros(2), 1.0)[0]
    assert abs(float(host(loss)[0]) - want) < 1e-5


def test_sample_rows_numbers_against_the_logits():
    """Random numbers that rank the tokens almost against their logits: the best
    scored tokens lie outside the nucleus one after another."""
    def u_of(rng, B, V):
        x = make_rows(np.random.default_rng([V, 0, 4]), B, V, "flat").astype(np.float64)
        score = -1.3 * x + 1e-3 * rng.random((B, V))           # wanted Gumbel part
        score += 6.0 - score.max(axis=1, keepdims=True)
        return np.exp(-np.exp(-np.maximum(score, -3.0))).astype(np.float32)
    settings = [(1.0, 0, 0.5, 0.0), (1.0, 0, 0.9, 0.0), (0.7, 0, 0.05, 0.0), (1.0, 0, 0.7, 0.01)]
    for V, dtype in ((4013, "f32"), (50000, "bf16"), (128256, "bf16")):
        check_sample(V, dtype, "flat", False, B=8, u_of=u_of, settings=settings)


def test_sample_rows_captured_in_a_graph():
    """The calls allocate nothing and may be captured: replays see new inputs."""
    import torch
    from grammar_constrained_decoding_gb300 import Ctx, Grammar, Vocab
    V, B, n = 5000, 9, 12
    side = torch.cuda.Stream()
    ctx = Ctx([Grammar.compile('root ::= "a"', "gbnf")], Vocab([i.to_bytes(3, "big") for i in range(V)]), side)
    rng = np.random.default_rng(0)
    x, _ = to_dev(make_rows(rng, B, V, "flat"), "bf16")
    u, tok, top_p = f32(rng.random((B, V))), empty((B,), torch.int32), f32([0.9] * B)
    ids, lps = empty((B, n), torch.int32), empty((B, n), torch.float32)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        ctx.sample_rows(x, u, tok, top_p=top_p)
        ctx.top_logprobs(x, ids, lps)
    for seed in (1, 2):
        new, v = to_dev(make_rows(np.random.default_rng(seed), B, V, "flat"), "bf16")
        x.copy_(new)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for b in range(B):
            row = R.allowed_logits(v[b], None, "bf16")
            want = R.sample_rows_row(row, 1.0, 0, float(np.float32(0.9)), 0.0, host(u)[b])
            assert int(host(tok)[b]) == want.tok or want.gap < TIE or want.margin < TIE
            assert host(ids).view(np.uint32)[b].tolist() == R.top_logprobs_row(row, n)[0].tolist()


def test_rows_beyond_32_bit_offsets():
    """A row stride that takes the last row past 2^32 elements, logits and random
    numbers and gradient alike."""
    import torch
    V, B, K, ld = 3001, 3, 7, 2 ** 31 + 24
    rng = np.random.default_rng(1)
    xs = make_rows(rng, B, V, "peaked")
    flat = torch.empty((B - 1) * ld + V, dtype=torch.bfloat16, device="cuda")
    x = flat.as_strided((B, V), (ld, 1))
    x.copy_(torch.from_numpy(xs))
    v = x.double().cpu().numpy()
    ids, t = teacher_list(rng, B, V, K, False)
    ctx, u = ctx_of(V), rng.random((B, V)).astype(np.float32)
    tok, best, lps, loss = empty((B,), torch.int32), empty((B, 5), torch.int32), empty((B, 5), torch.float32), empty((B,), torch.float32)
    ctx.sample_rows(x, f32(u), tok)
    ctx.top_logprobs(x, best, lps)
    ctx.distill_loss(x, u32(ids), f32(t), loss, out_grad=x)       # the gradient over the logits
    assert ctx.status() == 0
    for b in range(B):
        row = R.allowed_logits(v[b], None, "bf16")
        want = R.sample_rows_row(row, 1.0, 0, 1.0, 0.0, u[b])
        assert int(host(tok)[b]) == want.tok or want.gap < TIE
        assert host(best).view(np.uint32)[b].tolist() == R.top_logprobs_row(row, 5)[0].tolist()
        w_loss, _, w_grad = R.distill_row(row, ids[b], t[b], 1.0)
        assert abs(float(host(loss)[b]) - w_loss) <= 1e-4 * max(1.0, w_loss)
        assert np.abs(x[b].double().cpu().numpy() - w_grad).max() <= 2.0 ** -8


def test_longest_rows():
    """Float rows as long as a context's vocabulary may be, off the 16-byte grid and masked."""
    V = 388005
    check_sample(V, "f32", "flat", True, B=2, settings=[(0.7, 0, 0.9, 0.0), (1.0, 50, 0.9, 0.0)], pad=1, shift=1)
    check_distill(V, "f32", "flat", True, 8, 1.0, B=3, pad=1, shift=1)


def test_example_runs_them_together():
    """examples/grammar_distill.py: generation under a grammar, the record, and a
    student that learns from it."""
    from examples.grammar_distill import main
    first, final = main(rows=32, steps=12, n_best=12, epochs=25, verbose=False)
    assert 0.0 <= final < 0.5 * first


@pytest.mark.parametrize("V,dtype,B", [(200000, "bf16", 400), (70003, "f32", 300)])
def test_streamed_rows_give_the_same_bits_every_time(V, dtype, B):
    """Many rows through each ring, under the load of the gradient's stores: no chunk is
    replaced before it has been read."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(V)
    x = (torch.randn((B, V), generator=g, device="cuda") * 2).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    ids = torch.randint(0, V, (B, 300), generator=g, device="cuda").int()
    t = torch.randn((B, 300), generator=g, device="cuda")
    ctx, first = ctx_of(V), None
    for _ in range(40):
        loss, loss2, lse = (torch.empty(B, device="cuda") for _ in range(3))
        both, alone = torch.empty_like(x), torch.empty_like(x)
        ctx.distill_loss(x, ids, t, loss, out_lse=lse)
        ctx.distill_loss(x, ids, t, loss2, out_grad=both)
        ctx.distill_grad(x, ids, t, lse, alone)
        got = [loss, lse, loss2, both, alone]
        if first is None:
            first = got
        assert all(torch.equal(a, b) for a, b in zip(got, first))
    assert ctx.status() == 0


def test_repeated_calls_give_the_same_bits():
    import torch
    V, B = 128256, 12
    rng = np.random.default_rng(6)
    x, _ = to_dev(make_rows(rng, B, V, "flat"), "bf16")
    u = f32(rng.random((B, V)))
    temp, top_p = f32([0.9] * B), f32([0.97] * B)
    ids, t = teacher_list(rng, B, V, 64, True)
    ctx, seen = ctx_of(V), set()
    for _ in range(4):
        tok, lp, loss = empty((B,), torch.int32), empty((B,), torch.float32), empty((B,), torch.float32)
        bi, bl = empty((B, 300), torch.int32), empty((B, 300), torch.float32)
        g = torch.empty((B, V), dtype=torch.bfloat16, device="cuda")
        ctx.sample_rows(x, u, tok, temp=temp, top_p=top_p, out_logprob=lp)
        ctx.top_logprobs(x, bi, bl)
        ctx.distill_loss(x, u32(ids), f32(t), loss, out_grad=g)
        seen.add(b"".join(host(a.view(torch.int16) if a.dtype == torch.bfloat16 else a).tobytes()
                          for a in (tok, lp, loss, bi, bl, g)))
    assert len(seen) == 1


def test_empty_batch_and_refusals():
    import torch
    from grammar_constrained_decoding_gb300 import CgError, _lib
    V = 100
    ctx = ctx_of(V)
    z = torch.empty((0, V), device="cuda")
    zi, zf, zl = (torch.empty((0,), dtype=d, device="cuda") for d in (torch.int32, torch.float32, torch.float32))
    k0, t0 = torch.empty((0, 4), dtype=torch.int32, device="cuda"), torch.empty((0, 4), device="cuda")
    ctx.sample_rows(z, z, zi)
    ctx.top_logprobs(z, k0, t0)
    ctx.distill_loss(z, k0, t0, zl)
    ctx.distill_grad(z, k0, t0, zf, torch.empty((0, V), device="cuda"))
    assert ctx.status() == 0

    B = 3
    x, u, tok = torch.zeros((B, V), device="cuda"), torch.full((B, V), 0.5, device="cuda"), empty((B,), torch.int32)
    ids, t, f = torch.zeros((B, 4), dtype=torch.int32, device="cuda"), torch.zeros((B, 4), device="cuda"), empty((B,), torch.float32)
    wide = torch.zeros((B, 2 * V), device="cuda")
    bad = [
        lambda: ctx.sample_rows(x.cpu(), u, tok),
        lambda: ctx.sample_rows(x.half(), u, tok),
        lambda: ctx.sample_rows(x[:, :50], u, tok),
        lambda: ctx.sample_rows(wide[:, ::2], u, tok),
        lambda: ctx.sample_rows(x[:1].expand(B, V), u, tok),
        lambda: ctx.sample_rows(x, u[:2], tok),
        lambda: ctx.sample_rows(x, None, tok),
        lambda: ctx.sample_rows(x, u, tok[:2]),
        lambda: ctx.sample_rows(x, u, tok, temp=torch.ones(B, device="cuda", dtype=torch.float64)),
        lambda: ctx.sample_rows(x, u, tok, top_k=torch.ones(B, device="cuda")),
        lambda: ctx.sample_rows(x, u, tok, bitmask=torch.zeros((B, 3), dtype=torch.int32, device="cuda")),
        lambda: ctx.top_logprobs(x, ids, t[:, :3]),
        lambda: ctx.distill_loss(x, ids, t, f, temp=0.0),
        lambda: ctx.distill_loss(x, ids, t, f, temp=float("inf")),
        lambda: ctx.distill_loss(x, ids, t, f, out_grad=torch.zeros((B, V), device="cuda", dtype=torch.bfloat16)),
        lambda: ctx.distill_loss(wide[:, :V], ids, t, f, out_grad=wide[:, V // 2:V // 2 + V]),
        lambda: ctx.distill_grad(x, ids, t, f, torch.zeros((1, V), device="cuda").expand(B, V)),
    ]
    for call in bad:
        with pytest.raises(CgError) as e:
            call()
        assert e.value.code == _lib.CG_E_ARG
    big_i = torch.zeros((B, 1025), dtype=torch.int32, device="cuda")
    big_f = torch.zeros((B, 1025), device="cuda")
    for call in (lambda: ctx.top_logprobs(x, big_i, big_f), lambda: ctx.distill_loss(x, big_i, big_f, f)):
        with pytest.raises(CgError) as e:
            call()
        assert e.value.code == _lib.CG_E_LIMIT
    # halves of one buffer, side by side, do not overlap
    ctx.distill_loss(wide[:, :V], ids, t, f, out_grad=wide[:, V:])
    torch.cuda.synchronize()
    assert ctx.status() == 0 and (host(tok) == host(tok)).all()
