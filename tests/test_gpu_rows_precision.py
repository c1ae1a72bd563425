"""Log-probabilities near 0.  Where the best token has nearly all the mass, its
log-probability is -log(1 + r) with r the mass of the others in units of its own,
and the result is as good as r, not as good as 1 + r.

Tolerance.  r is a sum of exponentials: rel_sum(V) for the sum, 3 |z| 2^-24 for
each argument (a difference, a scale and a product), 8 x 2^-24 for the joins over
warps and blocks and the logarithm.  Masses of tokens more than 45 nats down add
less than e^-45 V, which is added to the bound."""

import numpy as np
import pytest

from oracle import rows as R
from tests.gpu_helpers import empty, host
from tests.rows_ctx import ctx_of, f32_dev, rel_sum

pytestmark = pytest.mark.gpu
ABOVE = [2.0, 6.0, 9.0, 12.0, 15.0, 18.0, 22.0, 26.0, 30.0, 34.0, 38.0, 24.5]


def make(rng, B, V, dtype, temp):
    """Rows whose best token leads the others by about a few to tens of nats at temp."""
    import torch
    x = rng.normal(0, 1, (B, V)) * temp
    at = rng.integers(0, V, B)
    for b in range(B):
        x[b, at[b]] = x[b].max() + ABOVE[b % len(ABOVE)] * temp
    t = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    return t.cuda(), t.double().numpy(), at


def close(got, v, temp, V, b):
    z = (v - v.max()) / temp
    rest = np.exp(np.delete(z, np.argmax(z))).sum()
    want = -np.log1p(rest)
    span = min(45.0, float(-z.min()))
    tol = abs(want) * (rel_sum(V) + (3 * span + 8) * 2.0 ** -24) + np.exp(-45.0) * V + 1e-44
    assert abs(float(got) - want) <= tol, (b, float(got), want, abs(float(got) - want) / abs(want))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,B", [(33, 12), (4013, 12), (32000, 1), (32000, 12), (128256, 24), (32003, 400)])
def test_top_logprobs_near_zero(V, B, dtype):
    import torch
    rng = np.random.default_rng([V, B])
    x, v, at = make(rng, B, V, dtype, 1.0)
    ids, lps, lse = empty((B, 3), torch.int32), empty((B, 3), torch.float32), empty((B,), torch.float32)
    ctx = ctx_of(V)
    ctx.top_logprobs(x, ids, lps, out_lse=lse)
    assert ctx.status() == 0 and host(ids)[:, 0].tolist() == at.tolist()
    for b in range(0, B, 1 + B // 60):
        close(host(lps)[b, 0], v[b], 1.0, V, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,B", [(33, 12), (4013, 12), (32000, 1), (32000, 12), (128256, 24), (32003, 400)])
@pytest.mark.parametrize("settings", [(0.0, 0, 1.0, 0.0), (1.0, 0, 1.0, 0.0), (0.7, 50, 0.9, 0.0), (0.7, 0, 0.9, 0.0),
                                      (1.3, 0, 1.0, 0.05), (1.0, 5000, 1.0, 0.0)])
def test_sampled_logprobs_near_zero(V, B, dtype, settings):
    import torch
    from tests.gpu_helpers import u32
    T = np.float32(settings[0])
    scale = float(T) if T > 0 else 1.0
    rng = np.random.default_rng([V, B, 1])
    x, v, at = make(rng, B, V, dtype, scale)
    tok, lp = empty((B,), torch.int32), empty((B,), torch.float32)
    u = f32_dev(np.full((1, V), 0.5))          # equal random numbers: the best token is drawn
    ctx = ctx_of(V)
    ctx.sample_rows(x, u, tok, temp=f32_dev([T] * B), top_k=u32([settings[1]] * B), top_p=f32_dev([settings[2]] * B),
                    min_p=f32_dev([settings[3]] * B), out_logprob=lp)
    assert ctx.status() == 0 and host(tok).tolist() == at.tolist()
    for b in range(0, B, 1 + B // 60):
        close(host(lp)[b], v[b], scale, V, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_logprobs_near_zero_beside_masked_and_equal_tokens(dtype):
    """A row of one allowed token has log-probability exactly 0; two equal best
    tokens share the mass, and the rest still counts to the last bit of r."""
    import torch
    V = 4013
    rng = np.random.default_rng(9)
    x, v, at = make(rng, 4, V, dtype, 1.0)
    x[1, (int(at[1]) + 700) % V] = x[1, int(at[1])]
    mask = torch.zeros((4, (V + 31) // 32), dtype=torch.int32, device="cuda") - 1
    mask[0] = 0
    bit = int(at[0]) % 32
    mask[0, int(at[0]) // 32] = -2 ** 31 if bit == 31 else 1 << bit
    ids, lps = empty((4, 2), torch.int32), empty((4, 2), torch.float32)
    ctx = ctx_of(V)
    ctx.top_logprobs(x, ids, lps, bitmask=mask)
    assert ctx.status() == 0
    got, w = host(lps), x.double().cpu().numpy()
    assert got[0, 0] == 0.0 and got[0, 1] == -np.inf
    want = R.log_softmax(w[1])[0].max()
    assert abs(got[1, 0] - want) <= rel_sum(V) + abs(want) * 2.0 ** -21
    for b in (2, 3):
        close(got[b, 0], w[b], 1.0, V, b)
