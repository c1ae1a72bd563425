"""Settings that a row of sample_rows does not read, and outputs that a refused
call leaves alone."""

import numpy as np
import pytest

from tests.gpu_helpers import empty, host, u32
from tests.rows_ctx import ctx_of, f32_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V,dtype", [(100, "f32"), (5003, "bf16"), (128256, "bf16")])
def test_greedy_rows_read_no_other_setting(V, dtype):
    """T = 0 (of either sign) takes the maximum whatever the other settings hold."""
    import torch
    nan, B = float("nan"), 8
    rng = np.random.default_rng(V)
    x = torch.from_numpy(rng.normal(0, 2, (B, V)).astype(np.float32)).to(
        torch.bfloat16 if dtype == "bf16" else torch.float32)
    want = np.argmax(x.double().numpy(), axis=1)
    ctx, x = ctx_of(V), x.cuda()
    T = f32_dev([0.0, -0.0] * (B // 2))
    clean, lp0 = empty((B,), torch.int32), empty((B,), torch.float32)
    ctx.sample_rows(x, None, clean, temp=T, out_logprob=lp0)
    assert ctx.status() == 0 and host(clean).tolist() == want.tolist()
    u = f32_dev(np.full((B, V), nan))
    tok, lp = empty((B,), torch.int32), empty((B,), torch.float32)
    ctx.sample_rows(x, u, tok, temp=T, top_k=u32([0xFFFFFFFF, 1] * (B // 2)), top_p=f32_dev([nan, nan, -1.0, nan] * (B // 4)),
                    min_p=f32_dev([nan, 0.5, nan, 7.0] * (B // 4)), out_logprob=lp)
    assert ctx.status() == 0
    assert host(tok).tolist() == want.tolist() and np.array_equal(host(lp), host(lp0))
    # beside a sampled row whose setting is not a number: that row alone is refused
    T2, p2 = f32_dev([0.0, 1.0] * (B // 2)), f32_dev([nan] * B)
    ctx.sample_rows(x, f32_dev(np.full((B, V), 0.5)), tok, temp=T2, top_p=p2, out_logprob=lp)
    assert ctx.status() == 10                                     # CG_DEV_BAD_PARAM
    assert (host(tok)[0::2] == want[0::2]).all() and (host(tok)[1::2] == -1).all()


def test_min_p_outside_its_range():
    """Below 0 it keeps every token, above 1 only the maximum."""
    import torch
    from oracle import rows as R
    V, B = 3001, 8
    rng = np.random.default_rng(2)
    x, u = f32_dev(rng.normal(0, 2, (B, V))), rng.random((B, V)).astype(np.float32)
    tok, ctx = empty((B,), torch.int32), ctx_of(V)
    ctx.sample_rows(x, f32_dev(u), tok, min_p=f32_dev([-0.5, 2.0] * (B // 2)))
    assert ctx.status() == 0
    v = host(x).astype(np.float64)
    for b in range(B):
        want = R.sample_rows_row(v[b], 1.0, 0, 1.0, 0.0 if b % 2 == 0 else 1.0, u[b])
        assert want.gap > 1e-4 and int(host(tok)[b]) == want.tok, b


def test_refused_calls_leave_the_outputs_alone():
    import torch
    from grammar_constrained_decoding_gb300 import CgError
    V, B, K = 100, 3, 4
    ctx = ctx_of(V)
    x, u = torch.zeros((B, V), device="cuda"), torch.full((B, V), 0.5, device="cuda")
    ids, t = torch.zeros((B, K), dtype=torch.int32, device="cuda"), torch.zeros((B, K), device="cuda")
    ints = [torch.full(s, -77, dtype=torch.int32, device="cuda") for s in ((B,), (B, K))]
    floats = [torch.full(s, -77.0, device="cuda") for s in ((B,), (B, K), (B,), (B, 2), (B, V))]
    (tok, best), (lp, lps, loss, norm, grad) = ints, floats
    bad_mask = torch.zeros((B, 3), dtype=torch.int32, device="cuda")
    for call in (lambda: ctx.sample_rows(x, u[:2], tok, out_logprob=lp),
                 lambda: ctx.sample_rows(x, None, tok, out_logprob=lp),
                 lambda: ctx.sample_rows(x, u, tok, bitmask=bad_mask, out_logprob=lp),
                 lambda: ctx.top_logprobs(x, best, lps, bitmask=bad_mask, out_lse=lp),
                 lambda: ctx.distill_loss(x, ids, t, loss, temp=-1.0, out_norm=norm, out_grad=grad),
                 lambda: ctx.distill_loss(x, ids, t, loss, bitmask=bad_mask, out_norm=norm, out_grad=grad),
                 lambda: ctx.distill_grad(x, ids, t, lp, grad, temp=float("nan"))):
        with pytest.raises(CgError):
            call()
    assert ctx.status() == 0
    assert all((a == -77).all() for a in ints + floats)
