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
