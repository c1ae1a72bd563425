"""A block of a cluster whose bounded wait ran out stays until the others, who may
still send to its shared memory, have done so; the context stays usable."""

import time

import numpy as np
import pytest

from tests.gpu_helpers import empty, host
from tests.rows_ctx import ctx_of, f32_dev

pytestmark = pytest.mark.gpu
CG_DEV_TIMEOUT = 8


def test_a_block_that_gave_up_leaves_last():
    import torch
    V, B = 1000, 4
    ctx, out = ctx_of(V), empty((1,), torch.int32)
    out.fill_(-1)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    ctx.self_test_cluster_timeout(out)
    code = ctx.status()
    assert time.perf_counter() - t0 < 20.0
    assert code == CG_DEV_TIMEOUT and host(out).tolist() == [6]
    assert ctx.status() == 0
    x, tok = f32_dev(np.eye(B, V)), empty((B,), torch.int32)
    ctx.sample_rows(x, None, tok, temp=f32_dev([0.0] * B))
    assert ctx.status() == 0 and host(tok).tolist() == list(range(B))
