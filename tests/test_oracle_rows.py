"""CPU tests of the per-row operators: the oracle against independent
statements of the same mathematics, and the library's host-side refusals."""

import ctypes

import numpy as np
import pytest

from oracle import rows as R

gcd = pytest.importorskip("grammar_constrained_decoding_gb300")
from grammar_constrained_decoding_gb300 import _lib  # noqa: E402


def test_cuts_keep_the_sets_their_names_say():
    """Distribution (0.4, 0.3, 0.2, 0.1): with equal random numbers the best kept
    token is the first, with u raised for one token that token wins iff kept."""
    v = np.log(np.array([0.2, 0.4, 0.1, 0.3]))
    u = np.full(4, 0.5)

    def kept(**kw):
        a = dict(temp=1.0, top_k=0, top_p=1.0, min_p=0.0)
        a.update(kw)
        out = set()
        for t in range(4):
            w = u.copy()
            w[t] = 1.0 - 2.0 ** -24
            if R.sample_rows_row(v, a["temp"], a["top_k"], a["top_p"], a["min_p"], w).tok == t:
                out.add(t)
        return out

    assert kept() == {0, 1, 2, 3}
    assert kept(top_k=2) == {1, 3}
    assert kept(top_p=0.6) == {1, 3}
    assert kept(top_p=0.75) == {0, 1, 3}
    assert kept(top_p=0.0) == {1}
    assert kept(min_p=0.3) == {0, 1, 3}
    assert kept(top_k=3, top_p=0.7) == {1, 3}          # 0.7 of 0.9, not of 1
    assert kept(temp=0.0) <= {1}
    assert R.sample_rows_row(v, 1.0, 0, 1.0, 0.0, u).logprob == pytest.approx(np.log(0.4))


def test_draws_follow_the_distribution():
    """Over many random rows the argmax of z - log(-log u) has frequency p
    (chi-square, 4 degrees of freedom, 1e-6 point at 33.4)."""
    v = np.array([0.0, 1.0, -0.5, 2.0, 0.3])
    p = np.exp(v) / np.exp(v).sum()
    rng = np.random.default_rng(5)
    n = 20000
    hits = np.zeros(5)
    for _ in range(n):
        hits[R.sample_rows_row(v, 1.0, 0, 1.0, 0.0, rng.random(5)).tok] += 1
    assert (((hits - n * p) ** 2) / (n * p)).sum() < 33.4


def test_distill_gradient_is_the_derivative():
    """Central differences of the loss, step 1e-5: truncation and cancellation
    both below 1e-8 for losses of this size."""
    rng = np.random.default_rng(2)
    for temp in (0.5, 1.0, 3.0):
        v = rng.normal(0, 2, 40)
        v[[3, 17]] = -np.inf
        ids = np.array([5, 9, 9, 3, R.NO_TOKEN, 20], dtype=np.uint32)
        t = rng.normal(0, 2, 6)
        _, _, g = R.distill_row(v, ids, t, temp)
        for i in range(40):
            if v[i] == -np.inf:
                assert g[i] == 0.0
                continue
            a, b = v.copy(), v.copy()
            a[i] += 1e-5
            b[i] -= 1e-5
            d = (R.distill_row(a, ids, t, temp)[0] - R.distill_row(b, ids, t, temp)[0]) / 2e-5
            assert abs(d - g[i]) < 1e-8
        assert abs(g.sum()) < 1e-12


def test_top_rows_are_ordered_with_ties_by_id():
    v = np.array([1.0, 3.0, -np.inf, 3.0, 2.0])
    ids, lps, lse = R.top_logprobs_row(v, 6)
    assert ids.tolist() == [1, 3, 4, 0, R.NO_TOKEN, R.NO_TOKEN]
    assert lps[4] == -np.inf and np.exp(lps[:4]).sum() == pytest.approx(1.0)
    assert lse == pytest.approx(np.log(np.exp(v[[0, 1, 3, 4]]).sum()))


def test_calls_refuse_a_missing_context_before_any_device_call():
    lib = _lib.lib()
    buf = (ctypes.c_float * 64)()
    p = ctypes.cast(buf, ctypes.c_void_p)
    f32 = _lib.CG_F32
    assert lib.cg_sample_rows(None, p, f32, 1, 8, 8, None, None, None, None, None, p, 8, p, None) == _lib.CG_E_ARG
    assert lib.cg_top_logprobs(None, p, f32, 1, 8, 8, None, 4, p, p, None) == _lib.CG_E_ARG
    assert lib.cg_distill_loss(None, p, f32, 1, 8, 8, None, p, p, 4, 1.0, p, None, None, None, 0) == _lib.CG_E_ARG
    assert lib.cg_distill_grad(None, p, f32, 1, 8, 8, None, p, p, 4, 1.0, p, None, p, 8) == _lib.CG_E_ARG


def test_python_entry_points_refuse_host_tensors():
    import torch
    from grammar_constrained_decoding_gb300 import CgError, _rows

    with pytest.raises(CgError) as e:
        _rows.rows_of("cg_sample_rows", torch.zeros(2, 8), "logits", _rows.LOGITS, (2, 8))
    assert e.value.code == _lib.CG_E_ARG
    with pytest.raises(CgError):
        _rows.want("cg_sample_rows", torch.zeros(2), "temp", _rows.F32, (2,))
    assert _rows.opt("cg_sample_rows", None, "temp", _rows.F32, (2,)) is None
