"""Per-row sampling, best tokens and distillation on the CPU (oracle), in float64.

The definitions are those of include/cg.h ("per-row sampling, best tokens,
distillation"), written down directly: a logit that is -inf or NaN, or whose
mask bit is clear, is not allowed; +inf counts as the largest finite value.
``gap`` and ``margin`` of a sampled row say by how much its outcome stands: the
distance between the two best scores, and of the top-p and min-p thresholds
from the nearest value they could have been -- an implementation in 32 bits may
differ only where one of them is below its rounding error.
"""

from __future__ import annotations

from dataclasses import dataclass

import numpy as np

NO_TOKEN = 0xFFFFFFFF
U_LO, U_HI = 2.0 ** -32, 1.0 - 2.0 ** -24
MAX_BF16 = float.fromhex("0x1.fep+127")
MAX_F32 = float(np.finfo(np.float32).max)


def allowed_logits(x: np.ndarray, mask: np.ndarray | None, dtype: str) -> np.ndarray:
    """float64 [V]: -inf where not allowed, +inf replaced."""
    v = np.array(x, dtype=np.float64)
    v[np.isnan(v)] = -np.inf
    v[v == np.inf] = MAX_BF16 if dtype == "bf16" else MAX_F32
    if mask is not None:
        v[~mask] = -np.inf
    return v


def log_softmax(v: np.ndarray) -> tuple[np.ndarray, float]:
    """(log softmax, log sum exp), the first without the rounding of the second:
    (v - m) - log sum exp(v - m)."""
    m = v.max(initial=-np.inf)
    if m == -np.inf:
        return np.full(v.shape, -np.inf), -np.inf
    d = v - m
    log_s = float(np.log(np.exp(d).sum()))
    return d - log_s, float(m + log_s)


@dataclass
class RowSample:
    tok: int
    logprob: float
    gap: float
    margin: float


def sample_rows_row(v: np.ndarray, temp: float, top_k: int, top_p: float, min_p: float, u: np.ndarray | None) -> RowSample:
    """v from allowed_logits; the settings as the binary32 values passed."""
    ids = np.flatnonzero(v > -np.inf)
    if ids.size == 0:
        return RowSample(NO_TOKEN, -np.inf, np.inf, np.inf)
    x = v[ids]
    m = x.max()
    if temp == 0.0:
        i = int(np.argmax(x))  # first of the largest
        return RowSample(int(ids[i]), float(x[i] - m) - float(np.log(np.exp(x - m).sum())), np.inf, np.inf)
    z = (x - m) / temp
    e = np.exp(z)
    logp = z - np.log(e.sum())
    keep = np.ones(x.size, dtype=bool)
    margin = np.inf
    if 0 < top_k < x.size:
        keep = x >= np.sort(x)[::-1][top_k - 1]
    if top_p < 1.0:
        values, where = np.unique(x[keep], return_inverse=True)
        mass = np.bincount(where.reshape(-1), weights=e[keep])[::-1]
        cum = np.cumsum(mass) / mass.sum()
        hit = np.flatnonzero(cum >= max(top_p, 0.0))
        j = int(hit[0]) if hit.size else values.size - 1
        keep &= x >= values[::-1][j]
        margin = min(cum[j] - top_p, (top_p - cum[j - 1]) if j else np.inf)
        margin = np.inf if j == 0 and top_p <= 0.0 else abs(margin)
    if min_p > 0.0:
        floor = np.log(min(min_p, 1.0))
        keep &= z >= floor
        if floor < 0.0:
            margin = min(margin, float(np.abs(z - floor).min()))
    g = -np.log(-np.log(np.clip(np.nan_to_num(u[ids].astype(np.float64), nan=0.0), U_LO, U_HI)))
    score = np.where(keep, z + g, -np.inf)
    i = int(np.argmax(score))
    rest = np.sort(score[keep])
    gap = float(rest[-1] - rest[-2]) if rest.size > 1 else np.inf
    return RowSample(int(ids[i]), float(logp[i]), gap, float(margin))


def top_logprobs_row(v: np.ndarray, n: int):
    """(ids u32 [n], logprobs [n], lse)."""
    logp, lse = log_softmax(v)
    order = np.lexsort((np.arange(v.size), -v))
    order = order[v[order] > -np.inf][:n]
    ids = np.full(n, NO_TOKEN, dtype=np.uint32)
    lps = np.full(n, -np.inf)
    ids[:order.size] = order
    lps[:order.size] = logp[order]
    return ids, lps, lse


def distill_row(v: np.ndarray, ids: np.ndarray, teacher: np.ndarray, temp: float):
    """(loss, lse of v / temp, dloss/dv [V])."""
    logp, lse = log_softmax(v / temp)
    t = np.array(teacher, dtype=np.float64)
    t[t == np.inf] = MAX_F32
    ids = np.asarray(ids, dtype=np.int64)
    ok = (ids < v.size) & (t > -np.inf)      # false for a NaN
    ok[ok] = v[ids[ok]] > -np.inf
    grad = np.zeros(v.size)
    if not ok.any():
        return 0.0, lse, grad
    log_q, _ = log_softmax(t[ok] / temp)
    q = np.exp(log_q)
    terms = np.where(q > 0.0, q * (np.where(q > 0.0, log_q, 0.0) - logp[ids[ok]]), 0.0)
    live = v > -np.inf
    grad[live] = np.exp(logp[live])
    np.subtract.at(grad, ids[ok], q)
    return temp * temp * float(terms.sum()), lse, temp * grad
