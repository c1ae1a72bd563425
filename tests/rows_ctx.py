"""A context of V tokens for tests of the per-row operators, and the bound of a
normaliser's relative error (derived in test_gpu_rows.py)."""

import functools


def rel_sum(V):
    return 2.0 ** -21 + (V / 512 + 32) * 2.0 ** -24


@functools.lru_cache(maxsize=4)
def ctx_of(V):
    import grammar_constrained_decoding_gb300 as cg
    return cg.Ctx([cg.Grammar.compile('root ::= "a"', "gbnf")], cg.Vocab([i.to_bytes(3, "big") for i in range(V)]))


def f32_dev(a):
    import numpy as np
    import torch
    return torch.tensor(np.asarray(a, dtype=np.float32), device="cuda")
