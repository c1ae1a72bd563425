"""Host-side checks of the per-row operators that need no GPU."""

import ctypes

import pytest

gcd = pytest.importorskip("grammar_constrained_decoding_gb300")
from grammar_constrained_decoding_gb300 import _lib  # noqa: E402


def test_two_value_normaliser_calls_refuse_a_missing_context():
    lib = _lib.lib()
    buf = (ctypes.c_float * 64)()
    p = ctypes.cast(buf, ctypes.c_void_p)
    f32 = _lib.CG_F32
    assert lib.cg_distill_loss_norm(None, p, f32, 1, 8, 8, None, p, p, 4, 1.0, p, p, p, None, None, 0) == _lib.CG_E_ARG
    assert lib.cg_distill_grad_norm(None, p, f32, 1, 8, 8, None, p, p, 4, 1.0, p, None, p, 8) == _lib.CG_E_ARG
