"""Host-side checks of the per-row operators that need no GPU."""

import ctypes
import os
import subprocess

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


class Stub:
    """What the checks look at of a tensor, on any device."""

    def __init__(self, shape, dtype, device):
        self.shape, self.dtype, self.device = shape, dtype, device
        self.is_cuda = device >= 0

    def get_device(self):
        return self.device

    def is_contiguous(self):
        return True

    def stride(self, i):
        return (self.shape[1], 1)[i]

    def data_ptr(self):
        return 4096


def calls_on(device):
    """A context on CUDA device 1 whose library accepts every call: name -> (method, tensors on `device`)."""
    import torch
    ctx = object.__new__(gcd.Ctx)
    ctx._h, ctx._dev, ctx.V, ctx.W = None, 1, 64, 2
    from grammar_constrained_decoding_gb300 import _rows
    ctx._rows = _rows
    B, K = 3, 4
    f = lambda *shape: Stub(shape, torch.float32, device)  # noqa: E731
    i = lambda *shape: Stub(shape, torch.int32, device)    # noqa: E731
    lists = dict(logits=f(B, 64), ids=i(B, K), teacher=f(B, K), bitmask=i(B, 2), grad_loss=f(B), out_grad=f(B, 64))
    return {
        "sample_rows": (ctx.sample_rows, dict(logits=f(B, 64), uniform=f(B, 64), out_tok=i(B), bitmask=i(B, 2), temp=f(B),
                                              top_k=i(B), top_p=f(B), min_p=f(B), out_logprob=f(B))),
        "top_logprobs": (ctx.top_logprobs, dict(logits=f(B, 64), out_ids=i(B, K), out_logprobs=f(B, K), bitmask=i(B, 2),
                                                out_lse=f(B))),
        "distill_loss": (ctx.distill_loss, dict(lists, out_loss=f(B), out_lse=f(B), out_norm=f(B, 2))),
        "distill_grad": (ctx.distill_grad, dict(lists, lse=f(B))),
        "distill_grad_norm": (lambda **k: ctx.distill_grad(lse=None, **k), dict(lists, norm=f(B, 2))),
    }


class AcceptingLibrary:
    calls = 0

    def __getattr__(self, name):
        def entry(*args):
            AcceptingLibrary.calls += 1
            return _lib.CG_OK
        return entry


@pytest.mark.parametrize("name", ["sample_rows", "top_logprobs", "distill_loss", "distill_grad", "distill_grad_norm"])
def test_tensors_of_another_device_are_refused(monkeypatch, name):
    """Each argument in turn on device 0 (and on the host) where the context is on device 1:
    refused before the library is called."""
    library = AcceptingLibrary()
    monkeypatch.setattr(_lib, "lib", lambda: library)
    call, there = calls_on(1)[name]
    AcceptingLibrary.calls = 0
    call(**there)
    assert AcceptingLibrary.calls == 1
    for device in (0, -1):
        elsewhere = calls_on(device)[name][1]
        for arg in there:
            with pytest.raises(gcd.CgError) as e:
                call(**{**there, arg: elsewhere[arg]})
            assert e.value.code == _lib.CG_E_ARG and "cuda:1" in str(e.value), arg
    assert AcceptingLibrary.calls == 1


DEVICE_ANSWERS = r"""
#include <cstdio>
#include "device_answers.h"
int main() {
  static cgk::DeviceAnswers known;
  int asked = 0;
  auto ask = [&](int v) { return [&asked, v] { ++asked; return v; }; };
  bool ok = known.get(0, ask(36)) == 36 && known.get(1, ask(18)) == 18;   // each device its own
  ok = ok && known.get(0, ask(5)) == 36 && known.get(1, ask(5)) == 18 && asked == 2;
  ok = ok && known.get(2, ask(0)) == 0 && known.get(2, ask(7)) == 7;      // a failed answer is not kept
  ok = ok && known.get(63, ask(3)) == 3 && known.get(63, ask(4)) == 3;
  ok = ok && known.get(64, ask(9)) == 9 && known.get(64, ask(11)) == 11;  // past the table: asked
  ok = ok && known.get(128, ask(13)) == 13 && known.get(0, ask(5)) == 36;
  std::puts(ok ? "ok" : "wrong");
}
"""


def test_answers_are_kept_for_each_device(tmp_path):
    csrc = os.path.join(os.path.dirname(gcd.__file__), "csrc")
    (tmp_path / "t.cpp").write_text(DEVICE_ANSWERS)
    subprocess.run(["g++", "-std=c++17", "-Wall", f"-I{csrc}", str(tmp_path / "t.cpp"), "-o", str(tmp_path / "t")], check=True)
    assert subprocess.run([str(tmp_path / "t")], capture_output=True, text=True).stdout.strip() == "ok"


def test_process_wide_answers_of_the_row_operators_are_kept_per_device():
    """No answer of a device is kept in a variable of its own beside the table."""
    csrc = os.path.join(os.path.dirname(gcd.__file__), "csrc")
    for name in ("logit_row.cuh", "kernel_distill.cu", "kernel_draw.cu", "kernel_top.cu"):
        with open(os.path.join(csrc, name)) as f:
            assert "static std::atomic" not in f.read(), name


def test_cluster_self_test_refuses_missing_arguments():
    lib = _lib.lib()
    p = ctypes.cast((ctypes.c_uint32 * 4)(), ctypes.c_void_p)
    assert lib.cg_self_test_cluster_timeout(None, p) == _lib.CG_E_ARG
    assert lib.cg_self_test_cluster_timeout(None, None) == _lib.CG_E_ARG
