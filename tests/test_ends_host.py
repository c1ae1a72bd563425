"""Host-side checks of the embedding and the output layer's calls that need no GPU."""

import ctypes
import os
import subprocess

import pytest

gcd = pytest.importorskip("grammar_constrained_decoding_gb300")
from grammar_constrained_decoding_gb300 import _lib  # noqa: E402


class Stub:
    """What the checks look at of a tensor, on any device."""

    def __init__(self, shape, dtype, device):
        import torch
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, device

    def get_device(self):
        return self.device

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def numel(self):
        return self.shape.numel()

    def stride(self, i):
        return (self.shape[1], 1)[i]

    def data_ptr(self):
        return 4096


def calls_on(device):
    """A context on CUDA device 1 whose library accepts every call: name -> (method, tensors on `device`)."""
    import torch
    from grammar_constrained_decoding_gb300 import _rows
    ctx = object.__new__(gcd.Ctx)
    ctx._h, ctx._dev, ctx.V, ctx.W, ctx._rows = None, 1, 64, 2, _rows
    B, D = 3, 8
    f = lambda *shape: Stub(shape, torch.float32, device)  # noqa: E731
    i = lambda *shape: Stub(shape, torch.int32, device)    # noqa: E731
    work = Stub((4096,), torch.uint8, device)
    head = dict(hidden=f(B, D), weight=f(64, D), target=i(B), bitmask=i(B, 2), workspace=work)
    return {
        "embed": (ctx.embed, dict(table=f(64, D), tokens=i(B), out=f(B, D))),
        "embed_grad": (ctx.embed_grad, dict(grad=f(B, D), tokens=i(B), out_grad=f(64, D), workspace=work)),
        "head_loss": (ctx.head_loss, dict(head, out_loss=f(B), out_lse=f(B), out_norm=f(B, 2))),
        "head_grad": (ctx.head_grad, dict(head, loss=f(B), norm=f(B, 2), out_grad_hidden=f(B, D), out_grad_weight=f(64, D),
                                          grad_loss=f(B))),
    }


class AcceptingLibrary:
    """Every call that takes a workspace (its last two arguments) wants 1024 bytes; the calls that were accepted."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def entry(*args):
            if name.endswith("_workspace"):
                args[-1]._obj.value = 1024
                return _lib.CG_OK
            if name != "cg_embed" and args[-1] < 1024:
                return _lib.CG_E_NOMEM
            self.calls.append(name)
            return _lib.CG_OK
        return entry


@pytest.mark.parametrize("name", ["embed", "embed_grad", "head_loss", "head_grad"])
def test_tensors_of_another_device_are_refused(monkeypatch, name):
    """Each argument in turn on device 0 (and on the host) where the context is on device 1:
    refused before the library is called."""
    library = AcceptingLibrary()
    monkeypatch.setattr(_lib, "lib", lambda: library)
    call, there = calls_on(1)[name]
    call(**there)
    assert library.calls == ["cg_" + name]
    for device in (0, -1):
        elsewhere = calls_on(device)[name][1]
        for arg in there:
            with pytest.raises(gcd.CgError) as e:
                call(**{**there, arg: elsewhere[arg]})
            assert e.value.code == _lib.CG_E_ARG and "cuda:1" in str(e.value), arg
    assert len(library.calls) == 1


@pytest.mark.parametrize("name", ["embed_grad", "head_loss", "head_grad"])
def test_a_small_workspace_is_refused(monkeypatch, name):
    import torch
    library = AcceptingLibrary()
    monkeypatch.setattr(_lib, "lib", lambda: library)
    call, there = calls_on(1)[name]
    with pytest.raises(gcd.CgError) as e:
        call(**{**there, "workspace": Stub((1023,), torch.uint8, 1)})
    assert e.value.code == _lib.CG_E_NOMEM
    with pytest.raises(gcd.CgError):
        call(**{**there, "workspace": Stub((4096,), torch.int32, 1)})
    assert not library.calls


def test_calls_refuse_a_missing_context():
    lib = _lib.lib()
    buf = (ctypes.c_float * 64)()
    p = ctypes.cast(buf, ctypes.c_void_p)
    n = ctypes.c_size_t(7)
    f32 = _lib.CG_F32
    assert lib.cg_embed(None, p, f32, 8, 8, 8, p, 1, 1.0, p, 8) == _lib.CG_E_ARG
    assert lib.cg_embed_workspace(None, f32, 1, 8, ctypes.byref(n)) == _lib.CG_E_ARG
    assert lib.cg_embed_grad(None, p, f32, 1, 8, 8, 8, p, 1.0, 0, p, 8, p, 256) == _lib.CG_E_ARG
    assert lib.cg_head_workspace(None, p, p, f32, 1, 8, 8, 8, 8, 0, ctypes.byref(n)) == _lib.CG_E_ARG
    assert lib.cg_head_loss(None, p, p, f32, 1, 8, 8, 8, 8, None, p, 1.0, p, None, None, p, 256) == _lib.CG_E_ARG
    assert lib.cg_head_grad(None, p, p, f32, 1, 8, 8, 8, 8, None, p, 1.0, p, p, None, p, 8, p, 8, p, 256) == _lib.CG_E_ARG
    assert n.value == 7


MATRICES = r"""
#include <cstdio>
#include "matrix_args.h"
using namespace cgk;
int main() {
  char* b = reinterpret_cast<char*>(1 << 20);
  bool ok = true;
  // [rows][ld] at an address, D = 8 columns of 4 bytes: apart, side by side, over one another
  ok = ok && !matrices_meet(b, 4, 8, b + 4 * 8 * 4, 4, 8, 8, 4) && matrices_meet(b, 4, 8, b + 4 * 8 * 4 - 4, 4, 8, 8, 4);
  ok = ok && !matrices_meet(b, 4, 16, b + 8 * 4, 4, 16, 8, 4) && !matrices_meet(b + 8 * 4, 4, 16, b, 4, 16, 8, 4);
  ok = ok && matrices_meet(b, 4, 16, b + 7 * 4, 4, 16, 8, 4) && matrices_meet(b, 4, 16, b + 16 * 4 - 4, 4, 16, 8, 4);
  ok = ok && matrices_meet(b, 4, 16, b + 9 * 4, 4, 16, 8, 4);              // its last columns are the next rows' first
  ok = ok && matrices_meet(b, 4, 16, b + 8 * 4, 4, 17, 8, 4);              // other pitches: not told apart
  ok = ok && !matrices_meet(b, 0, 8, b, 4, 8, 8, 4) && matrices_meet(b, 1, 8, b, 1, 8, 8, 4);
  ok = ok && matrix_ok(b, CG_BF16, 1, 8, 8) && matrix_ok(b + 2, CG_BF16, 1, 8, 9) && !matrix_ok(b + 1, CG_BF16, 1, 8, 8);
  ok = ok && !matrix_ok(b + 2, CG_F32, 1, 8, 8) && !matrix_ok(b, CG_F32, 1, 8, 7) && !matrix_ok(nullptr, CG_F32, 1, 8, 8);
  ok = ok && matrix_ok(nullptr, CG_F32, 0, 8, 8) && !matrix_ok(b, CG_F32, 1, 8, (uint64_t(1) << 32) + 1);
  std::puts(ok ? "ok" : "wrong");
}
"""


def test_matrix_checks(tmp_path):
    csrc = os.path.join(os.path.dirname(gcd.__file__), "csrc")
    (tmp_path / "t.cpp").write_text(MATRICES)
    subprocess.run(["g++", "-std=c++17", "-Wall", f"-I{csrc}", str(tmp_path / "t.cpp"), "-o", str(tmp_path / "t")], check=True)
    assert subprocess.run([str(tmp_path / "t")], capture_output=True, text=True).stdout.strip() == "ok"


@pytest.mark.parametrize("pairs", [1, 2, 5, 76])
def test_every_item_of_a_launch_is_dealt_out_once(pairs):
    """The rule by which the takers of a launch find their items, restated: the first product's go
    round; a taker without one in the last round takes `early` of the second's meanwhile."""
    for first in (0, 1, 4, 75, 76, 77, 128, 300):
        for second in (0, 1, 3, 100, 1000):
            for early in (0, 1, 8, 40):
                mine, extra = divmod(first, pairs)
                got = [[], []]
                for pair in range(pairs):
                    got[0] += [pair + i * pairs for i in range(mine + (pair < extra))]
                    k, own_early = 0, 0 if pair < extra else early
                    while True:
                        t = k * (pairs - extra) + pair - extra if k < own_early else early * (pairs - extra) + (k - own_early) * pairs + pair
                        if t >= second:
                            break
                        got[1].append(t)
                        k += 1
                assert sorted(got[0]) == list(range(first)) and sorted(got[1]) == list(range(second))
