"""Host-side checks of what the output layer's launches are made of (csrc/head_jobs.h), compiled without a GPU."""

import os
import re
import subprocess

import pytest

gcd = pytest.importorskip("grammar_constrained_decoding_gb300")
from grammar_constrained_decoding_gb300 import build  # noqa: E402

CSRC = os.path.join(os.path.dirname(gcd.__file__), "csrc")


def compile_and_run(tmp_path, program, *args):
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build._nvcc()))), "include")
    source, binary = str(tmp_path / "t.cpp"), str(tmp_path / "t")
    with open(source, "w") as f:
        f.write(program)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", f"-I{CSRC}", f"-isystem{include}", source, "-o", binary], check=True)
    return subprocess.run([binary, *args], capture_output=True, text=True, check=True).stdout


JOB = r"""
#include <cstdio>
#include <type_traits>
#include "head_jobs.h"
using namespace cgk;
static_assert(!std::is_default_constructible_v<Job>, "a launch cannot be made without what all of them read");
static_assert(std::is_trivially_copyable_v<Job>, "a kernel's argument");
int main() {
  uint32_t status, mask, target;
  const HeadArgs a{nullptr, nullptr, 0, 300, 5000, 64, 64, 64, &mask, &target, 0.5f};
  const Job j(a, 157, &status, 512, 256);
  const bool ok = j.status == &status && j.bitmask == &mask && j.target == &target && j.temp == 0.5f && j.rows == 300 &&
                  j.W == 157 && j.v0 == 512 && j.tokens == 256 && j.p[0].splits == 0 && j.p[1].splits == 0 && !j.w && !j.terms.up;
  std::puts(ok ? "ok" : "wrong");
}
"""


def test_every_launch_has_what_all_of_them_read(tmp_path):
    """The status among it, which a wait that runs out writes to: no launch is made but by the constructor."""
    assert compile_and_run(tmp_path, JOB).strip() == "ok"
    with open(os.path.join(CSRC, "kernel_head.cu")) as f:
        source = f.read()
    made = [line for line in re.findall(r"^ +Job \w+.*;$", source, re.M) if "= logits_of(a, p, v, v0, n);" not in line]
    assert len(made) == 2 and all(line.endswith("(a, v.t.W, v.t.status, v0, n);") for line in made), made


def test_a_warp_gives_up_a_wait_as_one():
    """A wait by all lanes of a warp may run out for some of them alone: what follows is for whole warps (tensor
    memory, __syncwarp), so the warp votes.  Shown by reading: waits are by one lane, or under a vote."""
    with open(os.path.join(CSRC, "kernel_head.cu")) as f:
        source = f.read()
    readers = source[source.index("} else if (warp >= kFirstReader) {"):source.index("constexpr size_t product_smem()")]
    waits = re.findall(r"const bool (\w+) = mbar_wait\([^;]*;\s*if \(!__all_sync\(0xFFFFFFFFu, (\w+)\)\)", readers)
    assert waits == [("there", "there")] and readers.count("mbar_wait(") == 1


ONE_ROW = r"""
#include <cstdio>
#include <initializer_list>
#include "matrix_args.h"
using namespace cgk;
int main() {
  char* b = reinterpret_cast<char*>(1 << 20);
  bool ok = true;
  // one row of 8 columns of 4 bytes in a buffer of pitch 16, whatever its own pitch is said to be, beside 4 rows and over them
  for (uint64_t ld : {8, 9, 16, 100}) {
    ok = ok && !matrices_meet(b + 8 * 4, 1, ld, b, 4, 16, 8, 4) && !matrices_meet(b, 4, 16, b + 8 * 4, 1, ld, 8, 4);
    ok = ok && !matrices_meet(b + (32 + 8) * 4, 1, ld, b, 4, 16, 8, 4) && !matrices_meet(b, 4, 16, b + (32 + 8) * 4, 1, ld, 8, 4);
    for (int at : {0, 1, 7, 9, 15, 16, 32, 48}) ok = ok && matrices_meet(b + at * 4, 1, ld, b, 4, 16, 8, 4) && matrices_meet(b, 4, 16, b + at * 4, 1, ld, 8, 4);
    ok = ok && !matrices_meet(b + 64 * 4, 1, ld, b, 4, 16, 8, 4) && !matrices_meet(b, 4, 16, b - 8 * 4, 1, ld, 8, 4);
    ok = ok && matrices_meet(b, 1, ld, b + 7 * 4, 1, 8, 8, 4) && !matrices_meet(b, 1, ld, b + 8 * 4, 1, 8, 8, 4);
  }
  std::puts(ok ? "ok" : "wrong");
}
"""


def test_one_row_beside_a_matrix(tmp_path):
    """One row's pitch says nothing: a row in other columns of a matrix's buffer shares no memory with it."""
    assert compile_and_run(tmp_path, ONE_ROW).strip() == "ok"
