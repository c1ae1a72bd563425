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


DEALT = r"""
#include <cstdio>
#include <vector>
#include "head_jobs.h"
using namespace cgk;
template <bool TWO>
bool dealt_once(uint32_t pairs, uint32_t tiles, uint32_t splits, uint32_t second_items, uint32_t early) {
  const HeadArgs a{};
  uint32_t status;
  Job j(a, 0, &status, 0, 0);
  j.p[0].n_m = tiles ? 1 : 0;
  j.p[0].n_n = tiles;
  j.p[0].splits = splits;
  j.p[1].n_m = second_items ? 1 : 0;
  j.p[1].n_n = second_items;
  j.p[1].splits = 1;
  j.early = early;
  const uint32_t items[2] = {tiles * splits, TWO ? second_items : 0};
  std::vector<int> seen[2] = {std::vector<int>(items[0]), std::vector<int>(items[1])};
  for (uint32_t pair = 0; pair < pairs; ++pair) {
    Turns<TWO> turns(j, pair, pairs);
    bool second, before = false;
    uint32_t t, most = items[0] + items[1];
    while (turns.next(second, t)) {
      if (t >= items[second] || seen[second][t]++ || (before && !second) || most-- == 0) return false;
      before = second;
    }
  }
  for (auto& s : seen)
    for (int n : s)
      if (n != 1) return false;
  return true;
}
bool stages_once(uint32_t tiles, uint32_t splits, uint32_t blocks) {
  Product p = {};
  p.n_m = 1;
  p.n_n = tiles;
  p.splits = splits;
  p.blocks = blocks;
  std::vector<uint32_t> to(tiles), many(tiles);
  for (uint32_t t = 0; t < tiles * splits; ++t) {   // a tile's splits follow one another in k
    Work w;
    stages_of(p, t, w);
    const uint32_t tile = t - w.split * tiles;
    if (tile >= tiles || w.k0 != to[tile] || w.k1 < w.k0 || w.split != many[tile]++) return false;
    to[tile] = w.k1;
  }
  for (uint32_t t = 0; t < tiles; ++t)
    if (to[t] != blocks || many[t] != splits) return false;
  return true;
}
int main() {
  for (uint32_t pairs : {1u, 2u, 5u, 76u, 152u})
    for (uint32_t tiles : {0u, 1u, 4u, 75u, 76u, 77u, 128u, 300u})
      for (uint32_t splits : {1u, 2u, 9u})
        for (uint32_t second : {0u, 1u, 3u, 100u, 1000u})
          for (uint32_t early : {0u, 1u, 8u, 40u})
            if (!dealt_once<true>(pairs, tiles, splits, second, early) || !dealt_once<false>(pairs, tiles, splits, second, 0))
              return std::printf("dealt: %u takers, %u x %u, %u, %u\n", pairs, tiles, splits, second, early), 0;
  for (uint32_t splits : {1u, 2u, 7u, 152u})
    for (uint32_t blocks : {1u, 6u, 8u, 500u, 6145u})
      if (!stages_once(3, splits, blocks)) return std::printf("stages: %u of %u\n", splits, blocks), 0;
  std::puts("ok");
}
"""


def test_the_kernels_rule_deals_every_item_out_once(tmp_path):
    """Turns and stages_of, as the kernel includes them: every item of either product to one taker, the first
    product's before the second's; every stage to one split, in order."""
    assert compile_and_run(tmp_path, DEALT).strip() == "ok"
