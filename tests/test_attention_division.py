"""How the attention over the paged cache divides its work, checked by a host compiler: a launch that joins the parts of split
tiles follows wherever the kernels can split one."""
import os
import subprocess

from nvfp4_block_scaled_moe_amd.build import CSRC

# Every page size, every table of up to 8000 tokens, every length that it holds and every share of up to 40 blocks: a tile in
# several parts means that the host, which knows the table's columns alone, launches the join.
WALK = r"""
#include <cstdio>
#include "kv_division.h"
using namespace nvfp4moe;
int main() {
  const Division all[] = {few_division(false), few_division(true), chunk_division(4), chunk_division(8)};
  const char* names[] = {"16 rows bf16", "16 rows e4m3", "128 rows", "256 rows"};
  long split = 0, bad = 0;
  for (int i = 0; i < 4; ++i)
    for (int page = 16; page <= 1024; page *= 2)
      for (long cols = 1; cols * page <= 8000; ++cols)
        for (long len = 0; len <= cols * page; ++len)
          for (int chunk = all[i].min_blocks; chunk <= 40; ++chunk) {
            if (parts_of((uint32_t)blocks_of(len, all[i].block_log), (uint32_t)chunk) < 2) break;   // (nor for any larger share)
            ++split;
            if (!all[i].can_split(cols * page) && ++bad <= 10)
              std::printf("%s: %ld tokens in %ld columns of %d are split and not joined\n", names[i], len, cols, page);
          }
  std::printf("%ld split, %ld of them not joined\n", split, bad);
  return bad != 0 || split == 0;
}
"""


def test_every_split_tile_is_joined(tmp_path):
    source, program = tmp_path / "walk.cpp", tmp_path / "walk"
    source.write_text(WALK)
    subprocess.run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", f"-I{CSRC}", str(source), "-o", str(program)], check=True)
    r = subprocess.run([str(program)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
