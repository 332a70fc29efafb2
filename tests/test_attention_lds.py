"""Where paged attention keeps its pieces in LDS, for every head count and head size (CPU).

A piece is joined while the next one's results are written, so two neighbouring pieces must
not share a place.  The last block of query heads may have fewer heads than the others.
"""

import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gram_hash_memory_amd", "csrc")

PROGRAM = r"""
#include <algorithm>
#include <cstdio>
#include "attention_lds.hpp"
using namespace engram::attn;
int main() {
  int bad = 0, seen = 0;
  for (int acc = 2; acc <= 16; acc += 2)                       // head sizes 32 .. 256
    for (int group = 1; group <= 300; ++group) {
      const int block = std::min(kHeadBlock, group);           // heads of all blocks but the last
      const int last = group - (group - 1) / kHeadBlock * kHeadBlock;
      for (int even : {block, last})
        for (int odd : {block, last}) {
          const int a0 = part_begin(acc, block, 0), a1 = a0 + part_places(acc, even);
          const int b0 = part_begin(acc, block, 1), b1 = b0 + part_places(acc, odd);
          const bool apart = !two_buffers(acc, block) || a1 <= b0 || b1 <= a0;
          const bool inside = 16u * std::max(a1, b1) <= result_bytes(acc, block);
          seen += two_buffers(acc, block);
          if (!apart || !inside) {
            if (!bad++)
              std::printf("%d heads of %d: pieces of %d and %d heads at %d..%d and %d..%d\n", group, 16 * acc, even,
                          odd, a0, a1, b0, b1);
          }
        }
    }
  std::printf("%d bad of %d with two buffers\n", bad, seen);
  return bad || !seen;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_neighbouring_pieces_share_no_place(tmp_path):
    src, exe = tmp_path / "lds.cpp", tmp_path / "lds"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", f"-I{CSRC}", str(src), "-o", str(exe)], check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True)
    assert res.returncode == 0, res.stdout
