"""The places of a path move in an 8-bit cache, on the CPU: the kernel's index
arithmetic (path_places.h) compiled for the host and run over paths that are
longer than their sequence's new tokens.  Every table slot that it names lies in
the table, and every place that a token can move into is met once."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "smc_speculative_decoding_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "path_places.h"
using smcsd::PathPlaces;
static long wrong = 0, calls = 0;
static void walk(int T, int block, int len, int held, int n, int room) {
  const PathPlaces p{len - held, held, n, block};
  std::vector<int> met(n, 0);
  ++calls;
  int at = 0, turns = 0;
  while (at < n) {
    const int end = p.end(at, room);
    if (end <= at || end > n || end - at > room || ++turns > n) { ++wrong; return; }
    for (int from = at, last = p.moves_end(end); from < last;) {
      const int slot = p.slot(from), to = p.slot_end(from, last);
      if (slot < 0 || slot >= T) ++wrong;                    // outside the table
      if (to <= from || to > last) { ++wrong; return; }
      for (int i = from; i < to; ++i) {
        ++met[i];
        if ((p.first + i) / block != slot) ++wrong;          // another block's
      }
      // a block is taken whole: its next place belongs to no later turn
      if (to == last && end < n && to < held && (p.first + to) / block == slot) ++wrong;
      from = to;
    }
    at = end;
  }
  for (int i = 0; i < n; ++i) if (met[i] != (i < held)) ++wrong;
}
int main() {
  for (int block : {1, 2, 3, 7, 16, 20, 1000, 1024})
    for (int T : {1, 2, 3, 9})
      for (int spare : {0, 1, block / 2, block - 1}) {
        const int len = T * block - spare;
        for (int held : {0, 1, 2, 3, 17, block, len / 2, len})
          if (held <= len)
            for (int n : {0, 1, 2, 3, 16, 100, block + 1, 2 * block, len, len + 1, 5000})
              walk(T, block, len, held, n, 1024);
      }
  for (int held : {0, 1, 50}) walk(2147479552 / 16, 16, 2147479552, held, 4000, 1024);  // the largest table
  std::printf("%ld %ld\n", calls, wrong);
}
"""


def test_no_place_past_the_new_tokens_is_looked_up(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    src, exe = tmp_path / "places.cpp", tmp_path / "places"
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=undefined", "-fno-sanitize-recover",
                    f"-I{CSRC}", str(src), "-o", str(exe)], check=True, capture_output=True)
    calls, wrong = map(int, subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split())
    assert calls > 1000 and wrong == 0


def test_the_kernel_goes_by_these_places():
    """It has no limits of its own beside them."""
    text = open(os.path.join(CSRC, "cache_pages8.cu")).read()
    assert "PathPlaces places{first, si.n, n, bs}" in text
    assert "places.moves_end(i1)" in text and "places.slot(from)" in text and "places.slot_end(from, last)" in text
