"""The attention kernel's schedule, run on the host (tests/attn_plan_check.cc)."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "speculative_decoding_verification_68_gb300", "csrc")


def test_every_block_is_in_one_run_and_large_schedules_are_cut_right(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path / "attn_plan_check")
    subprocess.check_call([cxx, "-std=c++17", "-O2", "-Wall", "-Werror", "-Wno-unused-function", "-fsanitize=undefined",
                           "-fno-sanitize-recover=undefined", "-I", CSRC, "-o", exe, os.path.join(HERE, "attn_plan_check.cc")])
    done = subprocess.run([exe], stdout=subprocess.PIPE, text=True)
    assert done.returncode == 0 and done.stdout.startswith("ok"), done.stdout


def test_positions_of_the_longest_sequences_fit_32_bits(tmp_path):
    """Every block of a sequence of LEN_MAX tokens, cached or packed, and the three after it."""
    src = tmp_path / "longest.cc"
    src.write_text("""
#include <initializer_list>

#include "attn_plan.cuh"
int main() {
  for (int rows : {1, 2, 16, 25, 128, 256})
    for (int n : {1, 7, 128, 5000, LEN_MAX})
      for (int causal : {0, 1}) {
        const Seq s{0, n, LEN_MAX, (n + rows - 1) / rows, false};
        const int last = tile_blocks(s, s.tiles - 1, rows, causal);
        if (last != (int)((LEN_MAX + 127ll) / 128)) return 1;
        const int next = (last + 2) * BN + BN - 1;       // positions that copies and conversions look ahead to
        if (next < LEN_MAX || tiles_before(s, s.tiles, rows, causal) < last) return 2;
      }
  return 0;
}
""")
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path / "longest")
    subprocess.check_call([cxx, "-std=c++17", "-O1", "-Wno-unused-function", "-fsanitize=undefined", "-fno-sanitize-recover=undefined",
                           "-I", CSRC, "-o", exe, str(src)])
    assert subprocess.run([exe]).returncode == 0
