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
