"""The host-only half of the row operators' launcher (extents, overlap, limits,
spreads; precision_optimizer_state_amd/csrc/fo_rows_args.hpp) against brute
force, under AddressSanitizer and UndefinedBehaviorSanitizer, compiled here by
g++ with tests/host/rows_args_check.cpp."""

import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
SRC = os.path.join(HERE, "host", "rows_args_check.cpp")


def test_extents_overlap_and_spreads(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path / "rows_args_check")
    subprocess.run(["g++", "-O1", "-g", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=all", SRC, "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=120,
                         env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout + out.stderr
