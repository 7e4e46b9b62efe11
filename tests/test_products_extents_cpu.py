"""More of the host-only half of the products' launcher against brute force, compiled here
by g++ with tests/host/products_extents_check.cpp: where the backward pass of the loss
keeps statistics, float32 sums of long k, and the threads of a launch."""

import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


def test_extents_chains_and_launches(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path / "products_extents_check")
    src = os.path.join(HERE, "host", "products_extents_check.cpp")
    subprocess.run(["g++", "-O1", "-g", "-std=c++17", "-Wall", "-Wextra", "-Werror", src, "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout + out.stderr
