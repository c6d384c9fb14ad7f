"""The launch shapes of the expert-sorted rows, checked on the host.

tests/sort_grid_check.cpp compiles the library's own grid functions
(mixture_experts_layer_offsets_amd/csrc/sort_grid.h) with g++ and walks them
over tokens up to 2^24, rows of 16 bytes to 4 MiB, and up to 1024 experts with
and without padding rows.
"""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


def test_every_accepted_size_has_a_grid(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path / "sort_grid_check")
    subprocess.run([gxx, "-O2", "-std=c++17", "-Wall", "-Werror", "-o", exe,
                    os.path.join(HERE, "sort_grid_check.cpp")], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout[-4000:]
    assert r.stdout.strip() == "ok"
