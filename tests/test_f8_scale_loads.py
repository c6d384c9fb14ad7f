"""The loads of scales in the 8-bit weight gradient's loop stay inside the buffer.

tests/f8_scales_check.cpp compiles the kernel's own address functions
(csrc/f8_scales.h) with g++.  What a buffer's range check covers is the vector offset
and the constant one, so the kernel's loads into LDS keep to those: their scalar
offset is zero."""
import os
import re
import shutil
import subprocess

import pytest

import mixture_experts_layer_offsets_amd as m

HERE = os.path.dirname(os.path.abspath(__file__))
SOURCE = os.path.join(os.path.dirname(HERE), "mixture_experts_layer_offsets_amd", "csrc", "f8_gemm.hip")


def test_addresses(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path / "f8_scales_check")
    subprocess.run([gxx, "-O2", "-std=c++17", "-Wall", "-Werror", "-o", exe,
                    os.path.join(HERE, "f8_scales_check.cpp")], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout[-4000:]
    assert r.stdout.strip() == "ok"


def test_no_scalar_offsets():
    text = re.sub(r"//[^\n]*", "", open(SOURCE).read())
    calls = re.findall(r"raw_ptr_buffer_load_lds\((.*?)\);", text, re.S)
    assert calls
    for call in calls:
        depth, args = 0, [""]
        for ch in call:
            depth += (ch in "([") - (ch in ")]")
            if ch == "," and not depth:
                args.append("")
            else:
                args[-1] += ch
        # resource, LDS address, size, vector offset, scalar offset, constant offset, flags
        assert len(args) == 7 and args[4].strip() == "0", call


@pytest.mark.parametrize("n", [1, 16, 17, 255, 256, 257, 272, 273, 300, 512])
@pytest.mark.parametrize("rows", [1000, 2049, 3000])
def test_last_stage_ends_in_the_workspace(n, rows):
    """The stages' scales [stage][columns rounded up to 16], and what lies before them."""
    groups, k = 1, 272
    stages, cols = rows // 128 + groups, -(-n // 16) * 16
    up = lambda v: -(-v // 256) * 256  # noqa: E731
    before = up(stages * k * 128) + up(stages * (-(-k // 16) * 16) * 4) + up(stages * cols * 128)
    last = before + 4 * ((stages - 1) * cols + cols)
    assert last <= m.moe_f8_wgrad_workspace_bytes(m.F8Shape(groups, n, k), rows)
