"""LDS passed between a wave's lanes: by a barrier that the compiler moves no
access across.  __builtin_amdgcn_wave_barrier touches no memory as far as the
compiler knows, so it orders nothing by itself; kernels use wave_lds_sync,
which puts it between a release and an acquire fence of the wave."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "mixture_experts_layer_offsets_amd", "csrc")


def test_wave_barriers_stand_between_fences():
    seen = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        lines = open(path).read().splitlines()
        for i, line in enumerate(lines):
            if "__builtin_amdgcn_wave_barrier" in line:
                seen += 1
                where = f"{os.path.basename(path)}:{i + 1}"
                assert re.search(r'amdgcn_fence\(__ATOMIC_RELEASE, "wavefront"\)', lines[i - 1]), where
                assert re.search(r'amdgcn_fence\(__ATOMIC_ACQUIRE, "wavefront"\)', lines[i + 1]), where
    assert seen
