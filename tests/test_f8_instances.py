"""The library holds no kernel for weights that no call gives it: 8-bit weights go through
the few-token layer's kernels (w4_ffn.hip), not through the 4-bit products' (w4_linear.hip),
whose entry points take 4-bit shapes only."""
import os
import re

import pytest

from mixture_experts_layer_offsets_amd import _lib


@pytest.fixture(scope="module")
def kernels():
    """Names of the library's kernels, as it registers them."""
    if not os.path.exists(_lib.LIB_PATH):
        from mixture_experts_layer_offsets_amd import build
        build.build(verbose=False)
    data = open(_lib.LIB_PATH, "rb").read()
    return {n.decode() for n in re.findall(rb"_ZN3moe[A-Za-z0-9_]+", data)}


def test_formats_of_the_kernels(kernels):
    linear = {n for n in kernels if re.search(r"\dw4_linear(_rows)?_kernel", n)}
    layer = {n for n in kernels if re.search(r"\dw4_(gate_up|down)\w*_kernel", n)}
    for names in (linear, layer):
        assert any("MxFmt" in n for n in names) and any("IntFmt" in n for n in names)
    assert any("F8Fmt" in n for n in layer)
    assert not sorted(n for n in linear if "F8Fmt" in n)
