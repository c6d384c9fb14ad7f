"""Sizes of the expert-sorted rows at the ends of their limits, on the host."""
import os

import pytest

import mixture_experts_layer_offsets_amd as m
from mixture_experts_layer_offsets_amd import _lib


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not os.path.exists(_lib.LIB_PATH):
        from mixture_experts_layer_offsets_amd import build
        build.build(verbose=False)
    m.load()


@pytest.mark.parametrize("tokens", [0, 1, 1023, 1025, 1 << 17, 1 << 24])
@pytest.mark.parametrize("experts", [1, 64, 65, 128, 1024])
def test_the_workspace_holds_a_histogram_for_every_1024_slots(tokens, experts):
    """An empty batch still counts into one histogram of `experts` words; at
    most 128 histograms."""
    need = 4 * experts * min(128, max(1, -(-tokens // 1024)))
    assert m.moe_sort_workspace_bytes(m.SortShape(tokens, experts, 1, 64)) >= need
