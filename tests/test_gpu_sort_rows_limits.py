"""The expert-sorted rows at the ends of their limits."""
import os

import pytest
import torch

import mixture_experts_layer_offsets_amd as m
from gpu_util import note

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mixture_experts_layer_offsets_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from mixture_experts_layer_offsets_amd import build
        build.build(verbose=False)
    m.load()


@pytest.mark.parametrize("experts", [1, 64, 65, 1024])
@pytest.mark.parametrize("align", [1, 16])
def test_an_empty_batch_stays_in_its_workspace(experts, align):
    """No tokens: zero counts and offsets, and nothing behind the workspace's
    reported size is written."""
    shape = m.SortShape(0, experts, 3, 64, align=align)
    note(f"empty batch, {experts} experts")
    need = m.moe_sort_workspace_bytes(shape)
    assert need >= 4 * experts
    buf = torch.full((need + 8192,), 0x5A, dtype=torch.uint8, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    empty = torch.empty((0, 3), **i32)
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    for call in (lambda c, o, ws: m.moe_sort_layout(shape, empty, c, o, empty, empty, ws),
                 lambda c, o, ws: m.moe_sort_fwd(shape, x, empty, c, o, empty, empty, x, ws)):
        counts, offsets = torch.full((experts,), -7, **i32), torch.full((experts + 1,), -7, **i32)
        call(counts, offsets, buf[:need])
        assert torch.all(counts == 0) and torch.all(offsets == 0)
        assert torch.all(buf[need:] == 0x5A)
