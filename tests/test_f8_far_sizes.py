"""Sizes past 32 bits at the 8-bit products' entry points: refused, not taken by their low
bits (no GPU: every call returns before it touches the device)."""
import os

import pytest
import torch

import mixture_experts_layer_offsets_amd as m
from mixture_experts_layer_offsets_amd import _lib

FAKE, OTHER = 1 << 40, 1 << 48
S = m.F8Shape(1, 48, 256)


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from mixture_experts_layer_offsets_amd import build
        build.build(verbose=False)
    return _lib.load()


class Rows:
    """A tensor of so many rows, as far as the binding looks."""

    def __init__(self, rows, width, at=FAKE):
        self.shape, self._at = (rows, width), at

    def data_ptr(self):
        return self._at

    def stride(self, dim):
        return (self.shape[1], 1)[dim]

    def numel(self):
        return 1 << 60

    def element_size(self):
        return 1


FAR = pytest.mark.parametrize("rows", [1 << 31, (1 << 32) + 5, (1 << 40) + 1])


@FAR
def test_rows(rows):
    assert m.moe_f8_linear_workspace_bytes(S, rows) == 0 and m.moe_f8_wgrad_workspace_bytes(S, rows) == 0
    ws = Rows(1, 1)
    for call in (lambda: m.moe_f8_linear(S, Rows(rows, 256), None, FAKE, Rows(rows, 48, OTHER), ws, 0),
                 lambda: m.moe_f8_linear_codes(S, FAKE, FAKE, None, FAKE, Rows(rows, 48, OTHER), 0),
                 lambda: m.moe_f8_wgrad(S, Rows(rows, 256), Rows(rows, 48), None, OTHER, ws, 0),
                 lambda: m.moe_f8_quantize_rows(S, Rows(rows, 256), FAKE, FAKE, 0)):
        with pytest.raises(m.MoeError) as e:
            call()
        assert e.value.code == _lib.MOE_ERR_UNSUPPORTED
    lin = m.F8Linear(S, torch.empty(m.moe_f8_bytes(S), dtype=torch.uint8))
    x = torch.empty((rows, 256), dtype=torch.bfloat16, device="meta")
    lin.packed = lin.packed.to("meta")
    with pytest.raises(ValueError, match="limits"):
        lin(x)
    with pytest.raises(ValueError, match="limits"):
        lin.weight_gradient(x, torch.empty((rows, 48), dtype=torch.bfloat16, device="meta"))


@FAR
@pytest.mark.parametrize("field", ["groups", "n", "k", "row_type"])
def test_shapes(field, rows):
    for value in (rows, -rows):
        sizes = dict(groups=1, n=48, k=256, row_type=m.MOE_ROW_BF16)
        sizes[field] = value
        assert m.moe_f8_bytes(m.F8Shape(**sizes)) == 0


def test_first_expert():
    """An expert that no 32-bit id names is not expert 0."""
    e = m.F8Experts(*[torch.zeros(1)] * 3, first_expert=1 << 32)
    assert e.c().first_expert == (1 << 31) - 1
    assert m.F8Experts(*[torch.zeros(1)] * 3, first_expert=-3).c().first_expert == -3


@pytest.mark.parametrize("change", [dict(row_type=m.MOE_ROW_F32), dict(row_type=7), dict(groups=0), dict(n=1 << 21)])
def test_weight_gradient_of_a_refused_shape(change):
    """The class's own error, before its tensors are looked at."""
    sizes = {**dict(groups=1, n=48, k=256, row_type=m.MOE_ROW_BF16), **change}
    lin = m.F8Linear(m.F8Shape(**sizes), torch.empty(0, dtype=torch.uint8))
    with pytest.raises(ValueError, match="limits"):
        lin.weight_gradient(torch.zeros((3, 256)), torch.zeros((3, 48)))
