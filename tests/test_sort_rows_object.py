"""TokenSort's own layout, on the host."""
import contextlib
import os

import pytest
import torch

import mixture_experts_layer_offsets_amd as m
from mixture_experts_layer_offsets_amd import _lib


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not os.path.exists(_lib.LIB_PATH):
        from mixture_experts_layer_offsets_amd import build
        build.build(verbose=False)
    m.load()


@pytest.mark.parametrize("tokens", [0, 6])
def test_nothing_moves_before_the_first_sort(tokens):
    """The layout of a new object is whatever lay in its memory: calls that
    would take row numbers from it are refused."""
    op = m.TokenSort(m.SortShape(tokens, 4, 2, 16, align=8), device="cpu")
    x, y, w = op.token_rows(), op.sorted_rows(), torch.ones((tokens, 2))
    for call in (lambda: op.sort_again(x), lambda: op.sort_backward(y), lambda: op.unsort(y),
                 lambda: op.unsort(y, w, add=x), lambda: op.unsort_backward(x, y, w)):
        with pytest.raises(ValueError, match="no layout"):
            call()


def test_the_first_sort_makes_the_layout(monkeypatch):
    """... and a sort that the library refuses does not."""
    op = m.TokenSort(m.SortShape(6, 4, 2, 16), device="cpu")
    x, idx = op.token_rows(), torch.zeros((6, 2), dtype=torch.int32)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    calls = []

    def refuse(*a):
        raise _lib.MoeError(_lib.MOE_ERR_HIP, "moe_sort_fwd")
    monkeypatch.setattr(_lib, "moe_sort_fwd", refuse)
    with pytest.raises(m.MoeError):
        op.sort(x, idx)
    with pytest.raises(ValueError, match="no layout"):
        op.sort_again(x)
    for name in ("moe_sort_fwd", "moe_sort_rows", "moe_sort_bwd", "moe_unsort_fwd", "moe_unsort_bwd"):
        monkeypatch.setattr(_lib, name, lambda *a, name=name: calls.append(name))
    xs = op.sort(x, idx)
    op.sort_again(x)
    op.sort_backward(xs)
    op.unsort(xs)
    op.unsort_backward(x, xs, torch.ones((6, 2)))
    assert calls == ["moe_sort_fwd", "moe_sort_rows", "moe_sort_bwd", "moe_unsort_fwd", "moe_unsort_bwd"]


def test_the_unweighted_return_has_a_gradient(monkeypatch):
    """unsort without weights: dy by the rows' copy, no dtopk_w; a buffer for it
    has nothing to be filled with."""
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    calls = []
    for name in ("moe_sort_fwd", "moe_sort_rows", "moe_unsort_bwd"):
        monkeypatch.setattr(_lib, name, lambda *a, name=name: calls.append(name))
    op = m.TokenSort(m.SortShape(6, 4, 2, 16), device="cpu")
    dout, y = op.token_rows(), op.sort(op.token_rows(), torch.zeros((6, 2), dtype=torch.int32))
    dy = op.sorted_rows()
    got, dw = op.unsort_backward(dout, y, None, dy=dy)
    assert got is dy and dw is None and calls == ["moe_sort_fwd", "moe_sort_rows"]
    with pytest.raises(ValueError, match="dtopk_w"):
        op.unsort_backward(dout, y, None, dtopk_w=torch.empty((6, 2)))
    with pytest.raises(ValueError):
        op.unsort_backward(dout, y[:-1], None)
