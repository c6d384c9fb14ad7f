"""Refusals and sizes of the expert-sorted rows' entry points (no GPU: every
call returns before it touches the device), and the checks of TokenSort."""
import ctypes
import dataclasses
import os
import re

import pytest
import torch

import mixture_experts_layer_offsets_amd as m
import rows_oracle as ro
from mixture_experts_layer_offsets_amd import _lib

FAKE = 1 << 40
OK = m.SortShape(16, 8, 4, 64)
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe.h")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from mixture_experts_layer_offsets_amd import build
        build.build(verbose=False)
    return _lib.load()


def every_call(lib, shape, p=FAKE, ws=1 << 40):
    s = None if shape is None else ctypes.byref(shape.c())
    return {
        "layout": lib.moe_sort_layout(s, p, p, p, p, p, p, ws, None),
        "rows": lib.moe_sort_rows(s, p, p, p, p, p, None),
        "fwd": lib.moe_sort_fwd(s, p, p, p, p, p, p, p, p, ws, None),
        "bwd": lib.moe_sort_bwd(s, p, p, p, None),
        "unsort": lib.moe_unsort_fwd(s, p, p, p, p, p, None),
        "unsort_bwd": lib.moe_unsort_bwd(s, p, p, p, p, p, p, p, p, None),
    }


@pytest.mark.parametrize("change,code", [
    (dict(tokens=-1), _lib.MOE_ERR_INVALID_ARG), (dict(experts=0), _lib.MOE_ERR_INVALID_ARG),
    (dict(top_k=0), _lib.MOE_ERR_INVALID_ARG), (dict(width=0), _lib.MOE_ERR_INVALID_ARG),
    (dict(align=-1), _lib.MOE_ERR_INVALID_ARG), (dict(row_type=3), _lib.MOE_ERR_INVALID_ARG),
    (dict(row_type=-1), _lib.MOE_ERR_INVALID_ARG),
    (dict(token_stride=63), _lib.MOE_ERR_INVALID_ARG),
    (dict(row_stride=63), _lib.MOE_ERR_INVALID_ARG),
    (dict(row_stride=-64), _lib.MOE_ERR_INVALID_ARG),
    (dict(experts=1025), _lib.MOE_ERR_UNSUPPORTED), (dict(top_k=17), _lib.MOE_ERR_UNSUPPORTED),
    (dict(align=1025), _lib.MOE_ERR_UNSUPPORTED),
    (dict(tokens=(1 << 24) + 1), _lib.MOE_ERR_UNSUPPORTED),
    (dict(width=(1 << 20) + 1), _lib.MOE_ERR_UNSUPPORTED),
    (dict(token_stride=(1 << 32) + 1), _lib.MOE_ERR_UNSUPPORTED),
])
def test_shapes_outside_the_limits(lib, change, code):
    shape = dataclasses.replace(OK, **change)
    assert set(every_call(lib, shape).values()) == {code}
    assert m.moe_sort_max_rows(shape) == -1 and m.moe_sort_workspace_bytes(shape) == 0
    with pytest.raises(ValueError):
        m.TokenSort(shape, device="cpu")


def test_missing_pointers_and_workspace(lib):
    assert set(every_call(lib, None).values()) == {_lib.MOE_ERR_INVALID_ARG}
    assert set(every_call(lib, OK, p=None).values()) == {_lib.MOE_ERR_INVALID_ARG}
    s = ctypes.byref(OK.c())
    need = m.moe_sort_workspace_bytes(OK)
    for n in (0, need - 1):
        assert lib.moe_sort_layout(s, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, n, None) == \
            _lib.MOE_ERR_WORKSPACE
        assert lib.moe_sort_fwd(s, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, n, None) == \
            _lib.MOE_ERR_WORKSPACE
    # dtopk_w needs y
    assert lib.moe_unsort_bwd(s, FAKE, None, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None) == \
        _lib.MOE_ERR_INVALID_ARG
    # every required pointer by itself
    for i in range(1, 7):
        a = [FAKE] * 6
        a[i - 1] = None
        assert lib.moe_sort_layout(s, *a, 1 << 40, None) == _lib.MOE_ERR_INVALID_ARG
    for i in range(5):
        a = [FAKE] * 5
        a[i] = None
        assert lib.moe_sort_rows(s, *a, None) == _lib.MOE_ERR_INVALID_ARG


def test_no_call_in_place(lib):
    s, bad = ctypes.byref(OK.c()), _lib.MOE_ERR_INVALID_ARG
    p, q, r = FAKE, FAKE + (1 << 30), FAKE + (1 << 31)
    assert lib.moe_sort_rows(s, p, q, q, q, p, None) == bad
    assert lib.moe_sort_fwd(s, p, q, q, q, q, q, p, q, 1 << 40, None) == bad
    assert lib.moe_sort_bwd(s, p, q, p, None) == bad
    assert lib.moe_unsort_fwd(s, p, q, q, None, p, None) == bad
    assert lib.moe_unsort_fwd(s, r, q, q, p, p, None) == bad
    assert lib.moe_unsort_bwd(s, p, r, q, q, q, q, p, q, None) == bad
    assert lib.moe_unsort_bwd(s, r, p, q, q, q, q, p, q, None) == bad


def test_sizes(lib):
    assert m.moe_sort_max_rows(OK) == 64
    assert m.moe_sort_max_rows(dataclasses.replace(OK, align=16)) == 64 + 8 * 15
    assert m.moe_sort_max_rows(dataclasses.replace(OK, tokens=1, top_k=3, align=16)) == 3 + 3 * 15
    assert m.moe_sort_max_rows(dataclasses.replace(OK, tokens=0, align=16)) == 0
    assert m.moe_sort_workspace_bytes(OK) % 256 == 0 and m.moe_sort_workspace_bytes(OK) > 0
    # bounded histograms: the workspace does not grow with the token count
    big = m.SortShape(1 << 24, 1024, 16, 64)
    assert m.moe_sort_workspace_bytes(big) <= (128 * 1024 + 1) * 4 + 256


def test_struct_matches_header(lib):
    text = open(HEADER).read()
    body = re.search(r"typedef struct moe_sort_shape \{(.*?)\} moe_sort_shape;", text, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    fields = [(d.split()[0], d.split()[1]) for d in body.split(";")[:-1]]
    ct = {"int32_t": ctypes.c_int32, "int64_t": ctypes.c_int64}
    assert [(n, ct[t]) for t, n in fields] == _lib.MoeSortShape._fields_


def test_token_sort_checks_its_tensors():
    shape = m.SortShape(6, 4, 2, 16, align=2, token_stride=20)
    op = m.TokenSort(shape, device="cpu")
    x, idx = op.token_rows(), torch.zeros((6, 2), dtype=torch.int32)
    assert x.stride() == (20, 1) and op.sorted_rows().shape == (12 + 4, 16)
    w = torch.zeros((6, 2))
    bad = [lambda: op.sort(x[:5], idx), lambda: op.sort(x.contiguous(), idx),
           lambda: op.sort(x.float(), idx), lambda: op.sort(x, idx.long()),
           lambda: op.sort(x, idx.t().contiguous().t()), lambda: op.sort(x, idx, out=x),
           lambda: op.unsort(x, w), lambda: op.unsort(op.sorted_rows(), w.double()),
           lambda: op.unsort(op.sorted_rows(), w, add=op.sorted_rows()),
           lambda: op.unsort_backward(op.sorted_rows(), op.sorted_rows(), w),
           lambda: op.unsort_backward(x, op.sorted_rows(), w[:, :1]),
           lambda: op.sort_backward(x), lambda: op.sort_again(op.sorted_rows()),
           lambda: op.sort(torch.empty_like(x, device="meta"), idx)]
    for call in bad:
        with pytest.raises(ValueError):
            call()


def test_plain_layout_is_the_definition():
    """The tests' own plain layout on a case worked by hand."""
    import numpy as np
    idx = np.array([[7, 5], [5, 9], [-1, 7], [6, 5]], np.int32)
    counts, offsets, perm, inv = ro.layout(idx, 3, first=5, align=4)
    assert counts.tolist() == [3, 1, 2] and offsets.tolist() == [0, 4, 8, 12]
    assert perm.tolist() == [1, 2, 7, -1, 6, -1, -1, -1, 0, 5, -1, -1] + [-1] * 5
    assert inv.tolist() == [[8, 0], [1, -1], [-1, 9], [4, 2]]
    assert ro.padding_rows(counts, offsets).tolist() == [3, 5, 6, 7, 10, 11]
