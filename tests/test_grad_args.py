"""Refusals of the gradient norm's entry points and of its classes (no GPU)."""
import ctypes
import math
import os

import pytest
import torch

import mixture_experts_layer_offsets_amd as m
from mixture_experts_layer_offsets_amd import _lib

FAKE, OTHER = 1 << 40, 1 << 44
INVALID, UNSUPPORTED, OK = _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_UNSUPPORTED, _lib.MOE_OK


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from mixture_experts_layer_offsets_amd import build
        build.build(verbose=False)
    return _lib.load()


def tensors(*entries):
    out = (_lib.MoeGradTensor * len(entries))()
    for i, e in enumerate(entries):
        out[i] = _lib.MoeGradTensor(*e)
    return out


def every_call(lib, t, count=None, kind=0, ws=FAKE, n=0, max_norm=1.0):
    """The rc of every entry point; with n = 0 a set that fits ends at the workspace."""
    c = len(t) if count is None else count
    return (lib.moe_grad_norm(c, t, kind, FAKE, FAKE, ws, n, None),
            lib.moe_grad_clip(c, t, kind, max_norm, FAKE, ws, n, None))


def test_sets_outside_the_limits(lib):
    good = (FAKE, OTHER, 100, m.MOE_ROW_F32)
    assert set(every_call(lib, tensors(good))) == {_lib.MOE_ERR_WORKSPACE}
    for bad, code in (((None, OTHER, 100, 2), INVALID), ((FAKE, OTHER, -1, 2), INVALID),
                      ((FAKE, OTHER, 100, 3), INVALID), ((FAKE, OTHER, 100, -1), INVALID),
                      ((FAKE + 2, OTHER, 100, 2), INVALID), ((FAKE + 1, OTHER, 100, 0), INVALID),
                      ((FAKE, OTHER, (1 << 40) + 1, 2), UNSUPPORTED)):
        t = tensors(good, bad)
        assert set(every_call(lib, t)) == {code}, bad
        assert lib.moe_grad_workspace_bytes(2, t) == 0
        assert lib.moe_grad_scale(2, t, 0, FAKE, 1.0, None, None) == code
    # outs: only where they are written
    for out in (None, OTHER + 2, FAKE + 4, FAKE - 396):
        t = tensors((FAKE, out, 100, 2))
        assert every_call(lib, t) == (_lib.MOE_ERR_WORKSPACE, INVALID), out
        assert lib.moe_grad_scale(1, t, 0, FAKE, 1.0, None, None) == INVALID
        assert lib.moe_grad_workspace_bytes(1, t) > 0
    # in place, next to each other, and values of 16 bits at odd places
    for t in (tensors((FAKE, FAKE, 100, 2)), tensors((FAKE, FAKE + 400, 100, 2)), tensors((FAKE + 2, OTHER + 2, 7, 1))):
        assert set(every_call(lib, t)) == {_lib.MOE_ERR_WORKSPACE}
    assert set(every_call(lib, None, count=1)) == {INVALID} and set(every_call(lib, tensors(good), count=-1)) == {INVALID}
    assert set(every_call(lib, tensors(good), count=(1 << 20) + 1)) == {UNSUPPORTED}
    assert set(every_call(lib, tensors(good), kind=2)) == {INVALID}
    assert set(every_call(lib, tensors(good), ws=None)) == {INVALID}
    assert set(every_call(lib, tensors(good), ws=FAKE + 4)) == {INVALID}
    for norm in (-1.0, math.nan):
        assert every_call(lib, tensors(good), max_norm=norm)[1] == INVALID
        assert lib.moe_grad_scale(1, tensors(good), 0, FAKE, norm, None, None) == INVALID
    assert lib.moe_grad_norm(1, tensors(good), 0, None, None, FAKE, 1 << 40, None) == INVALID
    assert lib.moe_grad_scale(1, tensors(good), 0, None, 1.0, None, None) == INVALID


def test_workspace(lib):
    """A partial sum a workgroup, about 2048 in all and no less than 256 a launch."""
    def n(*sizes):
        t = tensors(*[(FAKE, FAKE, s, 2) for s in sizes])
        return lib.moe_grad_workspace_bytes(len(sizes), t)
    assert n() == 256 and n(0) == 256 and n(1) == 256
    assert n(1 << 30) == 2049 * 8 // 256 * 256 + 256
    assert n(*[1 << 24] * 1280) == 10 * 256 * 8 + 256
    assert m.moe_grad_workspace_bytes(tensors()) == 256


def test_sets_check_their_tensors():
    t = torch.zeros((4, 6))
    for grads, outs, what in (
            ([t.double()], None, "float64"), ([t[:, ::2]], None, "dense"), ([t[:, :3]], None, "dense"),
            ([t.expand(2, 4, 6)], None, "dense"), ([t, t], None, "overlap"), ([t, t[1]], None, "overlap"),
            ([t], [t.half()], "type"), ([t], [torch.zeros((6, 4))], "type"), ([t], [torch.zeros((6, 4)).t()], "type"),
            ([t[:2]], [t[1:3]], "overlap"), ([t], [], "outs"),
            ([t[:1], t[1:2]], [torch.zeros((2, 6))[:1], t[:1]], "overlap"),
            ([t], [torch.empty((4, 6), device="meta")], "on meta")):
        with pytest.raises(ValueError, match=what):
            m.GradSet(grads, outs)
    s = m.GradSet([t, torch.zeros((3, 5)).t(), torch.zeros(0), torch.zeros(1)])
    assert len(s) == 4 and [c.numel for c in s.c()] == [24, 15, 0, 1] and s.c()[0].out == t.data_ptr()
    both = m.GradSet([t[:2]], [t[2:]])
    assert both.c()[0].out == t[2:].data_ptr()
    with pytest.raises(ValueError):
        m.GradClip(m.GradSet([]))
    with pytest.raises(ValueError):
        m.GradClip(s, norm_type=3)
    clip = m.GradClip(s)
    for norm in (-1.0, math.nan):
        with pytest.raises(ValueError, match="max_norm"):
            clip(norm)
    for total in (torch.zeros(1), torch.zeros(2, dtype=torch.float64)):
        with pytest.raises(ValueError, match="total"):
            clip.scale(total, 1.0)
